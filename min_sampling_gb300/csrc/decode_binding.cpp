// Python entries of the decode step: argument checks and marshalling of torch tensors for
// the C ABI, in C++.
//
// These calls run once or more per generated token, often on a few rows, where the host's
// time decides: with the checks in Python a call took 21 to 31 us of the host for kernels of 3 to 13;
// here it takes 5 to 11 (Grace).  Nothing is computed and nothing kept from one call for the
// next.  Every function returns its result, or an fs_status other than FS_OK as an int, which the caller in
// __init__.py raises.
#include <torch/csrc/Exceptions.h>
#include <torch/csrc/autograd/python_variable.h>

#include <ATen/core/grad_mode.h>
#include <ATen/ops/empty.h>
#include <ATen/ops/full.h>
#include <c10/core/DeviceGuard.h>
#include <c10/cuda/CUDAStream.h>

#include <algorithm>
#include <cmath>
#include <cstdint>
#include <initializer_list>
#include <string>
#include <utility>

#include "fs_sampling.h"

namespace {

struct Refused {
    std::string what;
};

[[noreturn]] void refuse(const std::string& what) { throw Refused{what}; }

bool none(PyObject* o) { return o == nullptr || o == Py_None; }

const at::Tensor* tensor(PyObject* o) { return THPVariable_Check(o) ? &THPVariable_Unpack(o) : nullptr; }

int dtype_of(at::ScalarType t) {
    switch (t) {
        case at::kFloat: return FS_F32;
        case at::kBFloat16: return FS_BF16;
        case at::kHalf: return FS_F16;
        default: return -1;
    }
}

std::string shape_text(at::IntArrayRef s) {
    std::string r = "[";
    for (size_t i = 0; i < s.size(); ++i) r += (i ? ", " : "") + (s[i] < 0 ? std::string("*") : std::to_string(s[i]));
    return r + "]";
}

// A CUDA tensor of a type the entries take, of lo to hi dimensions.
const at::Tensor& float_cuda(PyObject* o, const char* name, int lo, int hi) {
    const at::Tensor* t = tensor(o);
    if (!t || t->dim() < lo || t->dim() > hi)
        refuse(std::string(name) + " must be a " + (lo == hi ? "" : std::to_string(lo) + "-D or ") + std::to_string(hi) +
               "-D tensor");
    if (dtype_of(t->scalar_type()) < 0 || !t->is_cuda())
        refuse(std::string(name) + " must be a float32, bfloat16 or float16 CUDA tensor");
    return *t;
}

bool matches(const at::Tensor& t, at::IntArrayRef shape, at::ScalarType type, c10::DeviceIndex dev) {
    if (!t.is_cuda() || t.get_device() != dev || t.scalar_type() != type || t.dim() != int64_t(shape.size())) return false;
    for (size_t i = 0; i < shape.size(); ++i)
        if (shape[i] >= 0 && t.size(i) != shape[i]) return false;  // -1: any
    return true;
}

// A tensor of vectors (contiguous last dimension) of the given shape, type and device.
const at::Tensor& vectors(PyObject* o, const char* name, at::IntArrayRef shape, at::ScalarType type, c10::DeviceIndex dev) {
    const at::Tensor* t = tensor(o);
    if (!t || !matches(*t, shape, type, dev))
        refuse(std::string(name) + " must be a " + shape_text(shape) + " " + c10::toString(type) + " tensor on cuda:" +
               std::to_string(int(dev)));
    if (t->size(-1) > 1 && t->stride(-1) != 1) refuse(std::string(name) + "'s last dimension must be contiguous");
    return *t;
}

// A contiguous tensor of the given shape (-1: any size), type and device.
const at::Tensor& flat(PyObject* o, const char* name, at::IntArrayRef shape, at::ScalarType type, c10::DeviceIndex dev) {
    const at::Tensor* t = tensor(o);
    if (!t || !matches(*t, shape, type, dev) || !t->is_contiguous())
        refuse(std::string(name) + " must be a contiguous " + shape_text(shape) + " " + c10::toString(type) +
               " tensor on cuda:" + std::to_string(int(dev)));
    return *t;
}

template <typename X>
const X* flat_ptr(PyObject* o, const char* name, int64_t n, at::ScalarType type, c10::DeviceIndex dev) {
    return none(o) ? nullptr : static_cast<const X*>(flat(o, name, {n}, type, dev).data_ptr());
}

// Strides of the first n dimensions, 0 for a dimension of one element (its stride addresses nothing).
void strides(const at::Tensor& t, int n, int64_t* out) {
    for (int i = 0; i < n; ++i) out[i] = t.size(i) > 1 ? t.stride(i) : 0;
}

// ------------------------------------------------------------------ shared memory
//
// Two elements at index i of one tensor and j of another (or of the same) lie at one address where
//   sum_d i_d s_d - sum_d j_d t_d = the distance of their first elements,
// an equation in bounded integers.  Its terms are searched from the largest stride down: each coefficient has to leave a rest
// that the smaller terms can reach, which leaves one or two values for strides that nest (a
// dimension's stride is at least the extent of the smaller ones), as those of nearly all views do.

struct Term {
    int64_t stride, lo, hi;   // coefficients lo .. hi, lo <= 0 <= hi
};

struct Terms {
    Term t[16];
    int n = 0;
    void add(int64_t stride, int64_t lo, int64_t hi) {
        if (stride == 0 || lo == hi) return;
        int i = n;
        for (int j = 0; j < n; ++j)
            if (t[j].stride == stride) {
                t[j].lo += lo, t[j].hi += hi;
                return;
            }
        for (; i > 0 && t[i - 1].stride < stride; --i) t[i] = t[i - 1];
        t[i] = Term{stride, lo, hi};
        ++n;
    }
};

int64_t floor_div(int64_t a, int64_t b) { return a / b - (a % b != 0 && (a < 0) != (b < 0)); }

// Whether the terms from i on can sum to `rest`, with a coefficient other than 0 if `other` asks for one.  `tries` bounds the
// search; when it runs out the answer is yes.
bool reaches(const Terms& e, int i, int64_t rest, bool other, int& tries) {
    if (--tries < 0) return true;
    if (i == e.n) return rest == 0 && !other;
    int64_t least = 0, most = 0;   // of the smaller terms
    for (int j = i + 1; j < e.n; ++j) least += e.t[j].lo * e.t[j].stride, most += e.t[j].hi * e.t[j].stride;
    const Term& x = e.t[i];
    const int64_t from = std::max(x.lo, -floor_div(most - rest, x.stride)), to = std::min(x.hi, floor_div(rest - least, x.stride));
    for (int64_t c = from; c <= to; ++c)
        if (reaches(e, i + 1, rest - c * x.stride, other && c == 0, tries)) return true;
    return false;
}

constexpr int TRIES = 4096;

// A tensor's sizes, strides and the bytes from its first element to its last.
struct Span {
    const int64_t *sizes, *strides;
    int dims;
    intptr_t first, end;   // equal: no elements
    int64_t element;
    explicit Span(const at::Tensor& t) : sizes(t.sizes().data()), strides(t.strides().data()), dims(int(t.dim())), element(t.element_size()) {
        first = end = reinterpret_cast<intptr_t>(t.const_data_ptr());
        int64_t last = 0;
        for (int i = 0; i < dims; ++i) {
            if (sizes[i] == 0) return;
            last += (sizes[i] - 1) * strides[i];
        }
        end += (last + 1) * element;
    }
};

bool overlaps_itself(const Span& t) {
    if (t.first == t.end) return false;
    if (t.dims > 16) return true;
    Terms e;
    int dims = 0;
    for (int i = 0; i < t.dims; ++i) {
        if (t.sizes[i] < 2) continue;
        if (t.strides[i] == 0) return true;
        e.add(t.strides[i], 1 - t.sizes[i], t.sizes[i] - 1);
        ++dims;
    }
    if (dims != e.n) return true;   // two dimensions of one stride
    int64_t reach = 0;
    int i = e.n;
    for (; i > 0 && e.t[i - 1].stride > reach; --i) reach += e.t[i - 1].hi * e.t[i - 1].stride;
    if (i == 0) return false;       // the strides nest
    int tries = TRIES;
    return reaches(e, 0, 0, true, tries);
}

// (tensors of one element size)
bool shares_memory(const Span& a, const Span& b) {
    if (a.first == a.end || b.first == b.end || a.first >= b.end || b.first >= a.end) return false;
    if ((b.first - a.first) % a.element != 0 || a.dims + b.dims > 16) return true;
    Terms e;
    for (int i = 0; i < a.dims; ++i) e.add(a.strides[i], 0, a.sizes[i] - 1);
    for (int i = 0; i < b.dims; ++i) e.add(b.strides[i], 1 - b.sizes[i], 0);
    int tries = TRIES;
    return reaches(e, 0, (b.first - a.first) / a.element, false, tries);
}

bool same_view(const Span& a, const Span& b) {
    if (a.first != b.first || a.dims != b.dims) return false;
    for (int i = 0; i < a.dims; ++i)
        if (a.sizes[i] != b.sizes[i] || (a.sizes[i] > 1 && a.strides[i] != b.strides[i])) return false;
    return true;
}

// A tensor that is written: no two of its elements at one address, ...
void writable(const Span& t, const char* name) {
    if (overlaps_itself(t)) refuse(std::string(name) + " is written, but some of its elements share memory");
}
// ... and none where another tensor of the call has one.
void apart(const Span& written, const char* name, const Span& other, const char* other_name) {
    if (shares_memory(written, other)) refuse(std::string(name) + " is written, but shares memory with " + other_name);
}

// There is no backward pass and no forward-mode derivative: either would be lost without a word.
void no_gradient(std::initializer_list<const at::Tensor*> ts) {
    for (const at::Tensor* t : ts)
        if (t && t->_fw_grad(0).defined())
            refuse("there is no forward-mode derivative: take the primal of tensors with a tangent (torch.autograd.forward_ad.unpack_dual)");
    if (!at::GradMode::is_enabled()) return;
    for (const at::Tensor* t : ts)
        if (t && t->requires_grad()) refuse("there is no backward pass: detach tensors that require a gradient, or call under torch.no_grad()");
}

// The caller's tensors that a launch has written: autograd learns that what it saved of them has changed.
void written(std::initializer_list<const at::Tensor*> ts) {
    for (const at::Tensor* t : ts)
        if (t && !t->is_inference()) t->unsafeGetTensorImpl()->bump_version();
}

fs_paged_kv paged_kv(PyObject* k, PyObject* v) {
    const at::Tensor& kt = float_cuda(k, "k_cache", 4, 4);
    vectors(k, "k_cache", kt.sizes(), kt.scalar_type(), kt.get_device());
    const at::Tensor& vt = vectors(v, "v_cache", kt.sizes(), kt.scalar_type(), kt.get_device());
    if (kt.size(1) < 1 || kt.size(2) < 1 || kt.size(3) < 1)
        refuse("the caches must be [num_pages, page_size, num_heads, head_dim] with at least one element a page");
    for (int i = 0; i < 4; ++i)
        if (kt.size(i) > INT32_MAX) refuse("the caches are too large in one dimension");
    fs_paged_kv kv;
    kv.k = kt.data_ptr();
    kv.v = vt.data_ptr();
    kv.dtype = dtype_of(kt.scalar_type());
    kv.num_pages = int32_t(kt.size(0));
    kv.page_size = int32_t(kt.size(1));
    kv.num_heads = int32_t(kt.size(2));
    kv.head_dim = int32_t(kt.size(3));
    strides(kt, 3, kv.k_strides);
    strides(vt, 3, kv.v_strides);
    return kv;
}

int32_t size32(int64_t n, const char* what) {
    if (n > INT32_MAX) refuse(std::string(what) + " is too large");
    return int32_t(n);
}

at::Tensor scratch(size_t bytes, const at::Tensor& like) {
    return at::empty({int64_t(bytes)}, like.options().dtype(at::kByte));
}

// Runs `f(stream)` with the device current; FS_OK -> `ok()`.
template <typename F, typename R>
PyObject* launch(const at::Tensor& on, F f, R ok) {
    const fs_status st = f(static_cast<void*>(c10::cuda::getCurrentCUDAStream(on.get_device()).stream()));
    return st == FS_OK ? ok() : PyLong_FromLong(st);
}

// A refusal becomes a ValueError; what torch throws (out of memory, say) its own Python error.
template <typename F>
PyObject* guarded(F f) {
    HANDLE_TH_ERRORS
    try {
        return f();
    } catch (const Refused& r) {
        PyErr_SetString(PyExc_ValueError, r.what.c_str());
        return nullptr;
    }
    END_HANDLE_TH_ERRORS
}

struct py_owned {
    PyObject* p;
    explicit py_owned(PyObject* o) : p(o) {}
    ~py_owned() { Py_XDECREF(p); }
};

PyObject* wrap(at::Tensor t) { return THPVariable_Wrap(std::move(t)); }

PyObject* pair(at::Tensor x, at::Tensor y) {
    PyObject* r = PyTuple_New(2);
    if (r) {
        PyTuple_SET_ITEM(r, 0, wrap(std::move(x)));
        PyTuple_SET_ITEM(r, 1, wrap(std::move(y)));
    }
    return r;
}

bool arity(Py_ssize_t n, Py_ssize_t want) {
    if (n == want) return true;
    PyErr_SetString(PyExc_TypeError, "wrong number of arguments");
    return false;
}

// (logits, uniforms, temperature, top_k, top_p, min_p, order, indices) -> (tokens, valid)
PyObject* from_uniforms(PyObject*, PyObject* const* a, Py_ssize_t n) {
    if (!arity(n, 8)) return nullptr;
    return guarded([&]() -> PyObject* {
        const at::Tensor& x = float_cuda(a[0], "logits", 2, 2);
        const int64_t b_in = x.size(0), V = x.size(1), stride = b_in > 1 ? x.stride(0) : V;
        const auto dev = x.get_device();
        if (V < 1 || (V > 1 && x.stride(1) != 1) || stride < V)
            refuse("logits must have at least one column, contiguous columns and rows that do not overlap");
        const at::Tensor* idx = none(a[7]) ? nullptr : &flat(a[7], "indices", {-1}, at::kInt, dev);
        const int32_t b_out = size32(idx ? idx->size(0) : b_in, "the batch");
        const c10::DeviceGuard guard(x.device());
        const auto* u = flat_ptr<float>(a[1], "uniforms", b_out, at::kFloat, dev);
        if (!u && none(a[1])) refuse("uniforms must be given");
        // Per-row parameters; a number is the same for every row.
        at::Tensor held[4];
        const void* ps[4];
        static const char* const names[4] = {"temperature", "top_k", "top_p", "min_p"};
        for (int i = 0; i < 4; ++i) {
            PyObject* o = a[2 + i];
            const auto type = i == 1 ? at::kInt : at::kFloat;
            ps[i] = nullptr;
            if (none(o)) continue;
            if (!tensor(o)) {
                const double v = PyFloat_AsDouble(o);
                if (v == -1.0 && PyErr_Occurred()) return nullptr;
                held[i] = at::full({b_out}, v, x.options().dtype(type));
                ps[i] = held[i].data_ptr();
            } else {
                ps[i] = flat(o, names[i], {b_out}, type, dev).data_ptr();
            }
        }
        const long order = PyLong_AsLong(a[6]);
        if (order == -1 && PyErr_Occurred()) return nullptr;
        const int dtype = dtype_of(x.scalar_type());
        size_t need = 0;
        const fs_status st = fs_from_uniforms_workspace_bytes(dtype, size32(b_in, "the batch"), size32(V, "the vocabulary"), &need);
        if (st != FS_OK) return PyLong_FromLong(st);
        const at::Tensor ws = scratch(need, x);
        at::Tensor tok = at::empty({b_out}, x.options().dtype(at::kInt)), valid = at::empty({b_out}, x.options().dtype(at::kByte));
        return launch(x, [&](void* s) {
            return fs_top_k_top_p_sampling_from_uniforms(
                x.data_ptr(), dtype, stride, int32_t(b_in), int32_t(V), idx ? static_cast<const int32_t*>(idx->data_ptr()) : nullptr,
                b_out, u, static_cast<const float*>(ps[0]), static_cast<const int32_t*>(ps[1]), static_cast<const float*>(ps[2]),
                static_cast<const float*>(ps[3]), int32_t(order), static_cast<int32_t*>(tok.data_ptr()),
                static_cast<uint8_t*>(valid.data_ptr()), ws.data_ptr(), need, s);
        }, [&] { return pair(tok, valid); });
    });
}

// (key, value, k_cache, v_cache, page_table, positions, rows, rotary_positions, inv_freq, interleaved, query, query_out)
// -> query_out or None
PyObject* append(PyObject*, PyObject* const* a, Py_ssize_t n) {
    if (!arity(n, 12)) return nullptr;
    return guarded([&]() -> PyObject* {
        const fs_paged_kv kv = paged_kv(a[2], a[3]);
        const at::Tensor& cache = *tensor(a[2]);
        const auto type = cache.scalar_type();
        const auto dev = cache.get_device();
        const at::Tensor& key = vectors(a[0], "key", {-1, kv.num_heads, kv.head_dim}, type, dev);
        const int32_t tokens = size32(key.size(0), "the number of tokens");
        const at::Tensor& value = vectors(a[1], "value", {tokens, kv.num_heads, kv.head_dim}, type, dev);
        const at::Tensor& table = flat(a[4], "page_table", {-1, -1}, at::kInt, dev);
        const auto* pos = static_cast<const int32_t*>(flat(a[5], "positions", {tokens}, at::kInt, dev).data_ptr());
        const auto* rows = flat_ptr<int32_t>(a[6], "rows", tokens, at::kInt, dev);
        if (none(a[6]) && table.size(0) < tokens) refuse("page_table needs a row for every token when rows is not given");
        const auto* rpos = flat_ptr<int32_t>(a[7], "rotary_positions", tokens, at::kInt, dev);
        const auto* freq = flat_ptr<float>(a[8], "inv_freq", -1, at::kFloat, dev);
        const int64_t rotary = none(a[8]) ? 0 : 2 * tensor(a[8])->size(0);
        if (rotary > kv.head_dim) refuse("inv_freq has more pairs than a head");
        const int interleaved = PyObject_IsTrue(a[9]);
        if (interleaved < 0) return nullptr;
        int64_t ks[2], vs[2], qs[2] = {0, 0}, qos[2] = {0, 0};
        strides(key, 2, ks);
        strides(value, 2, vs);
        const c10::DeviceGuard guard(cache.device());
        const at::Tensor* q = nullptr;
        at::Tensor qo;
        int32_t q_heads = 0;
        if (!none(a[10])) {
            q = &vectors(a[10], "query", {tokens, -1, kv.head_dim}, type, dev);
            q_heads = size32(q->size(1), "the number of heads");
            if (q_heads < 1) refuse("query must have at least one head");
            qo = none(a[11]) ? at::empty(q->sizes(), q->options()) : vectors(a[11], "query_out", q->sizes(), type, dev);
            strides(*q, 2, qs);
            strides(qo, 2, qos);
        } else if (!none(a[11])) {
            refuse("query_out needs a query");
        }
        const at::Tensor& v_cache = *tensor(a[3]);
        const Span k_span(cache), v_span(v_cache), in_key(key), in_value(value);
        writable(k_span, "k_cache");
        writable(v_span, "v_cache");
        apart(k_span, "k_cache", v_span, "v_cache");
        auto off_caches = [&](const Span& t, const char* name) {
            apart(k_span, "k_cache", t, name);
            apart(v_span, "v_cache", t, name);
        };
        off_caches(in_key, "key");
        off_caches(in_value, "value");
        if (q) {
            const Span in_query(*q);
            off_caches(in_query, "query");
            if (!none(a[11])) {
                const Span to(qo);
                writable(to, "query_out");
                off_caches(to, "query_out");
                apart(to, "query_out", in_key, "key");
                apart(to, "query_out", in_value, "value");
                if (!same_view(in_query, to)) apart(to, "query_out", in_query, "query");
            }
        }
        no_gradient({&key, &value, &cache, tensor(a[3]), q, tensor(a[11])});
        return launch(cache, [&](void* s) {
            return fs_append_paged_kv(&kv, key.data_ptr(), ks, value.data_ptr(), vs, tokens,
                                      static_cast<const int32_t*>(table.data_ptr()), size32(table.size(0), "the table"),
                                      size32(table.size(1), "the table"), rows, pos, rpos, freq, int32_t(rotary), interleaved,
                                      q ? q->data_ptr() : nullptr, qs, q_heads, q ? qo.data_ptr() : nullptr, qos, s);
        }, [&]() -> PyObject* {
            written({&cache, &v_cache, tensor(a[11])});
            if (!q) Py_RETURN_NONE;
            if (none(a[11])) return wrap(qo);
            Py_INCREF(a[11]);
            return a[11];
        });
    });
}

// (query, k_cache, v_cache, prefix_table, prefix_lens, suffix_table, suffix_lens, group_starts, scale, out, return_lse)
// -> out or (out, lse)
PyObject* attention(PyObject*, PyObject* const* a, Py_ssize_t n) {
    if (!arity(n, 11)) return nullptr;
    return guarded([&]() -> PyObject* {
        const fs_paged_kv kv = paged_kv(a[1], a[2]);
        const at::Tensor& cache = *tensor(a[1]);
        const auto type = cache.scalar_type();
        const auto dev = cache.get_device();
        const at::Tensor& given = float_cuda(a[0], "query", 3, 4);
        const at::Tensor& q = vectors(a[0], "query", given.sizes(), type, dev);
        const c10::DeviceGuard guard(cache.device());
        at::Tensor out = none(a[9]) ? at::empty(q.sizes(), q.options()) : vectors(a[9], "out", q.sizes(), type, dev);
        if (!none(a[9])) {
            const Span to(out), in_query(q);
            writable(to, "out");
            apart(to, "out", Span(cache), "k_cache");
            apart(to, "out", Span(*tensor(a[2])), "v_cache");
            if (!same_view(in_query, to)) apart(to, "out", in_query, "query");
        }
        no_gradient({&q, &cache, tensor(a[2]), tensor(a[9])});
        const bool one = q.dim() == 3;
        const int32_t B = size32(q.size(0), "the batch"), Q = one ? 1 : size32(q.size(1), "the number of queries");
        const int32_t Hq = size32(q.size(-2), "the number of heads");
        if (q.size(-1) != kv.head_dim || Q < 1 || Hq < 1 || Hq % kv.num_heads != 0)
            refuse("query must have the caches' head size, at least one token, and a multiple of their heads");
        int64_t qs[3], os[3];
        for (const auto& [t, s] : {std::pair<const at::Tensor&, int64_t*>(q, qs), std::pair<const at::Tensor&, int64_t*>(out, os)}) {
            strides(t, one ? 2 : 3, s);
            if (one) s[2] = s[1], s[1] = 0;
        }
        int32_t G = 0, pw = 0;
        const int32_t *ptab = nullptr, *plens = nullptr, *starts = nullptr;
        if (!none(a[3])) {
            const at::Tensor& t = flat(a[3], "prefix_table", {-1, -1}, at::kInt, dev);
            G = size32(t.size(0), "the table"), pw = size32(t.size(1), "the table");
            ptab = static_cast<const int32_t*>(t.data_ptr());
            plens = static_cast<const int32_t*>(flat(a[4], "prefix_lens", {G}, at::kInt, dev).data_ptr());
        } else if (!none(a[4]) || !none(a[7])) {
            refuse("prefix_lens and group_starts need a prefix_table");
        }
        starts = flat_ptr<int32_t>(a[7], "group_starts", int64_t(G) + 1, at::kInt, dev);
        if (G > 1 && none(a[7])) refuse("several prefixes need group_starts");
        const at::Tensor& stab = flat(a[5], "suffix_table", {B, -1}, at::kInt, dev);
        const int32_t sw = size32(stab.size(1), "the table");
        const auto* slens = static_cast<const int32_t*>(flat(a[6], "suffix_lens", {B}, at::kInt, dev).data_ptr());
        double scale = 1.0 / std::sqrt(double(kv.head_dim));
        if (!none(a[8])) {
            scale = PyFloat_AsDouble(a[8]);
            if (scale == -1.0 && PyErr_Occurred()) return nullptr;
        }
        const int want_lse = PyObject_IsTrue(a[10]);
        if (want_lse < 0) return nullptr;
        at::Tensor lse;
        if (want_lse) lse = at::empty(q.sizes().slice(0, q.dim() - 1), q.options().dtype(at::kFloat));
        size_t need = 0;
        const fs_status st = fs_shared_prefix_attention_workspace_bytes(&kv, B, Q, Hq, G, pw, sw, &need);
        if (st != FS_OK) return PyLong_FromLong(st);
        const at::Tensor ws = scratch(need, q);
        return launch(q, [&](void* s) {
            return fs_shared_prefix_attention(&kv, q.data_ptr(), qs, B, Q, Hq, starts, G, ptab, pw, plens,
                                              static_cast<const int32_t*>(stab.data_ptr()), sw, slens, float(scale), out.data_ptr(), os,
                                              want_lse ? static_cast<float*>(lse.data_ptr()) : nullptr, ws.data_ptr(), need, s);
        }, [&]() -> PyObject* {
            written({tensor(a[9])});
            if (none(a[9])) return want_lse ? pair(out, lse) : wrap(out);
            PyObject* o = a[9];
            if (!want_lse) {
                Py_INCREF(o);
                return o;
            }
            return PyTuple_Pack(2, o, py_owned(wrap(lse)).p);
        });
    });
}

// (a, b) -> whether two elements of tensors of one type share memory; of one tensor, with itself.
PyObject* shares(PyObject*, PyObject* const* a, Py_ssize_t n) {
    if (!arity(n, 2)) return nullptr;
    return guarded([&]() -> PyObject* {
        const at::Tensor *x = tensor(a[0]), *y = tensor(a[1]);
        if (!x || !y || x->scalar_type() != y->scalar_type()) refuse("two tensors of one type are needed");
        return PyBool_FromLong(a[0] == a[1] ? overlaps_itself(Span(*x)) : shares_memory(Span(*x), Span(*y)));
    });
}

PyMethodDef METHODS[] = {
    {"from_uniforms", reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(from_uniforms)), METH_FASTCALL, nullptr},
    {"append", reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(append)), METH_FASTCALL, nullptr},
    {"attention", reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(attention)), METH_FASTCALL, nullptr},
    {"shares_memory", reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(shares)), METH_FASTCALL, nullptr},
    {nullptr, nullptr, 0, nullptr}};

PyModuleDef MODULE = {PyModuleDef_HEAD_INIT, "_decode", "The decode step's entries of libfs_sampling.so for torch tensors.",
                      -1, METHODS, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__decode() { return PyModule_Create(&MODULE); }
