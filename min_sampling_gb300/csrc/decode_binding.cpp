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

// (None is asked about first: whether it is an instance of a tensor's class takes Python about 0.1 us to answer)
const at::Tensor* tensor(PyObject* o) { return !none(o) && THPVariable_Check(o) ? &THPVariable_Unpack(o) : nullptr; }

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

// The same for a tensor of another type, by the bytes between first and last.
void apart_bytes(const Span& written, const char* name, const Span& other, const char* other_name) {
    if (written.first != written.end && other.first != other.end && written.first < other.end && other.first < written.end)
        refuse(std::string(name) + " is written, but shares memory with " + other_name);
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

// (key, value, k_cache, v_cache, page_table, positions, rows, rotary_positions, inv_freq, interleaved, query, query_out,
//  query_norm, key_norm, norm_eps) -> query_out or None
PyObject* append(PyObject*, PyObject* const* a, Py_ssize_t n) {
    if (!arity(n, 15)) return nullptr;
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
        const auto* q_norm = flat_ptr<float>(a[12], "query_norm", kv.head_dim, at::kFloat, dev);
        const auto* k_norm = flat_ptr<float>(a[13], "key_norm", kv.head_dim, at::kFloat, dev);
        double eps = 0.0;
        if (q_norm || k_norm) {
            if (q_norm && !q) refuse("query_norm needs a query");
            eps = PyFloat_AsDouble(a[14]);
            if (eps == -1.0 && PyErr_Occurred()) return nullptr;
            if (!(eps >= 0.0)) refuse("norm_eps must not be negative");
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
        no_gradient({&key, &value, &cache, tensor(a[3]), q, tensor(a[11]), tensor(a[12]), tensor(a[13])});
        return launch(cache, [&](void* s) {
            if (q_norm || k_norm)
                return fs_append_paged_kv_normed(&kv, key.data_ptr(), ks, value.data_ptr(), vs, tokens,
                                                 static_cast<const int32_t*>(table.data_ptr()), size32(table.size(0), "the table"),
                                                 size32(table.size(1), "the table"), rows, pos, rpos, freq, int32_t(rotary),
                                                 interleaved, q ? q->data_ptr() : nullptr, qs, q_heads, q ? qo.data_ptr() : nullptr,
                                                 qos, q_norm, k_norm, float(eps), s);
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

// (lens, new_lens, page_table, free_pages, free_count, page_size, max_tokens)
// -> (query_starts, rows, positions, totals, free_left)
PyObject* step_tables(PyObject*, PyObject* const* a, Py_ssize_t n) {
    if (!arity(n, 7)) return nullptr;
    return guarded([&]() -> PyObject* {
        const at::Tensor* t = tensor(a[2]);
        if (!t || !t->is_cuda()) refuse("page_table must be a CUDA tensor");
        const auto dev = t->get_device();
        const at::Tensor& table = flat(a[2], "page_table", {-1, -1}, at::kInt, dev);
        const int32_t R = size32(table.size(0), "the table"), width = size32(table.size(1), "the table");
        const at::Tensor& lens = flat(a[0], "lens", {R}, at::kInt, dev);
        const at::Tensor& fresh = flat(a[1], "new_lens", {R}, at::kInt, dev);
        const at::Tensor& pages = flat(a[3], "free_pages", {-1}, at::kInt, dev);
        const at::Tensor& count = flat(a[4], "free_count", {1}, at::kInt, dev);
        const int64_t page = PyLong_AsLongLong(a[5]), budget = page == -1 && PyErr_Occurred() ? -1 : PyLong_AsLongLong(a[6]);
        if (PyErr_Occurred()) return nullptr;
        if (page < 1 || page > INT32_MAX) refuse("page_size must be at least 1");
        if (budget < 0 || budget > INT32_MAX) refuse("max_tokens must not be negative");
        const Span to(table);
        apart(to, "page_table", Span(lens), "lens");
        apart(to, "page_table", Span(fresh), "new_lens");
        apart(to, "page_table", Span(pages), "free_pages");
        apart(to, "page_table", Span(count), "free_count");
        const c10::DeviceGuard guard(table.device());
        // The five results lie in one allocation, each from a multiple of 16 bytes on: five of them take the host
        // longer than the kernel the GPU.
        const int64_t sizes[5] = {int64_t(R) + 1, budget, budget, R, 1};
        int64_t at[5], ints = 0;
        for (int i = 0; i < 5; ++i) at[i] = ints, ints += (sizes[i] + 3) / 4 * 4;
        const at::Tensor all = at::empty({ints}, lens.options());
        at::Tensor made[5];
        for (int i = 0; i < 5; ++i) {
            made[i] = at::detail::make_tensor<c10::TensorImpl>(c10::Storage(all.storage()), all.key_set(), all.dtype());
            made[i].unsafeGetTensorImpl()->set_storage_offset(at[i]);
            made[i].unsafeGetTensorImpl()->set_sizes_contiguous(sizes[i]);
        }
        at::Tensor &starts = made[0], &rows = made[1], &pos = made[2], &totals = made[3], &left = made[4];
        auto in = [](const at::Tensor& x) { return static_cast<const int32_t*>(x.const_data_ptr()); };
        auto out = [](const at::Tensor& x) { return static_cast<int32_t*>(x.data_ptr()); };
        return launch(table, [&](void* s) {
            return fs_paged_step_tables(in(lens), in(fresh), R, out(table), width, in(pages), size32(pages.size(0), "free_pages"),
                                        in(count), int32_t(page), int32_t(budget), out(starts), out(rows), out(pos), out(totals),
                                        out(left), s);
        }, [&]() -> PyObject* {
            written({&table});
            PyObject* r = PyTuple_New(5);
            int i = 0;
            if (r)
                for (at::Tensor* x : {&starts, &rows, &pos, &totals, &left}) PyTuple_SET_ITEM(r, i++, wrap(std::move(*x)));
            return r;
        });
    });
}

// (query, k_cache, v_cache, page_table, query_starts, lens, window, sinks, max_queries, scale, out, return_lse)
// -> out or (out, lse)
PyObject* chunk_attention(PyObject*, PyObject* const* a, Py_ssize_t n) {
    if (!arity(n, 12)) return nullptr;
    return guarded([&]() -> PyObject* {
        const fs_paged_kv kv = paged_kv(a[1], a[2]);
        const at::Tensor& cache = *tensor(a[1]);
        const auto type = cache.scalar_type();
        const auto dev = cache.get_device();
        const at::Tensor& q = vectors(a[0], "query", {-1, -1, kv.head_dim}, type, dev);
        const c10::DeviceGuard guard(cache.device());
        at::Tensor out = none(a[10]) ? at::empty(q.sizes(), q.options()) : vectors(a[10], "out", q.sizes(), type, dev);
        if (!none(a[10])) {
            const Span to(out), in_query(q);
            writable(to, "out");
            apart(to, "out", Span(cache), "k_cache");
            apart(to, "out", Span(*tensor(a[2])), "v_cache");
            if (!same_view(in_query, to)) apart(to, "out", in_query, "query");
        }
        for (int i = 3; i < 6 && !none(a[10]); ++i) {
            static const char* const others[] = {"page_table", "query_starts", "lens"};
            if (const at::Tensor* t = tensor(a[i])) apart_bytes(Span(out), "out", Span(*t), others[i - 3]);
        }
        no_gradient({&q, &cache, tensor(a[2]), tensor(a[10])});
        const int32_t N = size32(q.size(0), "the number of tokens"), Hq = size32(q.size(1), "the number of heads");
        if (Hq < 1 || Hq % kv.num_heads != 0) refuse("query must have a multiple of the caches' heads");
        int64_t qs[2], os[2];
        strides(q, 2, qs);
        strides(out, 2, os);
        const at::Tensor& table = flat(a[3], "page_table", {-1, -1}, at::kInt, dev);
        const int32_t R = size32(table.size(0), "the table"), width = size32(table.size(1), "the table");
        const auto* starts = static_cast<const int32_t*>(flat(a[4], "query_starts", {int64_t(R) + 1}, at::kInt, dev).data_ptr());
        const auto* lens = static_cast<const int32_t*>(flat(a[5], "lens", {R}, at::kInt, dev).data_ptr());
        // None: no window; every token may be of one request
        int64_t window = 0, most = std::max(N, 1);
        if (!none(a[6])) {
            window = PyLong_AsLongLong(a[6]);
            if (window == -1 && PyErr_Occurred()) return nullptr;
            if (window < 1) refuse("window must be at least 1 (None: no window)");
        }
        const int64_t sinks = PyLong_AsLongLong(a[7]);
        if (sinks == -1 && PyErr_Occurred()) return nullptr;
        if (sinks < 0) refuse("sinks must not be negative");
        if (!none(a[8])) {
            most = PyLong_AsLongLong(a[8]);
            if (most == -1 && PyErr_Occurred()) return nullptr;
            if (most < 1) refuse("max_queries must be at least 1");
        }
        double scale = 1.0 / std::sqrt(double(kv.head_dim));
        if (!none(a[9])) {
            scale = PyFloat_AsDouble(a[9]);
            if (scale == -1.0 && PyErr_Occurred()) return nullptr;
        }
        const int want_lse = PyObject_IsTrue(a[11]);
        if (want_lse < 0) return nullptr;
        at::Tensor lse;
        // (what a given out keeps of rows of no request, its lse does not have)
        if (want_lse) lse = none(a[10]) ? at::empty({N, Hq}, q.options().dtype(at::kFloat))
                                        : at::full({N, Hq}, -INFINITY, q.options().dtype(at::kFloat));
        auto clamp32 = [](int64_t x) { return int32_t(std::min<int64_t>(x, INT32_MAX)); };
        size_t need = 0;
        const fs_status st = fs_paged_chunk_attention_workspace_bytes(&kv, N, R, Hq, width, clamp32(most), &need);
        if (st != FS_OK) return PyLong_FromLong(st);
        const at::Tensor ws = scratch(need, q);
        return launch(q, [&](void* s) {
            return fs_paged_chunk_attention(&kv, q.data_ptr(), qs, N, Hq, static_cast<const int32_t*>(table.data_ptr()), R, width, starts,
                                            lens, clamp32(most), clamp32(window), clamp32(sinks), float(scale), none(a[10]),
                                            out.data_ptr(), os, want_lse ? static_cast<float*>(lse.data_ptr()) : nullptr,
                                            ws.data_ptr(), need, s);
        }, [&]() -> PyObject* {
            written({tensor(a[10])});
            if (none(a[10])) return want_lse ? pair(out, lse) : wrap(out);
            PyObject* o = a[10];
            if (!want_lse) {
                Py_INCREF(o);
                return o;
            }
            return PyTuple_Pack(2, o, py_owned(wrap(lse)).p);
        });
    });
}

// (logits, tokens, lens, prompt_lens, repetition, presence, frequency, bias_starts, bias_tokens, bias_values, allowed,
//  allowed_rows, out) -> out
PyObject* adjust(PyObject*, PyObject* const* a, Py_ssize_t n) {
    if (!arity(n, 13)) return nullptr;
    return guarded([&]() -> PyObject* {
        const at::Tensor& x = float_cuda(a[0], "logits", 2, 2);
        const int64_t B = x.size(0), V = x.size(1), stride = B > 1 ? x.stride(0) : V;
        const auto dev = x.get_device();
        if (V < 1 || (V > 1 && x.stride(1) != 1) || stride < V)
            refuse("logits must have at least one column, contiguous columns and rows that do not overlap");
        const c10::DeviceGuard guard(x.device());
        at::Tensor out = none(a[12]) ? at::empty({B, V}, x.options()) : vectors(a[12], "out", x.sizes(), x.scalar_type(), dev);
        const int64_t out_stride = B > 1 ? out.stride(0) : V;
        if (out_stride < V) refuse("out must have rows that do not overlap");
        // the history
        const at::Tensor* tok = nullptr;
        const int32_t *lens = nullptr, *prompts = nullptr;
        if (!none(a[1])) {
            tok = &vectors(a[1], "tokens", {B, -1}, at::kInt, dev);
            lens = flat_ptr<int32_t>(a[2], "lens", B, at::kInt, dev);
            prompts = flat_ptr<int32_t>(a[3], "prompt_lens", B, at::kInt, dev);
        } else {
            for (int i = 2; i < 7; ++i)
                if (!none(a[i])) refuse("lens, prompt_lens and penalties need tokens");
        }
        const int64_t tok_stride = tok && B > 1 ? tok->stride(0) : tok ? tok->size(1) : 0;
        if (tok && tok_stride < tok->size(1)) refuse("tokens must have rows that do not overlap");
        at::Tensor held[3];
        const float* ps[3] = {};
        static const char* const names[3] = {"repetition", "presence", "frequency"};
        for (int i = 0; i < 3; ++i) {
            PyObject* o = a[4 + i];
            if (none(o)) continue;
            if (!tensor(o)) {
                const double v = PyFloat_AsDouble(o);
                if (v == -1.0 && PyErr_Occurred()) return nullptr;
                held[i] = at::full({B}, v, x.options().dtype(at::kFloat));
                ps[i] = static_cast<const float*>(held[i].data_ptr());
            } else {
                ps[i] = static_cast<const float*>(flat(o, names[i], {B}, at::kFloat, dev).data_ptr());
            }
        }
        // biases
        const bool biased = !none(a[7]);
        if (biased != !none(a[8]) || biased != !none(a[9])) refuse("bias_starts, bias_tokens and bias_values belong together");
        int32_t biases = 0;
        const int32_t *bs = nullptr, *bt = nullptr;
        const float* bv = nullptr;
        if (biased) {
            bs = static_cast<const int32_t*>(flat(a[7], "bias_starts", {B + 1}, at::kInt, dev).data_ptr());
            const at::Tensor& t = flat(a[8], "bias_tokens", {-1}, at::kInt, dev);
            biases = size32(t.size(0), "the number of biases");
            bt = static_cast<const int32_t*>(t.data_ptr());
            bv = static_cast<const float*>(flat(a[9], "bias_values", {biases}, at::kFloat, dev).data_ptr());
        }
        // masks
        int32_t masks = 0;
        const uint32_t* allowed = nullptr;
        const int32_t* mrows = nullptr;
        if (!none(a[10])) {
            const at::Tensor& t = flat(a[10], "allowed", {-1, (V + 31) / 32}, at::kInt, dev);
            masks = size32(t.size(0), "the number of masks");
            mrows = flat_ptr<int32_t>(a[11], "allowed_rows", B, at::kInt, dev);
            if (none(a[11]) && masks < B) refuse("allowed needs a mask for every row when allowed_rows is not given");
            // (no masks at all: every row's is one that does not exist, or none)
            allowed = masks > 0 ? static_cast<const uint32_t*>(t.const_data_ptr()) : reinterpret_cast<const uint32_t*>(mrows);
        } else if (!none(a[11])) {
            refuse("allowed_rows needs allowed");
        }
        if (!none(a[12])) {
            const Span to(out), in(x);
            writable(to, "out");
            if (!same_view(in, to)) apart(to, "out", in, "logits");
            static const char* const others[] = {"tokens", "lens", "prompt_lens", "repetition", "presence", "frequency",
                                                 "bias_starts", "bias_tokens", "bias_values", "allowed", "allowed_rows"};
            for (int i = 0; i < 11; ++i)
                if (const at::Tensor* t = tensor(a[1 + i])) apart_bytes(to, "out", Span(*t), others[i]);
        }
        no_gradient({&x, tensor(a[4]), tensor(a[5]), tensor(a[6]), tensor(a[9]), tensor(a[12])});
        return launch(x, [&](void* s) {
            const bool hist = tok && tok->size(1) > 0;   // (an empty history penalises nothing)
            return fs_adjust_logits(x.data_ptr(), dtype_of(x.scalar_type()), stride, size32(B, "the batch"), size32(V, "the vocabulary"),
                                    hist ? static_cast<const int32_t*>(tok->data_ptr()) : nullptr, tok_stride,
                                    hist ? size32(tok->size(1), "the history") : 0, hist ? lens : nullptr, hist ? prompts : nullptr,
                                    hist ? ps[0] : nullptr, hist ? ps[1] : nullptr, hist ? ps[2] : nullptr, biases ? bs : nullptr,
                                    biases ? bt : nullptr, biases ? bv : nullptr, biases, allowed, masks, mrows, out.data_ptr(),
                                    out_stride, s);
        }, [&]() -> PyObject* {
            written({tensor(a[12])});
            if (none(a[12])) return wrap(out);
            Py_INCREF(a[12]);
            return a[12];
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
    {"step_tables", reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(step_tables)), METH_FASTCALL, nullptr},
    {"chunk_attention", reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(chunk_attention)), METH_FASTCALL, nullptr},
    {"adjust", reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(adjust)), METH_FASTCALL, nullptr},
    {"shares_memory", reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(shares)), METH_FASTCALL, nullptr},
    {nullptr, nullptr, 0, nullptr}};

PyModuleDef MODULE = {PyModuleDef_HEAD_INIT, "_decode", "The decode step's entries of libfs_sampling.so for torch tensors.",
                      -1, METHODS, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__decode() { return PyModule_Create(&MODULE); }
