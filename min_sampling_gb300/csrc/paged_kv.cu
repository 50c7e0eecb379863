// Appending keys and values to a paged cache, with the position rotation applied on the
// way (sm_103a).
//
// Per token t with position p: every rotated pair (x, y) of a head becomes
//   (x cos a - y sin a, y cos a + x sin a),  a = p * inv_freq[i], i the pair's index;
// the key goes rotated, the value as it is, into slot p % page_size of page
// page_table[row][p / page_size]; the step's queries are rotated by the same angles.
//
// The angle is reduced exactly: inv_freq[i] / 2 pi as a 64-bit fraction of a turn
// (integer arithmetic on the float's 24-bit significand), times the position modulo
// 2^64, is the fraction of a turn for any 32-bit position (error at most 2^-33 turns;
// in float32, p * inv_freq alone would be off by 0.06 radians at p = 10^6).
//
// Bound by memory: every element is read once and written once.  One CTA row of threads
// per token: the token's cosines and sines are computed once into shared memory and serve
// all of its heads, and every thread has its first loads in flight before it computes
// them.
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include "fs_device.cuh"
#include "fs_host.h"

namespace fsd {

struct AppendArgs {
    const void* key;
    const void* value;
    const void* query;          // nullable
    void* query_out;
    void* k_cache;
    void* v_cache;
    int64_t key_t, key_h, val_t, val_h, q_t, q_h, qo_t, qo_h;  // token and head strides (elements)
    int64_t kc[3], vc[3];       // cache strides: page, slot, head
    int kv_heads, q_heads, dim, half, interleaved;  // half = rotated pairs per head
    int num_pages, page_size, table_rows, table_width, tokens;
    const int* table;
    const int* rows;            // nullable: token t belongs to row t
    const int* positions;
    const int* rotary_positions;  // nullable: positions
    const float* inv_freq;
};

// inv_freq / (2 pi) modulo 1 as a 64-bit fraction.  f = m * 2^e with a 24-bit m, so
// the product with 2^64 / (2 pi) has at most 86 bits and is shifted into place.
__device__ __forceinline__ uint64_t turn_fraction(float f) {
    constexpr uint64_t INV_2PI = 0x28BE60DB9391054Aull;  // floor(2^64 / (2 pi))
    const uint32_t u = __float_as_uint(f);
    const int ex = int((u >> 23) & 0xff);
    const uint64_t m = (u & 0x7fffffu) | (ex ? 0x800000u : 0u);
    const int e = (ex ? ex : 1) - 150;
    const uint64_t lo = m * INV_2PI, hi = __umul64hi(m, INV_2PI);
    uint64_t r;
    if (e >= 0) {
        r = e < 64 ? lo << e : 0;
    } else {
        const int s = -e;
        r = s < 64 ? (lo >> s) | (hi << (64 - s)) : (s < 128 ? hi >> (s - 64) : 0);
    }
    return (u >> 31) ? 0 - r : r;
}

__device__ __forceinline__ float2 cos_sin_of(float f, int pos) {
    const uint64_t turn = turn_fraction(f) * uint64_t(int64_t(pos));
    float s, c;
    sincospif(float(int32_t(uint32_t(turn >> 32))) * 0x1p-31f, &s, &c);  // the angle in half turns, [-1, 1)
    const float bad = f * 0.f;  // NaN for an infinite or NaN frequency
    return make_float2(c + bad, s + bad);
}

template <typename T> struct Io;
template <> struct Io<__nv_bfloat16> {
    static __device__ __forceinline__ float get(__nv_bfloat16 x) { return __bfloat162float(x); }
    static __device__ __forceinline__ __nv_bfloat16 put(float x) { return __float2bfloat16_rn(x); }
};
template <> struct Io<__half> {
    static __device__ __forceinline__ float get(__half x) { return __half2float(x); }
    static __device__ __forceinline__ __half put(float x) { return __float2half_rn(x); }
};
template <> struct Io<float> {
    static __device__ __forceinline__ float get(float x) { return x; }
    static __device__ __forceinline__ float put(float x) { return x; }
};

// VW consecutive elements, moved as one word.
template <typename T, int VW>
struct alignas(VW * sizeof(T)) Pack {
    T e[VW];
};

// One unit of a token's work: VW elements at `off` of a head and, for a rotation in
// halves (or of single elements), their partners at `off2`.
struct Unit {
    int src;    // 0 key, 1 value, 2 query, -1 none
    int head, off, off2, pair;  // pair: the first rotated pair's index, -1 for a plain copy
};

template <typename T, int VW>
__device__ __forceinline__ Unit unit_of(const AppendArgs& a, int i) {
    // Per rotated head: units of pairs, then the rest copied; per value head: copies.
    const int per_pairs = (a.interleaved && VW > 1) ? 2 * a.half / VW : a.half / VW;
    const int per_rot = per_pairs + (a.dim - 2 * a.half) / VW;
    const int per_val = a.dim / VW;
    const int nq = a.query ? a.q_heads * per_rot : 0, nk = a.kv_heads * per_rot;
    Unit u;
    u.off2 = -1;
    u.pair = -1;
    if (i < nq + nk) {
        u.src = i < nq ? 2 : 0;
        const int j = i < nq ? i : i - nq;
        u.head = j / per_rot;
        const int r = j - u.head * per_rot;
        if (r >= per_pairs) {
            u.off = 2 * a.half + (r - per_pairs) * VW;
        } else if (!a.interleaved) {
            u.off = r * VW;
            u.off2 = u.off + a.half;
            u.pair = u.off;
        } else if (VW > 1) {
            u.off = r * VW;
            u.pair = u.off / 2;
        } else {
            u.off = 2 * r;
            u.off2 = 2 * r + 1;
            u.pair = r;
        }
    } else {
        const int j = i - nq - nk;
        u.src = j < a.kv_heads * per_val ? 1 : -1;
        u.head = j / per_val;
        u.off = (j - u.head * per_val) * VW;
    }
    return u;
}

template <typename T, int VW>
__global__ void __launch_bounds__(256) append_kernel(const AppendArgs a) {
    extern __shared__ float2 turns[];  // [blockDim.y][half]
    using P = Pack<T, VW>;
    grid_dependency_wait();
    allow_dependents();
    const int t = blockIdx.x * blockDim.y + threadIdx.y;
    const bool live = t < a.tokens;
    const int per_pairs = (a.interleaved && VW > 1) ? 2 * a.half / VW : a.half / VW;
    const int per_rot = per_pairs + (a.dim - 2 * a.half) / VW;
    const int n = ((a.query ? a.q_heads : 0) + a.kv_heads) * per_rot + a.kv_heads * (a.dim / VW);

    auto load = [&](const Unit& u, P& x, P& y) {
        const T* p = u.src == 0   ? static_cast<const T*>(a.key) + t * a.key_t + u.head * a.key_h
                     : u.src == 1 ? static_cast<const T*>(a.value) + t * a.val_t + u.head * a.val_h
                                  : static_cast<const T*>(a.query) + t * a.q_t + u.head * a.q_h;
        x = *reinterpret_cast<const P*>(p + u.off);
        if (u.off2 >= 0) y = *reinterpret_cast<const P*>(p + u.off2);
    };
    // The first two units' loads go out before anything depends on the positions.
    constexpr int PRE = 2;
    Unit u[PRE];
    P x[PRE], y[PRE];
#pragma unroll
    for (int j = 0; j < PRE; ++j) {
        const int i = threadIdx.x + j * blockDim.x;
        u[j].src = -1;
        if (live && i < n) {
            u[j] = unit_of<T, VW>(a, i);
            load(u[j], x[j], y[j]);
        }
    }
    // Where the token goes.  A negative position marks padding; a row or page that does
    // not exist is not written either.
    int64_t k_at = -1, v_at = -1;
    bool pad = true;
    float2* cs = turns + threadIdx.y * a.half;
    if (live) {
        const int pos = a.positions[t];
        const int row = a.rows ? a.rows[t] : t;
        pad = pos < 0;
        const int pi = pad ? 0 : pos / a.page_size;
        if (!pad && row >= 0 && row < a.table_rows && pi < a.table_width) {
            const int page = a.table[int64_t(row) * a.table_width + pi];
            if (page >= 0 && page < a.num_pages) {
                const int slot = pos - pi * a.page_size;
                k_at = page * a.kc[0] + slot * a.kc[1];
                v_at = page * a.vc[0] + slot * a.vc[1];
            }
        }
        const int rp = a.rotary_positions ? a.rotary_positions[t] : pos;
        for (int i = threadIdx.x; i < a.half; i += blockDim.x)
            cs[i] = pad ? make_float2(1.f, 0.f) : cos_sin_of(a.inv_freq[i], rp);
    }
    __syncthreads();
    if (!live) return;

    auto finish = [&](const Unit& v, P& p, P& q) {
        if (v.pair >= 0 && !pad) {
            if (v.off2 >= 0) {
#pragma unroll
                for (int e = 0; e < VW; ++e) {
                    const float2 w = cs[v.pair + e];
                    const float f = Io<T>::get(p.e[e]), g = Io<T>::get(q.e[e]);
                    p.e[e] = Io<T>::put(f * w.x - g * w.y);
                    q.e[e] = Io<T>::put(g * w.x + f * w.y);
                }
            } else {
#pragma unroll
                for (int e = 0; e + 1 < VW; e += 2) {
                    const float2 w = cs[v.pair + e / 2];
                    const float f = Io<T>::get(p.e[e]), g = Io<T>::get(p.e[e + 1]);
                    p.e[e] = Io<T>::put(f * w.x - g * w.y);
                    p.e[e + 1] = Io<T>::put(g * w.x + f * w.y);
                }
            }
        }
        T* d;
        if (v.src == 2) {
            d = static_cast<T*>(a.query_out) + t * a.qo_t + v.head * a.qo_h;
        } else {
            if (k_at < 0) return;
            d = v.src == 0 ? static_cast<T*>(a.k_cache) + k_at + v.head * a.kc[2]
                           : static_cast<T*>(a.v_cache) + v_at + v.head * a.vc[2];
        }
        *reinterpret_cast<P*>(d + v.off) = p;
        if (v.off2 >= 0) *reinterpret_cast<P*>(d + v.off2) = q;
    };
#pragma unroll
    for (int j = 0; j < PRE; ++j)
        if (u[j].src >= 0) finish(u[j], x[j], y[j]);
    for (int i = threadIdx.x + PRE * blockDim.x; i < n; i += blockDim.x) {
        const Unit w = unit_of<T, VW>(a, i);
        P p, q;
        load(w, p, q);
        finish(w, p, q);
    }
}

template <typename T, int VW>
static fs_status launch_append(const AppendArgs& a, void* stream) {
    const int per_pairs = (a.interleaved && VW > 1) ? 2 * a.half / VW : a.half / VW;
    const int per_rot = per_pairs + (a.dim - 2 * a.half) / VW;
    const int64_t n = int64_t((a.query ? a.q_heads : 0) + a.kv_heads) * per_rot + int64_t(a.kv_heads) * (a.dim / VW);
    // Threads per token: two units a thread, whole warps, at most 256; small tokens share a CTA.
    int tx = int(n < 512 ? (n + 63) / 64 * 32 : 256);
    const int ty = 256 / tx;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(unsigned((a.tokens + ty - 1) / ty), 1, 1);
    cfg.blockDim = dim3(unsigned(tx), unsigned(ty), 1);
    cfg.dynamicSmemBytes = size_t(ty) * size_t(a.half) * sizeof(float2);
    cfg.stream = static_cast<cudaStream_t>(stream);
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    const cudaError_t e = cudaLaunchKernelEx(&cfg, append_kernel<T, VW>, a);
    return e == cudaSuccess ? FS_OK : cuda_fail(e);
}

}  // namespace fsd

extern "C" {

fs_status fs_append_paged_kv(const fs_paged_kv* cache, const void* key, const int64_t* key_strides, const void* value,
                             const int64_t* value_strides, int32_t tokens, const int32_t* page_table,
                             int32_t table_rows, int32_t table_width, const int32_t* rows, const int32_t* positions,
                             const int32_t* rotary_positions, const float* inv_freq, int32_t rotary_dim,
                             int32_t interleaved, const void* query, const int64_t* query_strides, int32_t q_heads,
                             void* query_out, const int64_t* query_out_strides, void* stream) {
    using namespace fsd;
    if (!cache || tokens < 0 || table_rows < 0 || table_width < 0 || rotary_dim < 0) return FS_ERR_INVALID_ARG;
    if (cache->num_pages < 0 || cache->page_size < 1 || cache->num_heads < 1 || cache->head_dim < 1)
        return FS_ERR_INVALID_ARG;
    if (rotary_dim % 2 != 0 || rotary_dim > cache->head_dim || (interleaved != 0 && interleaved != 1))
        return FS_ERR_INVALID_ARG;
    if (cache->dtype != FS_F32 && cache->dtype != FS_BF16 && cache->dtype != FS_F16) return FS_ERR_INVALID_ARG;
    if (!rows && table_rows < tokens) return FS_ERR_INVALID_ARG;
    if (query && (q_heads < 1 || !query_strides || !query_out || !query_out_strides)) return FS_ERR_INVALID_ARG;
    if (tokens == 0) return FS_OK;
    if (!key || !value || !key_strides || !value_strides || !positions) return FS_ERR_INVALID_ARG;
    if (cache->num_pages > 0 && (!cache->k || !cache->v)) return FS_ERR_INVALID_ARG;
    if (int64_t(table_rows) * table_width > 0 && !page_table) return FS_ERR_INVALID_ARG;
    if (rotary_dim > 0 && !inv_freq) return FS_ERR_INVALID_ARG;
    if (cache->head_dim > 1024 || cache->num_heads > 4096 || q_heads > 4096) return FS_ERR_UNSUPPORTED;
    AppendArgs a = {};
    a.key = key;
    a.value = value;
    a.query = query;
    a.query_out = query_out;
    a.k_cache = cache->k;
    a.v_cache = cache->v;
    a.key_t = key_strides[0];
    a.key_h = key_strides[1];
    a.val_t = value_strides[0];
    a.val_h = value_strides[1];
    if (query) {
        a.q_t = query_strides[0];
        a.q_h = query_strides[1];
        a.qo_t = query_out_strides[0];
        a.qo_h = query_out_strides[1];
    }
    uintptr_t bits = 0;  // every address and stride the kernel moves whole words by
    const int es = cache->dtype == FS_F32 ? 4 : 2;
    for (int i = 0; i < 3; ++i) {
        a.kc[i] = cache->k_strides[i];
        a.vc[i] = cache->v_strides[i];
        bits |= uintptr_t(a.kc[i] * es) | uintptr_t(a.vc[i] * es);
    }
    for (int64_t s : {a.key_t, a.key_h, a.val_t, a.val_h, a.q_t, a.q_h, a.qo_t, a.qo_h}) bits |= uintptr_t(s * es);
    for (const void* p : {key, value, query, static_cast<const void*>(query_out), static_cast<const void*>(cache->k),
                          static_cast<const void*>(cache->v)})
        bits |= reinterpret_cast<uintptr_t>(p);
    a.kv_heads = cache->num_heads;
    a.q_heads = query ? q_heads : 0;
    a.dim = cache->head_dim;
    a.half = rotary_dim / 2;
    a.interleaved = interleaved;
    a.num_pages = cache->num_pages;
    a.page_size = cache->page_size;
    a.table_rows = table_rows;
    a.table_width = table_width;
    a.tokens = tokens;
    a.table = page_table;
    a.rows = rows;
    a.positions = positions;
    a.rotary_positions = rotary_positions;
    a.inv_freq = inv_freq;
    // 16-byte words where everything is aligned to them and no word straddles the two
    // halves of a rotation or its end; single elements otherwise.
    const int vw = 16 / es;
    const bool wide = (bits & 15) == 0 && a.dim % vw == 0 && (interleaved ? rotary_dim : a.half) % vw == 0;
    switch (cache->dtype) {
        case FS_F32: return wide ? launch_append<float, 4>(a, stream) : launch_append<float, 1>(a, stream);
        case FS_BF16:
            return wide ? launch_append<__nv_bfloat16, 8>(a, stream) : launch_append<__nv_bfloat16, 1>(a, stream);
        default: return wide ? launch_append<__half, 8>(a, stream) : launch_append<__half, 1>(a, stream);
    }
}

}  // extern "C"
