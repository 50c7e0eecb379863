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
// Bound by memory: every element is read once and written once.  A CTA takes one to four
// tokens: their cosines and sines are computed once into shared memory and serve all their
// heads, and every thread has its first loads in flight before it computes them.  8190 tokens
// of 32 + 8 + 8 heads of 128 in bf16: 40.7 us, 4.9 TB/s of reads and writes; 64 tokens: 3.7 us.
#include <algorithm>

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
    // Units of a token (see unit_of): of a rotated head, of them pairs; of a value head; in all.
    int per_rot, per_pairs, per_val, units;
    int per_cta;                // tokens of a CTA
    uint32_t m_rot, m_val, m_units;  // for division by the above
    // Norms of each head before the rotation (append_norm_kernel).
    const float* q_weight;      // [dim], nullable: no norm
    const float* k_weight;
    float eps;
    int group;                  // lanes of a head, a power of two
};

// x / d for x d < 2^32 by m = floor(2^32 / d) + 1; m = 0: plain division.
__host__ __device__ inline uint32_t magic_of(uint32_t d, uint64_t most) { return d > 1 && most * d < (uint64_t(1) << 32) ? uint32_t((uint64_t(1) << 32) / d) + 1 : 0; }
__device__ __forceinline__ int quick_div(int x, int d, uint32_t m) { return m ? int(__umulhi(uint32_t(x), m)) : x / d; }

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
    int token, head, off, off2, pair;  // pair: the first rotated pair's index, -1 for a plain copy
};

// Unit i of a CTA's tokens: per token, the rotated heads' (queries, keys; per head units of
// pairs, then the rest copied), then the value heads'.
template <typename T, int VW>
__device__ __forceinline__ Unit unit_of(const AppendArgs& a, int i) {
    Unit u;
    u.token = quick_div(i, a.units, a.m_units);
    i -= u.token * a.units;
    const int nq = a.query ? a.q_heads * a.per_rot : 0, nk = a.kv_heads * a.per_rot;
    u.off2 = -1;
    u.pair = -1;
    if (i < nq + nk) {
        u.src = i < nq ? 2 : 0;
        const int j = i < nq ? i : i - nq;
        u.head = quick_div(j, a.per_rot, a.m_rot);
        const int r = j - u.head * a.per_rot;
        if (r >= a.per_pairs) {
            u.off = 2 * a.half + (r - a.per_pairs) * VW;
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
        u.src = 1;
        u.head = quick_div(j, a.per_val, a.m_val);
        u.off = (j - u.head * a.per_val) * VW;
    }
    return u;
}

// Any alignment: single elements (VW = 1).
template <typename T, int VW>
__global__ void __launch_bounds__(256, 4) append_kernel(const AppendArgs a) {
    // per token: cache offsets of keys and values, whether it is padding or not written, then the turns
    extern __shared__ __align__(16) unsigned char smem[];
    int64_t* slots = reinterpret_cast<int64_t*>(smem);            // [per_cta][2]
    int* pads = reinterpret_cast<int*>(slots + 2 * a.per_cta);    // [per_cta]
    float2* turns = reinterpret_cast<float2*>(slots + 3 * a.per_cta);  // [per_cta][half]
    using P = Pack<T, VW>;
    grid_dependency_wait();
    allow_dependents();
    const int t0 = blockIdx.x * a.per_cta, tokens = min(a.per_cta, a.tokens - t0);
    const int n = tokens * a.units;

    auto load = [&](const Unit& u, P& x, P& y) {
        const int64_t t = t0 + u.token;
        const T* p = u.src == 0   ? static_cast<const T*>(a.key) + t * a.key_t + u.head * a.key_h
                     : u.src == 1 ? static_cast<const T*>(a.value) + t * a.val_t + u.head * a.val_h
                                  : static_cast<const T*>(a.query) + t * a.q_t + u.head * a.q_h;
        x = *reinterpret_cast<const P*>(p + u.off);
        if (u.off2 >= 0) y = *reinterpret_cast<const P*>(p + u.off2);
    };
    constexpr int AT = 2;   // units in flight per thread
    P x[AT], y[AT];
    auto load_all = [&](int i0) {
#pragma unroll
        for (int j = 0; j < AT; ++j) {
            const int i = i0 + j * blockDim.x;
            if (i < n) load(unit_of<T, VW>(a, i), x[j], y[j]);
        }
    };
    // The first loads go out before anything depends on the positions.
    load_all(threadIdx.x);
    // Where each token goes.  A negative position marks padding; a row or page that does
    // not exist is not written either.
    if (int(threadIdx.x) < tokens) {
        const int t = t0 + threadIdx.x;
        const int pos = a.positions[t];
        const int row = a.rows ? a.rows[t] : t;
        const bool pad = pos < 0;
        const int pi = pad ? 0 : pos / a.page_size;
        int64_t k_at = 0, v_at = 0;
        bool there = false;
        if (!pad && row >= 0 && row < a.table_rows && pi < a.table_width) {
            const int page = a.table[int64_t(row) * a.table_width + pi];
            if (page >= 0 && page < a.num_pages) {
                const int slot = pos - pi * a.page_size;
                k_at = page * a.kc[0] + slot * a.kc[1];
                v_at = page * a.vc[0] + slot * a.vc[1];
                there = true;
            }
        }
        slots[2 * threadIdx.x] = k_at;
        slots[2 * threadIdx.x + 1] = v_at;
        pads[threadIdx.x] = pad ? 1 : (there ? 0 : 2);   // 1 padding, 2 not written
    }
    for (int i = threadIdx.x; i < tokens * a.half; i += blockDim.x) {
        const int k = i / a.half, t = t0 + k;
        const int pos = a.positions[t], rp = a.rotary_positions ? a.rotary_positions[t] : pos;
        turns[i] = pos < 0 ? make_float2(1.f, 0.f) : cos_sin_of(a.inv_freq[i - k * a.half], rp);
    }
    __syncthreads();

    auto finish = [&](const Unit& v, P& p, P& q) {
        const int state = pads[v.token];
        const float2* cs = turns + v.token * a.half;
        if (v.pair >= 0 && state != 1) {
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
            d = static_cast<T*>(a.query_out) + (t0 + v.token) * a.qo_t + v.head * a.qo_h;
        } else {
            if (state) return;
            d = v.src == 0 ? static_cast<T*>(a.k_cache) + slots[2 * v.token] + v.head * a.kc[2]
                           : static_cast<T*>(a.v_cache) + slots[2 * v.token + 1] + v.head * a.vc[2];
        }
        *reinterpret_cast<P*>(d + v.off) = p;
        if (v.off2 >= 0) *reinterpret_cast<P*>(d + v.off2) = q;
    };
    for (int i0 = threadIdx.x; i0 < n; i0 += AT * blockDim.x) {
        if (i0 != int(threadIdx.x)) load_all(i0);
#pragma unroll
        for (int j = 0; j < AT; ++j) {
            const int i = i0 + j * blockDim.x;
            if (i < n) finish(unit_of<T, VW>(a, i), x[j], y[j]);
        }
    }
}

// Two floats at a time.
__device__ __forceinline__ float2 mul2(float2 a, float2 b) {
    float2 r;
    asm("{ .reg .b64 x, y, z; mov.b64 x, {%2, %3}; mov.b64 y, {%4, %5}; mul.rn.f32x2 z, x, y; mov.b64 {%0, %1}, z; }"
        : "=f"(r.x), "=f"(r.y) : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y));
    return r;
}
__device__ __forceinline__ float2 fma2(float2 a, float2 b, float2 c) {
    float2 r;
    asm("{ .reg .b64 x, y, z, w; mov.b64 x, {%2, %3}; mov.b64 y, {%4, %5}; mov.b64 z, {%6, %7};"
        " fma.rn.f32x2 w, x, y, z; mov.b64 {%0, %1}, w; }"
        : "=f"(r.x), "=f"(r.y) : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y), "f"(c.x), "f"(c.y));
    return r;
}
template <typename T> struct Two;
template <> struct Two<__nv_bfloat16> {
    static __device__ __forceinline__ float2 get(const __nv_bfloat16* p) {
        const uint32_t u = *reinterpret_cast<const uint32_t*>(p);
        return make_float2(__uint_as_float(u << 16), __uint_as_float(u & 0xffff0000u));
    }
    static __device__ __forceinline__ void put(__nv_bfloat16* p, float2 v) {
        *reinterpret_cast<__nv_bfloat162*>(p) = __floats2bfloat162_rn(v.x, v.y);
    }
};
template <> struct Two<__half> {
    static __device__ __forceinline__ float2 get(const __half* p) { return __half22float2(*reinterpret_cast<const __half2*>(p)); }
    static __device__ __forceinline__ void put(__half* p, float2 v) { *reinterpret_cast<__half2*>(p) = __floats2half2_rn(v.x, v.y); }
};
template <> struct Two<float> {
    static __device__ __forceinline__ float2 get(const float* p) { return make_float2(p[0], p[1]); }
    static __device__ __forceinline__ void put(float* p, float2 v) { p[0] = v.x, p[1] = v.y; }
};

// Aligned data, words of VW elements.  A thread keeps one unit of a head (see unit_of) and
// takes every `lanes`-th rotated head of each of the CTA's tokens, so the unit's cosines and
// sines stay in registers across heads and addresses advance by strides.
template <typename T, int VW>
__global__ void __launch_bounds__(256, 4) append_heads_kernel(const AppendArgs a) {
    extern __shared__ __align__(16) unsigned char smem[];
    int64_t* slots = reinterpret_cast<int64_t*>(smem);            // [per_cta][2]
    int* pads = reinterpret_cast<int*>(slots + 2 * a.per_cta);    // [per_cta], padded to 8 bytes each
    float* cosines = reinterpret_cast<float*>(slots + 4 * a.per_cta);  // [per_cta][half]
    float* sines = cosines + a.per_cta * a.half;
    using P = Pack<T, VW>;
    grid_dependency_wait();
    allow_dependents();
    const int t0 = blockIdx.x * a.per_cta, tokens = min(a.per_cta, a.tokens - t0);
    const int lanes = blockDim.x / a.per_rot, hs = quick_div(threadIdx.x, a.per_rot, a.m_rot), c = threadIdx.x - hs * a.per_rot;
    const int nq = a.query ? a.q_heads : 0, heads = hs < lanes ? nq + a.kv_heads : 0;
    const bool rot = c < a.per_pairs, halves = rot && !a.interleaved;
    const int off = rot ? c * VW : 2 * a.half + (c - a.per_pairs) * VW;
    const int vals = a.kv_heads * a.per_val;

    auto load = [&](int t, int h, P& x, P& y) {
        const T* p = h < nq ? static_cast<const T*>(a.query) + t * a.q_t + h * a.q_h
                            : static_cast<const T*>(a.key) + t * a.key_t + (h - nq) * a.key_h;
        x = *reinterpret_cast<const P*>(p + off);
        if (halves) y = *reinterpret_cast<const P*>(p + off + a.half);
    };
    auto load_value = [&](int t, int i, P& x) {
        const int h = quick_div(i, a.per_val, a.m_val);
        x = *reinterpret_cast<const P*>(static_cast<const T*>(a.value) + t * a.val_t + h * a.val_h + (i - h * a.per_val) * VW);
    };
    constexpr int AT = 2;   // heads in flight per thread
    P x[AT], y[AT], v;
    auto load_token = [&](int t) {
#pragma unroll
        for (int j = 0; j < AT; ++j)
            if (hs + j * lanes < heads) load(t, hs + j * lanes, x[j], y[j]);
        if (int(threadIdx.x) < vals) load_value(t, threadIdx.x, v);
    };
    // The first loads go out before anything depends on the positions.
    load_token(t0);
    if (int(threadIdx.x) < tokens) {
        const int t = t0 + threadIdx.x;
        const int pos = a.positions[t];
        const int row = a.rows ? a.rows[t] : t;
        const bool pad = pos < 0;
        const int pi = pad ? 0 : pos / a.page_size;
        int64_t k_at = 0, v_at = 0;
        bool there = false;
        if (!pad && row >= 0 && row < a.table_rows && pi < a.table_width) {
            const int page = a.table[int64_t(row) * a.table_width + pi];
            if (page >= 0 && page < a.num_pages) {
                const int slot = pos - pi * a.page_size;
                k_at = page * a.kc[0] + slot * a.kc[1];
                v_at = page * a.vc[0] + slot * a.vc[1];
                there = true;
            }
        }
        slots[2 * threadIdx.x] = k_at;
        slots[2 * threadIdx.x + 1] = v_at;
        pads[threadIdx.x] = pad ? 1 : (there ? 0 : 2);   // 1 padding, 2 not written
    }
    for (int i = threadIdx.x; i < tokens * a.half; i += blockDim.x) {
        const int k = i / a.half, t = t0 + k;
        const int pos = a.positions[t], rp = a.rotary_positions ? a.rotary_positions[t] : pos;
        const float2 w = pos < 0 ? make_float2(1.f, 0.f) : cos_sin_of(a.inv_freq[i - k * a.half], rp);
        cosines[i] = w.x;
        sines[i] = w.y;
    }
    __syncthreads();

#pragma unroll 1
    for (int k = 0; k < tokens; ++k) {
        const int t = t0 + k, state = pads[k];
        if (k > 0) load_token(t);
        // The unit's pairs: VW for halves (pairs of this word and its partner), VW / 2 for neighbours.
        float2 cs[VW / 2], sn[VW / 2];
        const float* cp = cosines + k * a.half + (a.interleaved ? off / 2 : off);
        const float* sp = sines + k * a.half + (a.interleaved ? off / 2 : off);
        if (halves) {
#pragma unroll
            for (int e = 0; e < VW / 2; ++e) {
                cs[e] = *reinterpret_cast<const float2*>(cp + 2 * e);
                sn[e] = *reinterpret_cast<const float2*>(sp + 2 * e);
            }
        } else if (rot) {
#pragma unroll
            for (int e = 0; e < VW / 2; ++e) cs[e] = make_float2(cp[e], cp[e]), sn[e] = make_float2(-sp[e], sp[e]);
        }
        auto finish = [&](int h, P& p, P& q) {
            if (state != 1) {
                if (halves) {
#pragma unroll
                    for (int e = 0; e < VW / 2; ++e) {
                        const float2 f = Two<T>::get(p.e + 2 * e), g = Two<T>::get(q.e + 2 * e);
                        const float2 ns = make_float2(-sn[e].x, -sn[e].y);
                        Two<T>::put(p.e + 2 * e, fma2(f, cs[e], mul2(g, ns)));
                        Two<T>::put(q.e + 2 * e, fma2(g, cs[e], mul2(f, sn[e])));
                    }
                } else if (rot) {   // (x, y) (cos, cos) + (y, x) (-sin, sin)
#pragma unroll
                    for (int e = 0; e < VW / 2; ++e) {
                        const float2 f = Two<T>::get(p.e + 2 * e);
                        Two<T>::put(p.e + 2 * e, fma2(f, cs[e], mul2(make_float2(f.y, f.x), sn[e])));
                    }
                }
            }
            T* d;
            if (h < nq) {
                d = static_cast<T*>(a.query_out) + t * a.qo_t + h * a.qo_h;
            } else {
                if (state) return;
                d = static_cast<T*>(a.k_cache) + slots[2 * k] + (h - nq) * a.kc[2];
            }
            *reinterpret_cast<P*>(d + off) = p;
            if (halves) *reinterpret_cast<P*>(d + off + a.half) = q;
        };
        auto finish_value = [&](int i, const P& p) {
            const int h = quick_div(i, a.per_val, a.m_val);
            *reinterpret_cast<P*>(static_cast<T*>(a.v_cache) + slots[2 * k + 1] + h * a.vc[2] + (i - h * a.per_val) * VW) = p;
        };
#pragma unroll
        for (int j = 0; j < AT; ++j)
            if (hs + j * lanes < heads) finish(hs + j * lanes, x[j], y[j]);
        if (!state && int(threadIdx.x) < vals) finish_value(threadIdx.x, v);
        for (int h = hs + AT * lanes; h < heads; h += lanes) {
            load(t, h, x[0], y[0]);
            finish(h, x[0], y[0]);
        }
        for (int i = threadIdx.x + blockDim.x; !state && i < vals; i += blockDim.x) {
            load_value(t, i, v);
            finish_value(i, v);
        }
    }
}

// Keys and queries normed on the way: y = x / sqrt(mean(x^2) + eps) * weight over each head, in
// float32, then the rotation.  Bound by memory like appending without norms.  A head is one
// group of lanes (a power of two, so that its sum is a few shuffles), a lane has one unit of it (see unit_of):
// the unit's two words stay in registers between the sum and the rotation, and its
// weights, cosines and sines across the heads of a token.  ONE = false: heads of more units than lanes, read
// twice (the second time from L1).  8190 tokens of 32 + 8 + 8 heads of 128 in bf16: 44 us, 4.6 TB/s.
template <typename T, int VW, bool ONE>
__global__ void __launch_bounds__(256, 2) append_norm_kernel(const AppendArgs a) {
    extern __shared__ __align__(16) unsigned char smem[];
    int64_t* slots = reinterpret_cast<int64_t*>(smem);                  // [per_cta][2]
    int* pads = reinterpret_cast<int*>(slots + 2 * a.per_cta);          // [per_cta], padded to 8 bytes each
    float2* turns = reinterpret_cast<float2*>(slots + 3 * a.per_cta);   // [per_cta][half]
    using P = Pack<T, VW>;
    grid_dependency_wait();
    allow_dependents();
    const int t0 = blockIdx.x * a.per_cta, tokens = min(a.per_cta, a.tokens - t0);
    const int lane = threadIdx.x & (a.group - 1), hs = threadIdx.x / a.group, at_once = blockDim.x / a.group;
    const int nq = a.query ? a.q_heads : 0, heads = nq + a.kv_heads, vals = a.kv_heads * a.per_val;
    const float inv_dim = 1.f / float(a.dim);

    // Unit u of a head: its first element, its partner's (-1: none) and its first pair (-1: not rotated).
    auto place = [&](int u, int& off, int& off2, int& pair) {
        off2 = pair = -1;
        if (u >= a.per_pairs) {
            off = 2 * a.half + (u - a.per_pairs) * VW;
        } else if (!a.interleaved) {
            off = pair = u * VW;
            off2 = off + a.half;
        } else if (VW > 1) {
            off = u * VW;
            pair = off / 2;
        } else {
            off = 2 * u;
            off2 = off + 1;
            pair = u;
        }
    };
    auto head_at = [&](int t, int h) {
        return h < nq ? static_cast<const T*>(a.query) + t * a.q_t + h * a.q_h
                      : static_cast<const T*>(a.key) + t * a.key_t + (h - nq) * a.key_h;
    };
    auto load = [&](const T* p, int off, int off2, P& x, P& y) {
        x = *reinterpret_cast<const P*>(p + off);
        if (off2 >= 0) y = *reinterpret_cast<const P*>(p + off2);
    };
    auto squares = [&](const P& x, const P& y, bool both) {
        float s = 0.f;
#pragma unroll
        for (int e = 0; e < VW; ++e) s = fmaf(Io<T>::get(x.e[e]), Io<T>::get(x.e[e]), s);
        if (both) {
#pragma unroll
            for (int e = 0; e < VW; ++e) s = fmaf(Io<T>::get(y.e[e]), Io<T>::get(y.e[e]), s);
        }
        return s;
    };
    auto value_at = [&](int i, int& o) {
        const int h = quick_div(i, a.per_val, a.m_val);
        o = (i - h * a.per_val) * VW;
        return h;
    };
    // The first loads go out before anything depends on the positions.
    int off, off2, pair;
    place(lane, off, off2, pair);
    const bool mine = lane < a.per_rot;
    constexpr int AT = ONE ? 2 : 1;   // heads in flight per thread
    P x[AT], y[AT], v;
    auto load_token = [&](int t) {
        if (ONE && mine) {
#pragma unroll
            for (int j = 0; j < AT; ++j)
                if (hs + j * at_once < heads) load(head_at(t, hs + j * at_once), off, off2, x[j], y[j]);
        }
        if (int(threadIdx.x) < vals) {
            int o;
            const int h = value_at(threadIdx.x, o);
            v = *reinterpret_cast<const P*>(static_cast<const T*>(a.value) + t * a.val_t + h * a.val_h + o);
        }
    };
    load_token(t0);
    // This unit's weights, of queries and of keys.
    constexpr int KEEP = ONE ? VW : 1;
    float wq[2][KEEP] = {}, wk[2][KEEP] = {}, cs[KEEP] = {}, sn[KEEP] = {};
    if (ONE && mine) {
#pragma unroll
        for (int e = 0; e < KEEP; ++e) {
            wq[0][e] = a.q_weight ? a.q_weight[off + e] : 1.f;
            wk[0][e] = a.k_weight ? a.k_weight[off + e] : 1.f;
            wq[1][e] = a.q_weight && off2 >= 0 ? a.q_weight[off2 + e] : 1.f;
            wk[1][e] = a.k_weight && off2 >= 0 ? a.k_weight[off2 + e] : 1.f;
        }
    }
    if (int(threadIdx.x) < tokens) {
        const int t = t0 + threadIdx.x;
        const int pos = a.positions[t];
        const int row = a.rows ? a.rows[t] : t;
        const bool pad = pos < 0;
        const int pi = pad ? 0 : pos / a.page_size;
        int64_t k_at = 0, v_at = 0;
        bool there = false;
        if (!pad && row >= 0 && row < a.table_rows && pi < a.table_width) {
            const int page = a.table[int64_t(row) * a.table_width + pi];
            if (page >= 0 && page < a.num_pages) {
                const int slot = pos - pi * a.page_size;
                k_at = page * a.kc[0] + slot * a.kc[1];
                v_at = page * a.vc[0] + slot * a.vc[1];
                there = true;
            }
        }
        slots[2 * threadIdx.x] = k_at;
        slots[2 * threadIdx.x + 1] = v_at;
        pads[threadIdx.x] = pad ? 1 : (there ? 0 : 2);   // 1 padding, 2 not written
    }
    for (int i = threadIdx.x; i < tokens * a.half; i += blockDim.x) {
        const int k = i / a.half, t = t0 + k;
        const int pos = a.positions[t], rp = a.rotary_positions ? a.rotary_positions[t] : pos;
        turns[i] = pos < 0 ? make_float2(1.f, 0.f) : cos_sin_of(a.inv_freq[i - k * a.half], rp);
    }
    __syncthreads();

    // One unit of a head: scaled, weighted, rotated, stored.
    auto finish = [&](int k, int h, T* d, int off, int off2, int pair, P& x, P& y, float r) {
        const bool query = h < nq;
        const float* w = query ? a.q_weight : a.k_weight;
        const float2* turn = turns + k * a.half;
        if (!w) r = 1.f;
        // the e-th element of the unit's first or second word, normed
        auto normed = [&](T v, int e, int second) {
            const float f = Io<T>::get(v) * r;
            if constexpr (ONE) return f * (query ? wq[second][e] : wk[second][e]);
            else return w ? f * w[(second ? off2 : off) + e] : f;
        };
        auto cosine = [&](int e, int p) { if constexpr (ONE) return make_float2(cs[e], sn[e]); else return turn[p]; };
        if (pair >= 0 && off2 >= 0) {
#pragma unroll
            for (int e = 0; e < VW; ++e) {
                const float2 c = cosine(e, pair + e);
                const float f = normed(x.e[e], e, 0), g = normed(y.e[e], e, 1);
                x.e[e] = Io<T>::put(f * c.x - g * c.y);
                y.e[e] = Io<T>::put(g * c.x + f * c.y);
            }
        } else if (pair >= 0) {
#pragma unroll
            for (int e = 0; e + 1 < VW; e += 2) {
                const float2 c = cosine(e / 2, pair + e / 2);
                const float f = normed(x.e[e], e, 0), g = normed(x.e[e + 1], e + 1, 0);
                x.e[e] = Io<T>::put(f * c.x - g * c.y);
                x.e[e + 1] = Io<T>::put(g * c.x + f * c.y);
            }
        } else if (w) {
#pragma unroll
            for (int e = 0; e < VW; ++e) x.e[e] = Io<T>::put(normed(x.e[e], e, 0));
        }
        *reinterpret_cast<P*>(d + off) = x;
        if (off2 >= 0) *reinterpret_cast<P*>(d + off2) = y;
    };
    // A round of heads; whole warps, for the shuffles.  `there`: the units' words are in x and y.
    auto round = [&](int k, int t, int state, int h, P& x, P& y, bool there) {
        const bool on = h < heads;
        const T* p = head_at(t, on ? h : 0);
        float s = 0.f;
        if (ONE) {
            if (on && mine) {
                if (!there) load(p, off, off2, x, y);
                s = squares(x, y, off2 >= 0);
            }
        } else if (on) {
            for (int u = lane; u < a.per_rot; u += a.group) {
                int o1, o2, pr;
                place(u, o1, o2, pr);
                load(p, o1, o2, x, y);
                s += squares(x, y, o2 >= 0);
            }
        }
        for (int i = a.group >> 1; i > 0; i >>= 1) s += __shfl_xor_sync(FULL, s, i);
        if (!on || (h >= nq && state)) return;
        const float r = rsqrtf(fmaf(s, inv_dim, a.eps));
        T* d = h < nq ? static_cast<T*>(a.query_out) + t * a.qo_t + h * a.qo_h
                      : static_cast<T*>(a.k_cache) + slots[2 * k] + (h - nq) * a.kc[2];
        for (int u = lane; u < a.per_rot; u += a.group) {
            int o1 = off, o2 = off2, pr = pair;
            if (!ONE) {
                place(u, o1, o2, pr);
                load(p, o1, o2, x, y);
            }
            if (state != 1) {
                finish(k, h, d, o1, o2, pr, x, y, r);
            } else {   // padding: the query as it is
                *reinterpret_cast<P*>(d + o1) = x;
                if (o2 >= 0) *reinterpret_cast<P*>(d + o2) = y;
            }
        }
    };
#pragma unroll 1
    for (int k = 0; k < tokens; ++k) {
        const int t = t0 + k, state = pads[k];
        if (k > 0) load_token(t);
        if (ONE && mine && pair >= 0) {
#pragma unroll
            for (int e = 0; e < KEEP; ++e) {
                if (off2 < 0 && e >= (KEEP + 1) / 2) break;     // (neighbours: half as many pairs)
                const float2 c = turns[k * a.half + pair + e];
                cs[e] = c.x, sn[e] = c.y;
            }
        }
#pragma unroll
        for (int j = 0; j < AT; ++j) round(k, t, state, hs + j * at_once, x[j], y[j], ONE);
        for (int h0 = AT * at_once; h0 < heads; h0 += at_once) round(k, t, state, h0 + hs, x[0], y[0], false);
        for (int i = threadIdx.x; !state && i < vals; i += blockDim.x) {
            int o;
            const int h = value_at(i, o);
            if (i != int(threadIdx.x)) v = *reinterpret_cast<const P*>(static_cast<const T*>(a.value) + t * a.val_t + h * a.val_h + o);
            *reinterpret_cast<P*>(static_cast<T*>(a.v_cache) + slots[2 * k + 1] + h * a.vc[2] + o) = v;
        }
    }
}

template <typename T, int VW>
static fs_status launch_append(AppendArgs& a, void* stream) {
    int sms = 0;
    size_t optin = 0;
    const fs_status st = device_limits(sms, optin);
    if (st != FS_OK) return st;
    a.per_pairs = (a.interleaved && VW > 1) ? 2 * a.half / VW : a.half / VW;
    a.per_rot = a.per_pairs + (a.dim - 2 * a.half) / VW;
    a.per_val = a.dim / VW;
    const int64_t units = int64_t((a.query ? a.q_heads : 0) + a.kv_heads) * a.per_rot + int64_t(a.kv_heads) * a.per_val;
    a.units = int(units);
    const int heads = (a.query ? a.q_heads : 0) + a.kv_heads;
    int threads;
    int64_t per;   // tokens of a CTA, as long as every SM still gets four (eight) CTAs
    if (VW > 1) {
        // Whole rounds of heads: as few as 256 threads take, each as full as the others.
        const int rounds = (heads * a.per_rot + 255) / 256;
        const int at_once = std::min(256 / a.per_rot, (heads + rounds - 1) / rounds);
        threads = (at_once * a.per_rot + 31) / 32 * 32;
        per = std::min<int64_t>(4, a.tokens / (int64_t(sms) * 4));
    } else {
        threads = int(std::min<int64_t>(256, (units + 31) / 32 * 32));
        per = std::min<int64_t>((2048 + units - 1) / units, a.tokens / (int64_t(sms) * 8));
    }
    if (a.half > 0) per = std::min<int64_t>(per, 4096 / a.half);
    a.per_cta = int(std::max<int64_t>(1, std::min<int64_t>(per, 16)));
    const int64_t most = units * a.per_cta;
    a.m_units = magic_of(uint32_t(units), uint64_t(most));
    a.m_rot = magic_of(uint32_t(a.per_rot), uint64_t(units));
    a.m_val = magic_of(uint32_t(a.per_val), uint64_t(units));
    const bool norm = a.q_weight || a.k_weight;
    if (norm) {
        a.group = 1;
        while (a.group < a.per_rot && a.group < 32) a.group *= 2;
        // Whole rounds of heads, as above.
        const int rounds = (heads * a.group + 255) / 256, at_once = (heads + rounds - 1) / rounds;
        threads = (at_once * a.group + 31) / 32 * 32;
    }
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(unsigned((a.tokens + a.per_cta - 1) / a.per_cta), 1, 1);
    cfg.blockDim = dim3(unsigned(threads), 1, 1);
    cfg.dynamicSmemBytes = size_t(a.per_cta) * (32 + size_t(a.half) * sizeof(float2));
    cfg.stream = static_cast<cudaStream_t>(stream);
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    cudaError_t e;
    if (norm) e = a.per_rot <= a.group ? cudaLaunchKernelEx(&cfg, append_norm_kernel<T, VW, true>, a)
                                       : cudaLaunchKernelEx(&cfg, append_norm_kernel<T, VW, false>, a);
    else if constexpr (VW > 1) e = cudaLaunchKernelEx(&cfg, append_heads_kernel<T, VW>, a);
    else e = cudaLaunchKernelEx(&cfg, append_kernel<T, VW>, a);
    return e == cudaSuccess ? FS_OK : cuda_fail(e);
}

static fs_status append(const fs_paged_kv* cache, const void* key, const int64_t* key_strides, const void* value,
                        const int64_t* value_strides, int32_t tokens, const int32_t* page_table, int32_t table_rows,
                        int32_t table_width, const int32_t* rows, const int32_t* positions, const int32_t* rotary_positions,
                        const float* inv_freq, int32_t rotary_dim, int32_t interleaved, const void* query,
                        const int64_t* query_strides, int32_t q_heads, void* query_out, const int64_t* query_out_strides,
                        const float* query_weight, const float* key_weight, float eps, void* stream) {
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
    a.q_weight = query ? query_weight : nullptr;
    a.k_weight = key_weight;
    a.eps = eps;
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

}  // namespace fsd

extern "C" {

fs_status fs_append_paged_kv(const fs_paged_kv* cache, const void* key, const int64_t* key_strides, const void* value,
                             const int64_t* value_strides, int32_t tokens, const int32_t* page_table,
                             int32_t table_rows, int32_t table_width, const int32_t* rows, const int32_t* positions,
                             const int32_t* rotary_positions, const float* inv_freq, int32_t rotary_dim,
                             int32_t interleaved, const void* query, const int64_t* query_strides, int32_t q_heads,
                             void* query_out, const int64_t* query_out_strides, void* stream) {
    return fsd::append(cache, key, key_strides, value, value_strides, tokens, page_table, table_rows, table_width, rows, positions,
                       rotary_positions, inv_freq, rotary_dim, interleaved, query, query_strides, q_heads, query_out,
                       query_out_strides, nullptr, nullptr, 0.f, stream);
}

fs_status fs_append_paged_kv_normed(const fs_paged_kv* cache, const void* key, const int64_t* key_strides, const void* value,
                                    const int64_t* value_strides, int32_t tokens, const int32_t* page_table,
                                    int32_t table_rows, int32_t table_width, const int32_t* rows,
                                    const int32_t* positions, const int32_t* rotary_positions, const float* inv_freq,
                                    int32_t rotary_dim, int32_t interleaved, const void* query,
                                    const int64_t* query_strides, int32_t q_heads, void* query_out,
                                    const int64_t* query_out_strides, const float* query_weight, const float* key_weight,
                                    float eps, void* stream) {
    if (!(eps >= 0.f) || (query_weight && !query)) return FS_ERR_INVALID_ARG;
    return fsd::append(cache, key, key_strides, value, value_strides, tokens, page_table, table_rows, table_width, rows, positions,
                       rotary_positions, inv_freq, rotary_dim, interleaved, query, query_strides, q_heads, query_out,
                       query_out_strides, query_weight, key_weight, eps, stream);
}

}  // extern "C"
