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

// Where token t of a CTA's goes: its cache offsets, and 1 padding, 2 not written (a row or page that does not exist).
__device__ __forceinline__ int place_of(const AppendArgs& a, int t, int64_t& k_at, int64_t& v_at) {
    const int pos = a.positions[t], row = a.rows ? a.rows[t] : t;
    k_at = v_at = 0;
    if (pos < 0) return 1;
    const int pi = pos / a.page_size;
    if (row < 0 || row >= a.table_rows || pi >= a.table_width) return 2;
    const int page = a.table[int64_t(row) * a.table_width + pi];
    if (page < 0 || page >= a.num_pages) return 2;
    const int slot = pos - pi * a.page_size;
    k_at = page * a.kc[0] + slot * a.kc[1];
    v_at = page * a.vc[0] + slot * a.vc[1];
    return 0;
}

// Keys and queries normed on the way: y = x / sqrt(mean(x^2) + eps) * weight over each head, in float32, then the
// rotation.  Aligned data, heads of up to 32 units.  Bound by memory like appending without norms.  A head is one group
// of lanes (a power of two, so that its sum is a few shuffles), a lane has one unit of it: VW elements and, for a
// rotation in halves, their partners, which stay in registers between the sum and the rotation.  Norm
// and rotation are two products and a sum per element,
//   x' = r (x A - y B),  y' = r (y C + x D),  A = w_x cos, B = w_y sin, C = w_y cos, D = w_x sin,
// with r the head's scale and the coefficients in registers over a token's heads, queries first, then keys.  One or a few warps
// have a token, so that the coefficients are made once or a few times for it: with all eight warps of a CTA on a
// token their reads from L1 took 84 us for the 8190 tokens below.  8190 tokens of 32 + 8 + 8 heads of 128 in
// bf16: 49 us, 4.1 TB/s.
template <typename T, int VW>
__global__ void __launch_bounds__(256, 3) append_norm_heads_kernel(const AppendArgs a) {
    extern __shared__ __align__(16) unsigned char smem[];
    int64_t* slots = reinterpret_cast<int64_t*>(smem);                  // [per_cta][2]
    int* pads = reinterpret_cast<int*>(slots + 2 * a.per_cta);          // [per_cta], padded to 8 bytes each
    float* cosines = reinterpret_cast<float*>(slots + 4 * a.per_cta);   // [per_cta][half]
    float* sines = cosines + a.per_cta * a.half;
    using P = Pack<T, VW>;
    constexpr int H = VW / 2;
    grid_dependency_wait();
    allow_dependents();
    const int t0 = blockIdx.x * a.per_cta, tokens = min(a.per_cta, a.tokens - t0);
    // 256 / per_cta threads a token
    const int each = 256 / a.per_cta, k = threadIdx.x / each, me = threadIdx.x - k * each, t = t0 + k;
    const int lane = me & (a.group - 1), hs = me / a.group, at_once = each / a.group;
    const int nq = a.query ? a.q_heads : 0, vals = a.kv_heads * a.per_val;
    const float inv_dim = 1.f / float(a.dim);
    const bool here = k < tokens, mine = here && lane < a.per_rot, rot = lane < a.per_pairs, halves = rot && !a.interleaved;
    const int off = rot ? lane * VW : 2 * a.half + (lane - a.per_pairs) * VW;

    auto load = [&](int side, int h, P& x, P& y) {
        const T* p = side == 0 ? static_cast<const T*>(a.query) + t * a.q_t + h * a.q_h
                               : static_cast<const T*>(a.key) + t * a.key_t + h * a.key_h;
        x = *reinterpret_cast<const P*>(p + off);
        if (halves) y = *reinterpret_cast<const P*>(p + off + a.half);
    };
    auto load_value = [&](int i, P& v) {
        const int h = quick_div(i, a.per_val, a.m_val);
        v = *reinterpret_cast<const P*>(static_cast<const T*>(a.value) + t * a.val_t + h * a.val_h + (i - h * a.per_val) * VW);
    };
    // The first loads go out before anything depends on the positions: a head of each side, a piece of the values.
    P x[2], y[2], v;
    if (mine && hs < nq) load(0, hs, x[0], y[0]);
    if (mine && hs < a.kv_heads) load(1, hs, x[1], y[1]);
    if (here && me < vals) load_value(me, v);
    if (int(threadIdx.x) < tokens) pads[threadIdx.x] = place_of(a, t0 + threadIdx.x, slots[2 * threadIdx.x], slots[2 * threadIdx.x + 1]);
    for (int i = threadIdx.x; i < tokens * a.half; i += 256) {
        const int j = i / a.half, u = t0 + j;
        const int pos = a.positions[u], rp = a.rotary_positions ? a.rotary_positions[u] : pos;
        const float2 w = pos < 0 ? make_float2(1.f, 0.f) : cos_sin_of(a.inv_freq[i - j * a.half], rp);
        cosines[i] = w.x;
        sines[i] = w.y;
    }
    __syncthreads();
    const int state = here ? pads[k] : 2;
#pragma unroll
    for (int side = 0; side < 2; ++side) {
        const int heads = side == 0 ? nq : a.kv_heads;
        const float* w = side == 0 ? a.q_weight : a.k_weight;
        // this unit's coefficients
        float2 A[H], B[H], C[H], E[H];
        if (mine) {
            const float* cp = cosines + k * a.half + (a.interleaved ? off / 2 : off);
            const float* sp = sines + k * a.half + (a.interleaved ? off / 2 : off);
#pragma unroll
            for (int e = 0; e < H; ++e) {
                const float2 one = make_float2(1.f, 1.f), wx = w ? *reinterpret_cast<const float2*>(w + off + 2 * e) : one;
                if (halves) {
                    const float2 wy = w ? *reinterpret_cast<const float2*>(w + off + a.half + 2 * e) : one;
                    const float2 c = *reinterpret_cast<const float2*>(cp + 2 * e), s = *reinterpret_cast<const float2*>(sp + 2 * e);
                    A[e] = make_float2(wx.x * c.x, wx.y * c.y);
                    B[e] = make_float2(-wy.x * s.x, -wy.y * s.y);
                    C[e] = make_float2(wy.x * c.x, wy.y * c.y);
                    E[e] = make_float2(wx.x * s.x, wx.y * s.y);
                } else {    // (x, y) becomes (x, y) A + (y, x) B
                    const float c = rot ? cp[e] : 1.f, s = rot ? sp[e] : 0.f;
                    A[e] = make_float2(wx.x * c, wx.y * c);
                    B[e] = make_float2(-wx.y * s, wx.x * s);
                }
            }
        }
        P p = x[side], q = y[side];
#pragma unroll 1
        for (int h0 = 0; h0 < heads; h0 += at_once) {   // (whole warps, for the shuffles)
            const int h = h0 + hs;
            const bool on = h < heads && mine;
            P np, nq2;      // the next head is on its way
            if (mine && h + at_once < heads) load(side, h + at_once, np, nq2);
            float2 s2 = make_float2(0.f, 0.f);
            if (on) {
#pragma unroll
                for (int e = 0; e < H; ++e) {
                    const float2 f = Two<T>::get(p.e + 2 * e);
                    s2 = fma2(f, f, s2);
                    if (halves) {
                        const float2 g = Two<T>::get(q.e + 2 * e);
                        s2 = fma2(g, g, s2);
                    }
                }
            }
            float s = s2.x + s2.y;
            for (int i = a.group >> 1; i > 0; i >>= 1) s += __shfl_xor_sync(FULL, s, i);
            if (on && !(side == 1 && state)) {
                if (state != 1) {   // (padding: the query as it is)
                    const float r1 = w ? rsqrtf(fmaf(s, inv_dim, a.eps)) : 1.f;
                    const float2 r = make_float2(r1, r1);
#pragma unroll
                    for (int e = 0; e < H; ++e) {
                        const float2 f = Two<T>::get(p.e + 2 * e);
                        if (halves) {
                            const float2 g = Two<T>::get(q.e + 2 * e);
                            Two<T>::put(p.e + 2 * e, mul2(r, fma2(f, A[e], mul2(g, B[e]))));
                            Two<T>::put(q.e + 2 * e, mul2(r, fma2(g, C[e], mul2(f, E[e]))));
                        } else if (rot) {
                            Two<T>::put(p.e + 2 * e, mul2(r, fma2(f, A[e], mul2(make_float2(f.y, f.x), B[e]))));
                        } else if (w) {
                            Two<T>::put(p.e + 2 * e, mul2(r, mul2(f, A[e])));
                        }
                    }
                }
                T* d = side == 0 ? static_cast<T*>(a.query_out) + t * a.qo_t + h * a.qo_h
                                 : static_cast<T*>(a.k_cache) + slots[2 * k] + h * a.kc[2];
                *reinterpret_cast<P*>(d + off) = p;
                if (halves) *reinterpret_cast<P*>(d + off + a.half) = q;
            }
            p = np, q = nq2;
        }
    }
    for (int i = me; !state && i < vals; i += each) {
        if (i != me) load_value(i, v);
        const int h = quick_div(i, a.per_val, a.m_val);
        *reinterpret_cast<P*>(static_cast<T*>(a.v_cache) + slots[2 * k + 1] + h * a.vc[2] + (i - h * a.per_val) * VW) = v;
    }
}

// The same for any alignment (VW = 1) and longer heads: a head's units are read twice, the second time from L1.
template <typename T, int VW>
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
    if (int(threadIdx.x) < tokens) pads[threadIdx.x] = place_of(a, t0 + threadIdx.x, slots[2 * threadIdx.x], slots[2 * threadIdx.x + 1]);
    for (int i = threadIdx.x; i < tokens * a.half; i += blockDim.x) {
        const int k = i / a.half, t = t0 + k;
        const int pos = a.positions[t], rp = a.rotary_positions ? a.rotary_positions[t] : pos;
        turns[i] = pos < 0 ? make_float2(1.f, 0.f) : cos_sin_of(a.inv_freq[i - k * a.half], rp);
    }
    __syncthreads();
#pragma unroll 1
    for (int k = 0; k < tokens; ++k) {
        const int t = t0 + k, state = pads[k];
        const float2* turn = turns + k * a.half;
        for (int h0 = 0; h0 < heads; h0 += at_once) {   // (whole warps, for the shuffles)
            const int h = h0 + hs;
            const bool on = h < heads;
            const T* src = !on || h < nq ? static_cast<const T*>(a.query) + t * a.q_t + (on ? h : 0) * a.q_h
                                         : static_cast<const T*>(a.key) + t * a.key_t + (h - nq) * a.key_h;
            const float* w = h < nq ? a.q_weight : a.k_weight;
            float s = 0.f;
            for (int u = lane; on && u < a.per_rot; u += a.group) {
                int off, off2, pair;
                place(u, off, off2, pair);
                const P x = *reinterpret_cast<const P*>(src + off);
#pragma unroll
                for (int e = 0; e < VW; ++e) s = fmaf(Io<T>::get(x.e[e]), Io<T>::get(x.e[e]), s);
                if (off2 >= 0) {
                    const P y = *reinterpret_cast<const P*>(src + off2);
#pragma unroll
                    for (int e = 0; e < VW; ++e) s = fmaf(Io<T>::get(y.e[e]), Io<T>::get(y.e[e]), s);
                }
            }
            for (int i = a.group >> 1; i > 0; i >>= 1) s += __shfl_xor_sync(FULL, s, i);
            if (!on || (h >= nq && state)) continue;
            const float r = w ? rsqrtf(fmaf(s, inv_dim, a.eps)) : 1.f;
            T* d = h < nq ? static_cast<T*>(a.query_out) + t * a.qo_t + h * a.qo_h
                          : static_cast<T*>(a.k_cache) + slots[2 * k] + (h - nq) * a.kc[2];
            auto normed = [&](T v, int i) { return w ? Io<T>::get(v) * r * w[i] : Io<T>::get(v); };
            for (int u = lane; u < a.per_rot; u += a.group) {
                int off, off2, pair;
                place(u, off, off2, pair);
                P x = *reinterpret_cast<const P*>(src + off), y = x;
                if (off2 >= 0) y = *reinterpret_cast<const P*>(src + off2);
                if (state == 1) {
                    // padding: the query as it is
                } else if (off2 >= 0) {
#pragma unroll
                    for (int e = 0; e < VW; ++e) {
                        const float2 c = turn[pair + e];
                        const float f = normed(x.e[e], off + e), g = normed(y.e[e], off2 + e);
                        x.e[e] = Io<T>::put(f * c.x - g * c.y);
                        y.e[e] = Io<T>::put(g * c.x + f * c.y);
                    }
                } else if (pair >= 0) {
#pragma unroll
                    for (int e = 0; e + 1 < VW; e += 2) {
                        const float2 c = turn[pair + e / 2];
                        const float f = normed(x.e[e], off + e), g = normed(x.e[e + 1], off + e + 1);
                        x.e[e] = Io<T>::put(f * c.x - g * c.y);
                        x.e[e + 1] = Io<T>::put(g * c.x + f * c.y);
                    }
                } else if (w) {
#pragma unroll
                    for (int e = 0; e < VW; ++e) x.e[e] = Io<T>::put(normed(x.e[e], off + e));
                }
                *reinterpret_cast<P*>(d + off) = x;
                if (off2 >= 0) *reinterpret_cast<P*>(d + off2) = y;
            }
        }
        for (int i = threadIdx.x; !state && i < vals; i += blockDim.x) {
            const int h = quick_div(i, a.per_val, a.m_val), o = (i - h * a.per_val) * VW;
            *reinterpret_cast<P*>(static_cast<T*>(a.v_cache) + slots[2 * k + 1] + h * a.vc[2] + o) =
                *reinterpret_cast<const P*>(static_cast<const T*>(a.value) + t * a.val_t + h * a.val_h + o);
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
    bool wide = false;  // append_norm_heads_kernel
    if (norm) {
        a.group = 1;
        while (a.group < a.per_rot && a.group < 32) a.group *= 2;
        threads = 256;
        if constexpr (VW > 1) wide = a.per_rot <= 32 && ((reinterpret_cast<uintptr_t>(a.q_weight) | reinterpret_cast<uintptr_t>(a.k_weight)) & 7) == 0;
        if (wide) {     // one, two or four tokens, as long as every SM still gets four CTAs
            a.per_cta = 1;
            while (a.per_cta < 4 && a.tokens >= int64_t(sms) * 8 * a.per_cta) a.per_cta *= 2;
        }
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
    if (norm && !wide) e = cudaLaunchKernelEx(&cfg, append_norm_kernel<T, VW>, a);
    else if constexpr (VW > 1) e = norm ? cudaLaunchKernelEx(&cfg, append_norm_heads_kernel<T, VW>, a)
                                        : cudaLaunchKernelEx(&cfg, append_heads_kernel<T, VW>, a);
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
