// Sampling with temperature, top-k, top-p and min-p from given random numbers (sm_103a).
//
// One number u in [0, 1) per output row decides its token.  With w_i = exp((z_i - m) / T),
// m the row's maximum, and S the kept set (every filter is a threshold on z), the token is
//   the first i of S, in index order, with  sum_{j in S, j <= i} w_j > u * sum_{j in S} w_j.
// Unlike the rejection sampler this needs the masses themselves, not only an accepted
// draw, and the decisions (which token the top-p mass ends on, which token u falls on)
// are borders between neighbours that may differ by 10^-6 of the row: a float32 sum would
// answer another token for flat rows.  So weights are 64-bit fixed-point integers, 2^42 w to
// a relative 5e-10 (2e-10 rms) and half a unit (weight_of), and every sum and
// comparison is exact integer arithmetic.  Sums then do not depend on their order, the
// launch shape or atomics.
//
// Two launches.  seg_max_kernel streams every input row once, spread evenly over the GPU,
// and writes the largest order key of each segment (one 16-byte load per lane of a warp).
// uniform_kernel, one cluster of C CTAs per output row, reads those keys and then:
//   small sets  top-k: the segments whose maximum reaches the k-th largest segment maximum hold
//               every element of the top k; min-p: those whose maximum reaches the
//               threshold hold every kept element.  Their elements at or above the bound (for top-k
//               a few dozen more than k) go into a list in shared memory in index
//               order, and every decision is made there.  The whole row's mass, where top-p is
//               measured against it, is a float32 sum with a bound on its error; only a row with a
//               candidate inside that bound sums its weights exactly.
//   other sets  a histogram of the weights over bins linear in m - z finds the bin a
//               threshold lies in; one more pass lists that bin's elements and sums the masses of
//               the elements above it per segment; the list decides the threshold.  Bins too full for the list (16-bit
//               logits tie by thousands) are narrowed by histograms over the order keys.
//               The token is found from the segments' masses and one read of its segment.
// Back to back on a GB300: 64 rows of 151936 float32, top-k 50 and top-p 0.9, 15.6 us (a copy of
// the input at the memory's rate: 5.7); 64 of 151665 bf16, top-p 0.95, 61 to 72 (by the lists that the slowest row takes); 512 of 128256 f16 (128 rows),
// min-p about 0.05, 41; 256 of 256000 bf16, all filters in the joint order, 72.  Small sets are bound
// by the chain of barriers behind the scan, other sets by instructions (120 a logit).
#include <algorithm>

#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include <type_traits>

#include "fs_device.cuh"
#include "fs_host.h"

namespace fsd {

constexpr int UNT = 512;          // threads of uniform_kernel
constexpr int UNW = UNT / 32;
constexpr int UB = 2048;          // histogram bins (of the linear ones, 1377 are used)
constexpr int UCAP = 1024;        // candidates in a list
constexpr int USEG_TRIP = 4;      // segments a warp has in flight
constexpr uint32_t KEY_NINF = 0x007fffffu;  // order keys of -inf and +inf (a NaN's is above the latter or below the former)
constexpr uint32_t KEY_PINF = 0xff800000u;

struct UniformArgs {
    const void* x;              // [batch_in][stride] logits
    int64_t stride;
    int batch_in, V;
    const int* indices;         // nullable
    int nout;
    const float* u;
    const float* temperature;   // the rest nullable
    const int* top_k;
    const float* top_p;
    const float* min_p;
    int order;                  // 0 top_k_first, 1 joint
    int* out_token;
    unsigned char* out_valid;
    uint32_t* skey;             // [batch_in][ls] segment maxima
    float* ssum;                // [batch_in][ls] sums of exp((z - segment maximum) / T), nullable
    int ls;                     // segments of a row, at most
    int nsc;                    // segments per CTA of a cluster, at most
};

// ------------------------------------------------------------------ elements

// A row as words of 16 bytes: position p = index + a0, where a0 elements of the first
// word lie before the row.  Words inside the row are loaded whole, the words at its two
// ends element by element; elements outside the row read as -inf.
template <typename T>
struct URow {
    static constexpr int N = 16 / int(sizeof(T));  // elements per word
    static constexpr int SEG = 32 * N;             // positions per segment
    const T* x;
    int a0, end, nseg;
    __device__ __forceinline__ URow(const void* base, int64_t stride, int r, int V) {
        x = static_cast<const T*>(base) + r * stride;
        a0 = int((reinterpret_cast<uintptr_t>(x) & 15) / sizeof(T));
        end = a0 + V;
        nseg = (end + SEG - 1) / SEG;
    }
    __device__ __forceinline__ uint4 load(int seg, int lane) const {
        const int p = seg * SEG + lane * N;
        if (p >= a0 && p + N <= end) return __ldg(reinterpret_cast<const uint4*>(x + (p - a0)));
        uint4 w;
        T* e = reinterpret_cast<T*>(&w);
#pragma unroll
        for (int i = 0; i < N; ++i) e[i] = p + i >= a0 && p + i < end ? x[p + i - a0] : T(-INFINITY);
        return w;
    }
};
__device__ __forceinline__ void unpack(const uint4& w, float (&z)[4], float) {
    z[0] = __uint_as_float(w.x), z[1] = __uint_as_float(w.y), z[2] = __uint_as_float(w.z), z[3] = __uint_as_float(w.w);
}
__device__ __forceinline__ void unpack(const uint4& w, float (&z)[8], __nv_bfloat16) {
    const uint32_t u[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        z[2 * i] = __uint_as_float(u[i] << 16);
        z[2 * i + 1] = __uint_as_float(u[i] & 0xffff0000u);
    }
}
__device__ __forceinline__ void unpack(const uint4& w, float (&z)[8], __half) {
    const uint32_t u[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&u[i]));
        z[2 * i] = f.x;
        z[2 * i + 1] = f.y;
    }
}
// Element e of a word, e not known at compile time.
__device__ __forceinline__ float element(const uint4& w, int e, float) {
    return __uint_as_float(e < 2 ? (e == 0 ? w.x : w.y) : (e == 2 ? w.z : w.w));
}
template <typename H>
__device__ __forceinline__ uint32_t half_of(const uint4& w, int e, H) {
    const uint32_t v = e < 4 ? (e < 2 ? w.x : w.y) : (e < 6 ? w.z : w.w);
    return e & 1 ? v >> 16 : v & 0xffffu;
}
__device__ __forceinline__ float element(const uint4& w, int e, __nv_bfloat16 t) { return __uint_as_float(half_of(w, e, t) << 16); }
__device__ __forceinline__ float element(const uint4& w, int e, __half t) {
    return __half2float(__ushort_as_half((unsigned short)half_of(w, e, t)));
}
// The largest element of a word, NaN if one is.
__device__ __forceinline__ float max_nan(float x, float y) {
    float r;
    asm("max.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(x), "f"(y));
    return r;
}
__device__ __forceinline__ float max_of(const uint4& w, float) {
    return max_nan(max_nan(__uint_as_float(w.x), __uint_as_float(w.y)), max_nan(__uint_as_float(w.z), __uint_as_float(w.w)));
}
__device__ __forceinline__ float max_of(const uint4& w, __nv_bfloat16) {
    uint32_t x, y;
    asm("max.NaN.bf16x2 %0, %1, %2;" : "=r"(x) : "r"(w.x), "r"(w.y));
    asm("max.NaN.bf16x2 %0, %1, %2;" : "=r"(y) : "r"(w.z), "r"(w.w));
    asm("max.NaN.bf16x2 %0, %1, %2;" : "=r"(x) : "r"(x), "r"(y));
    return max_nan(__uint_as_float(x << 16), __uint_as_float(x & 0xffff0000u));
}
__device__ __forceinline__ float max_of(const uint4& w, __half) {
    uint32_t x, y;
    asm("max.NaN.f16x2 %0, %1, %2;" : "=r"(x) : "r"(w.x), "r"(w.y));
    asm("max.NaN.f16x2 %0, %1, %2;" : "=r"(y) : "r"(w.z), "r"(w.w));
    asm("max.NaN.f16x2 %0, %1, %2;" : "=r"(x) : "r"(x), "r"(y));
    const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&x));
    return max_nan(f.x, f.y);
}
// A bound for `hits`: rounded down to the type.
__device__ __forceinline__ uint32_t bound_of(float z, float) { return __float_as_uint(z); }
__device__ __forceinline__ uint32_t bound_of(float z, __nv_bfloat16) {
    const uint32_t h = __bfloat16_as_ushort(__float2bfloat16_rd(z));
    return h | h << 16;
}
__device__ __forceinline__ uint32_t bound_of(float z, __half) {
    const uint32_t h = __half_as_ushort(__float2half_rd(z));
    return h | h << 16;
}
// Bit e: element e of the word is at or above the bound (a NaN never is).  The 16-bit types compare two at a time.
__device__ __forceinline__ uint32_t hits(const uint4& w, uint32_t bound, float) {
    const float z = __uint_as_float(bound);
    return (__uint_as_float(w.x) >= z ? 1u : 0u) | (__uint_as_float(w.y) >= z ? 2u : 0u) |
           (__uint_as_float(w.z) >= z ? 4u : 0u) | (__uint_as_float(w.w) >= z ? 8u : 0u);
}
__device__ __forceinline__ uint32_t squeeze(uint32_t x, uint32_t y, uint32_t z, uint32_t w) {
    // words of 0xffff where a half passes: bits 2 j of the low halves, 2 j + 1 of the high ones
    const uint32_t m = (x & 0x00010001u) | (y & 0x00040004u) | (z & 0x00100010u) | (w & 0x00400040u);
    return (m | m >> 15) & 0xffu;
}
__device__ __forceinline__ uint32_t hits(const uint4& w, uint32_t bound, __nv_bfloat16) {
    const __nv_bfloat162 z = *reinterpret_cast<const __nv_bfloat162*>(&bound);
    const __nv_bfloat162* h = reinterpret_cast<const __nv_bfloat162*>(&w);
    return squeeze(__hge2_mask(h[0], z), __hge2_mask(h[1], z), __hge2_mask(h[2], z), __hge2_mask(h[3], z));
}
__device__ __forceinline__ uint32_t hits(const uint4& w, uint32_t bound, __half) {
    const __half2 z = *reinterpret_cast<const __half2*>(&bound);
    const __half2* h = reinterpret_cast<const __half2*>(&w);
    return squeeze(__hge2_mask(h[0], z), __hge2_mask(h[1], z), __hge2_mask(h[2], z), __hge2_mask(h[3], z));
}
// Order key with -0 equal to +0.
__device__ __forceinline__ uint32_t ukey(float z) { return logit_key(z + 0.f); }
__device__ __forceinline__ float exp2_approx(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

// ------------------------------------------------------------------ segment maxima

// Warp w of the grid takes trips of USEG_TRIP segments w, w + W, ...; bound by the HBM
// read: 64 rows of 151936 float32 in about 7 us cold, 256 of 256000 bf16 with SUMS in 37 (a grid of
// eight CTAs an SM, more than are resident at once, did better than one wave, and than the
// next trip's loads held in registers).  A NaN marks its segment with the largest key.
// With SUMS also each segment's float32 mass relative to its own maximum, at the row's
// temperature (rows map one to one): the total mass then takes no second read.
template <typename T, bool SUMS>
__global__ void __launch_bounds__(256) seg_max_kernel(const UniformArgs a) {
    using R = URow<T>;
    grid_dependency_wait();
    allow_dependents();
    const int lane = threadIdx.x & 31;
    const int trips = (a.ls + USEG_TRIP - 1) / USEG_TRIP;
    const uint32_t total = uint32_t(a.batch_in) * uint32_t(trips);   // (of 2 KB each: far below 2^32)
    for (uint32_t w = blockIdx.x * 8 + (threadIdx.x >> 5); w < total; w += gridDim.x * 8) {
        const int r = int(w / uint32_t(trips)), s0 = int(w - uint32_t(r) * uint32_t(trips)) * USEG_TRIP;
        const R row(a.x, a.stride, r, a.V);
        uint4 v[USEG_TRIP];
#pragma unroll
        for (int j = 0; j < USEG_TRIP; ++j)
            if (s0 + j < row.nseg) v[j] = row.load(s0 + j, lane);
#pragma unroll
        for (int j = 0; j < USEG_TRIP; ++j) {
            if (s0 + j >= row.nseg) continue;
            const float top = max_of(v[j], T());
            const uint32_t k = warp_max_u(top == top ? ukey(top) : 0xffffffffu);
            if (lane == 0) a.skey[int64_t(r) * a.ls + s0 + j] = k;
            if (SUMS) {
                // Without a finite logit nothing; a NaN (a row with one, or an infinite temperature) makes the sum NaN.
                const float c = 1.44269504f / (a.temperature ? a.temperature[r] : 1.f), mc = from_logit_key(k);
                float z[R::N], sum = 0.f;
                unpack(v[j], z, T());
#pragma unroll
                for (int e = 0; e < R::N; ++e) sum += exp2_approx((z[e] - mc) * c);
                sum = warp_sum(sum);
                if (lane == 0) a.ssum[int64_t(r) * a.ls + s0 + j] = k > KEY_NINF ? sum : 0.f;
            }
        }
    }
}

// ------------------------------------------------------------------ weights

// 2^(j / 256) * 2^31, rounded.
__constant__ uint32_t EXP2_256[256] = {
    0x80000000u, 0x8058d7d3u, 0x80b1ed50u, 0x810b40a2u, 0x8164d1f4u, 0x81bea171u, 0x8218af43u, 0x8272fb98u,
    0x82cd8699u, 0x83285072u, 0x8383594fu, 0x83dea15cu, 0x843a28c4u, 0x8495efb3u, 0x84f1f656u, 0x854e3cd9u,
    0x85aac368u, 0x86078a2fu, 0x8664915cu, 0x86c1d91au, 0x871f6197u, 0x877d2affu, 0x87db3580u, 0x88398147u,
    0x88980e81u, 0x88f6dd5bu, 0x8955ee03u, 0x89b540a8u, 0x8a14d575u, 0x8a74ac9au, 0x8ad4c645u, 0x8b3522a4u,
    0x8b95c1e4u, 0x8bf6a435u, 0x8c57c9c4u, 0x8cb932c2u, 0x8d1adf5bu, 0x8d7ccfc1u, 0x8ddf0420u, 0x8e417ca9u,
    0x8ea4398bu, 0x8f073af6u, 0x8f6a8118u, 0x8fce0c22u, 0x9031dc43u, 0x9095f1acu, 0x90fa4c8cu, 0x915eed14u,
    0x91c3d374u, 0x9228ffdcu, 0x928e727eu, 0x92f42b89u, 0x935a2b2fu, 0x93c071a1u, 0x9426ff10u, 0x948dd3adu,
    0x94f4efa9u, 0x955c5337u, 0x95c3fe87u, 0x962bf1ccu, 0x96942d37u, 0x96fcb0fbu, 0x97657d4au, 0x97ce9256u,
    0x9837f052u, 0x98a1976fu, 0x990b87e2u, 0x9975c1ddu, 0x99e04593u, 0x9a4b1337u, 0x9ab62afdu, 0x9b218d17u,
    0x9b8d39bau, 0x9bf93119u, 0x9c657368u, 0x9cd200dcu, 0x9d3ed9a7u, 0x9dabfdffu, 0x9e196e19u, 0x9e872a27u,
    0x9ef53261u, 0x9f6386f9u, 0x9fd22825u, 0xa041161bu, 0xa0b05110u, 0xa11fd938u, 0xa18faecbu, 0xa1ffd1fcu,
    0xa2704303u, 0xa2e10215u, 0xa3520f69u, 0xa3c36b34u, 0xa43515aeu, 0xa4a70f0du, 0xa5195787u, 0xa58bef53u,
    0xa5fed6aau, 0xa6720dc1u, 0xa6e594d0u, 0xa7596c0fu, 0xa7cd93b5u, 0xa8420bfau, 0xa8b6d516u, 0xa92bef42u,
    0xa9a15ab5u, 0xaa1717a8u, 0xaa8d2653u, 0xab0386efu, 0xab7a39b6u, 0xabf13edfu, 0xac6896a5u, 0xace04140u,
    0xad583eeau, 0xadd08fddu, 0xae493453u, 0xaec22c85u, 0xaf3b78adu, 0xafb51907u, 0xb02f0dccu, 0xb0a95736u,
    0xb123f582u, 0xb19ee8e9u, 0xb21a31a6u, 0xb295cff6u, 0xb311c413u, 0xb38e0e38u, 0xb40aaea2u, 0xb487a58du,
    0xb504f334u, 0xb58297d4u, 0xb60093a8u, 0xb67ee6efu, 0xb6fd91e3u, 0xb77c94c3u, 0xb7fbefcbu, 0xb87ba338u,
    0xb8fbaf47u, 0xb97c1437u, 0xb9fcd245u, 0xba7de9afu, 0xbaff5ab2u, 0xbb81258du, 0xbc034a7fu, 0xbc85c9c5u,
    0xbd08a39fu, 0xbd8bd84cu, 0xbe0f680au, 0xbe935318u, 0xbf1799b6u, 0xbf9c3c25u, 0xc0213aa2u, 0xc0a6956fu,
    0xc12c4ccau, 0xc1b260f6u, 0xc238d231u, 0xc2bfa0bdu, 0xc346ccdau, 0xc3ce56cau, 0xc4563eccu, 0xc4de8524u,
    0xc5672a11u, 0xc5f02dd7u, 0xc67990b6u, 0xc70352f0u, 0xc78d74c9u, 0xc817f681u, 0xc8a2d85du, 0xc92e1a9du,
    0xc9b9bd86u, 0xca45c15bu, 0xcad2265eu, 0xcb5eecd4u, 0xcbec14ffu, 0xcc799f24u, 0xcd078b86u, 0xcd95da6bu,
    0xce248c15u, 0xceb3a0cau, 0xcf4318cfu, 0xcfd2f468u, 0xd06333dbu, 0xd0f3d76cu, 0xd184df62u, 0xd2164c02u,
    0xd2a81d92u, 0xd33a5458u, 0xd3ccf09au, 0xd45ff29eu, 0xd4f35aacu, 0xd587290au, 0xd61b5dffu, 0xd6aff9d2u,
    0xd744fccbu, 0xd7da6731u, 0xd870394cu, 0xd9067365u, 0xd99d15c2u, 0xda3420aeu, 0xdacb946fu, 0xdb637150u,
    0xdbfbb798u, 0xdc946791u, 0xdd2d8185u, 0xddc705bdu, 0xde60f482u, 0xdefb4e20u, 0xdf9612dfu, 0xe031430au,
    0xe0ccdeecu, 0xe168e6d0u, 0xe2055b00u, 0xe2a23bc8u, 0xe33f8973u, 0xe3dd444cu, 0xe47b6ca0u, 0xe51a02bbu,
    0xe5b906e7u, 0xe6587973u, 0xe6f85aabu, 0xe798aadbu, 0xe8396a50u, 0xe8da9958u, 0xe97c3840u, 0xea1e4756u,
    0xeac0c6e8u, 0xeb63b743u, 0xec0718b6u, 0xecaaeb90u, 0xed4f301fu, 0xedf3e6b2u, 0xee990f98u, 0xef3eab21u,
    0xefe4b99cu, 0xf08b3b59u, 0xf13230a8u, 0xf1d999d9u, 0xf281773cu, 0xf329c923u, 0xf3d28fdeu, 0xf47bcbbeu,
    0xf5257d15u, 0xf5cfa434u, 0xf67a416cu, 0xf7255511u, 0xf7d0df73u, 0xf87ce0e6u, 0xf92959bbu, 0xf9d64a47u,
    0xfa83b2dbu, 0xfb3193ccu, 0xfbdfed6du, 0xfc8ec011u, 0xfd3e0c0du, 0xfdedd1b5u, 0xfe9e115cu, 0xff4ecb59u,};

// Two floats in one register pair.
__device__ __forceinline__ uint64_t two(float a, float b) {
    uint64_t r;
    asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(a), "f"(b));
    return r;
}
__device__ __forceinline__ float low2(uint64_t x) { return __uint_as_float(uint32_t(x)); }
__device__ __forceinline__ float high2(uint64_t x) { return __uint_as_float(uint32_t(x >> 32)); }
__device__ __forceinline__ uint64_t mul2(uint64_t a, uint64_t b) {
    uint64_t r;
    asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
    return r;
}
__device__ __forceinline__ uint64_t add2(uint64_t a, uint64_t b) {
    uint64_t r;
    asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
    return r;
}
__device__ __forceinline__ uint64_t fma2(uint64_t a, uint64_t b, uint64_t c) {
    uint64_t r;
    asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
    return r;
}

struct Weigher {
    float hm;          // m / 2
    float ch, cl;      // 2 log2(e) / T as a sum of two floats
    float m;
    const uint32_t* tab;  // EXP2_256 in shared memory
    __device__ __forceinline__ Weigher(float m_, float T, const uint32_t* t) : m(m_), tab(t) {
        hm = 0.5f * m_;
        // 2 log2(e) / T: the quotient, then the quotient of its remainder
        constexpr float K = 2.885390043258667f, KL = 3.8519254e-8f;
        ch = __fdiv_rn(K, T);
        cl = ch > 0.f ? __fdiv_rn(__fadd_rn(fmaf(-ch, T, K), KL), T) : 0.f;
    }
    // 2^42 exp((z - m) / T), z <= m, rounded; 0 below 2^-43.  The exponent (z - m) log2(e) / T as a sum of two
    // floats (halved operands, so that the difference cannot overflow; its rounding error
    // by the two-sum); split into n + j / 256 + r, |r| <= 1/512; 2^r - 1 as a cubic in float32 (below
    // 2^-9, so its rounding is 2^-33 of the weight); the table's 2^(j / 256) times that in
    // integers.  About 40 instructions, 30 by twos; with a table of 32 and 2^r - 1 in two
    // floats it took 58 for a relative 4e-11.
    __device__ __forceinline__ unsigned long long weight_of(float z) const {
        int q;
        return weight_of(z, q);
    }
    // ... and the exponent in 1/256 of a binary order, rounded, negated: 0 for the maximum.
    __device__ __forceinline__ unsigned long long weight_of(float z, int& steps) const {
        const float h = 0.5f * z;
        const float d = __fsub_rn(h, hm), bb = __fsub_rn(d, h);
        const float dl = __fadd_rn(__fsub_rn(h, __fsub_rn(d, bb)), __fsub_rn(-hm, bb));
        const float yh = __fmul_rn(d, ch);
        float yl = fmaf(d, ch, -yh);
        yl = fmaf(d, cl, yl);
        yl = fmaf(dl, ch, yl);
        const float t = fmaf(yh, 256.f, 12582912.f);  // + 1.5 * 2^23: the nearest integer in the low bits
        const float r = __fadd_rn(fmaf(__fsub_rn(t, 12582912.f), -0.00390625f, yh), yl);
        // (2^r - 1) 2^33
        const float s = __fmul_rn(r, fmaf(r, fmaf(r, 0.05550410866482158f * 0x1p33f, 0.2402265069591007f * 0x1p33f),
                                          0.6931471805599453f * 0x1p33f));
        return assemble(yh, t, s, steps);
    }
    // The same of two, by instructions on two floats: the same operations, the same results.
    __device__ __forceinline__ void weights_of(float z0, float z1, unsigned long long (&w)[2], int (&steps)[2]) const {
        const uint64_t one = two(-1.f, -1.f), h = mul2(two(z0, z1), two(0.5f, 0.5f)), nhm = two(-hm, -hm), c = two(ch, ch),
                       nc = two(-ch, -ch);
        const uint64_t d = add2(h, nhm), bb = fma2(h, one, d);
        const uint64_t dl = add2(fma2(fma2(bb, one, d), one, h), fma2(bb, one, nhm));
        const uint64_t yh = mul2(d, c);
        // the low part of the exponent, negated
        const uint64_t yl = fma2(dl, nc, fma2(d, two(-cl, -cl), fma2(d, nc, yh)));
        const uint64_t magic = two(12582912.f, 12582912.f), t = fma2(yh, two(256.f, 256.f), magic);
        const uint64_t r0 = fma2(add2(t, two(-12582912.f, -12582912.f)), two(-0.00390625f, -0.00390625f), yh);
        const uint64_t r = fma2(yl, one, r0);
        constexpr float C3 = 0.05550410866482158f * 0x1p33f, C2 = 0.2402265069591007f * 0x1p33f, C1 = 0.6931471805599453f * 0x1p33f;
        const uint64_t s = mul2(r, fma2(r, fma2(r, two(C3, C3), two(C2, C2)), two(C1, C1)));
        w[0] = assemble(low2(yh), low2(t), low2(s), steps[0]);
        w[1] = assemble(high2(yh), high2(t), high2(s), steps[1]);
    }
    // From the exponent yh, its steps t and 2^r - 1 (times 2^33): 2^42 of the weight, rounded.
    __device__ __forceinline__ unsigned long long assemble(float yh, float t, float s, int& steps) const {
        steps = LAST;
        if (!(yh > -43.f)) return 0;  // also -inf, whose product with a zero slope is NaN
        const uint32_t bits = __float_as_uint(t), tj = tab[bits & 255];
        const long long p = (long long)int(tj >> 1) * __float2int_rn(s) + (1ll << 31);
        const uint32_t v = tj + uint32_t(p >> 32);                // 2^31 times the significand
        const uint32_t n = (0x4B400000u >> 8) - (bits >> 8);       // its binary orders below the maximum
        steps = int(0x4B400000u - bits);
        // v 2^(11 - n): the product's low words while that is whole, else its high word (the factor is
        // 2^32 larger), rounded.
        const bool whole = n <= 11;
        const unsigned long long x = (unsigned long long)v * (1u << ((11 - n) & 31)) + (whole ? 0u : 0x80000000u);
        return whole ? x : x >> 32;
    }
    // Bin of z, 0 the largest: 8 of those steps (0.022 T).  Each operation is monotone in z, so a lower
    // bin means larger z; the last bin's weights round to 0, or to one unit (2^-42) just above its edge.
    static constexpr int STEPS = 8, LAST = 43 * 256;
    __device__ __forceinline__ int bin_of(float z) const {
        const float yh = __fmul_rn(__fsub_rn(0.5f * z, hm), ch);
        if (!(yh > -43.f)) return LAST / STEPS;
        return (0x4B400000 - __float_as_int(fmaf(yh, 256.f, 12582912.f))) / STEPS;
    }
    // m - z at the lower edge of bin q, at least.
    __device__ __forceinline__ float drop_of(int q) const { return float(q + 1) * float(2 * STEPS / 256.0) / ch; }
};

// f * x for a float f in (0, 1): the floor, and whether a fraction was cut off.
__device__ __forceinline__ unsigned long long mul_frac(float f, unsigned long long x, bool& cut) {
    const uint32_t b = __float_as_uint(f);
    const int ex = int(b >> 23);
    const unsigned long long mt = (b & 0x7fffffu) | (ex ? 0x800000u : 0u);
    const int s = 150 - (ex ? ex : 1);  // f = mt * 2^-s, s >= 24
    const unsigned long long lo = mt * x, hi = __umul64hi(mt, x);
    if (s < 64) {
        cut = (lo << (64 - s)) != 0;
        return (lo >> s) | (hi << (64 - s));
    }
    if (s < 128) {
        const int t = s - 64;
        cut = lo != 0 || (t > 0 && (hi << (64 - t)) != 0);
        return hi >> t;
    }
    cut = (lo | hi) != 0;
    return 0;
}

// ------------------------------------------------------------------ block and cluster steps

// Words every CTA holds; other CTAs of the cluster write `flag`, `cmass` and the totals.
struct UCtl {
    uint32_t tab[256];
    unsigned long long red[UNW];
    uint32_t redc[UNW];
    unsigned long long cmass[MAX_CLUSTER], cin[MAX_CLUSTER];
    unsigned long long above, in_mass;  // find_bin's results
    uint32_t above_cnt, in_cnt;
    int bin;
    int n;               // entries of the list
    int nlive;
    int flag, flag2;
    int cn[MAX_CLUSTER]; // every CTA's entries
    alignas(16) int wcnt[64];
    int seg;
    unsigned long long rest;
};

struct USmem {
    static constexpr size_t CTL = 0;
    static constexpr size_t LKEY = align16(sizeof(UCtl));        // this CTA's list: keys, places, weights
    static constexpr size_t LPOS = LKEY + UCAP * 4;
    static constexpr size_t LW = LPOS + UCAP * 4;
    static constexpr size_t AKEY = LW + UCAP * 8;                // the cluster's list: keys, weights
    static constexpr size_t AW = AKEY + UCAP * 4;
    static constexpr size_t HIST = AW + UCAP * 8;                // masses, counts, their totals; later the segments' masses
    static constexpr size_t HIST_BYTES = size_t(UB) * 24;
    static __host__ __device__ size_t seg_at(int nsc) { return HIST + (size_t(nsc) * 8 > HIST_BYTES ? align16(size_t(nsc) * 8) : HIST_BYTES); }
    static __host__ __device__ size_t total(int nsc, int ls) { return seg_at(nsc) + align16(size_t(ls) * 4); }
};

template <typename X>
__device__ __forceinline__ X* peer(X* p, int rank) {
    return static_cast<X*>(__cluster_map_shared_rank(p, unsigned(rank)));
}

// The cluster's barrier; a CTA's alone where the cluster is one.
__device__ __forceinline__ void sync(int C) {
    if (C == 1) __syncthreads();
    else cluster_sync();
}

// Sum over the warp of masses below 2^48 each, in every lane: three words whose sums fit in 32 bits.
__device__ __forceinline__ unsigned long long warp_mass(unsigned long long v) {
    const uint32_t a = __reduce_add_sync(FULL, uint32_t(v) & 0xffffffu), b = __reduce_add_sync(FULL, uint32_t(v >> 24) & 0xffffffu);
    return (unsigned long long)b * (1u << 24) + a;
}

// Block-wide sum of a 64-bit value, in every thread.
__device__ __forceinline__ unsigned long long block_sum(unsigned long long v, UCtl* c) {
    v = warp_sum_u64(v);
    __syncthreads();
    if ((threadIdx.x & 31) == 0) c->red[threadIdx.x >> 5] = v;
    __syncthreads();
    unsigned long long s = 0;
#pragma unroll
    for (int w = 0; w < UNW; ++w) s += c->red[w];
    return s;
}

// Block-wide exclusive prefix of (mass, count) over the threads.
__device__ __forceinline__ void block_prefix(unsigned long long& v, uint32_t& n, UCtl* c) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const unsigned long long iv = warp_incl_scan_u64(v, lane);
    const uint32_t in = warp_incl_scan_t(n, lane);
    __syncthreads();
    if (lane == 31) c->red[warp] = iv, c->redc[warp] = in;
    __syncthreads();
    unsigned long long b = 0;
    uint32_t bn = 0;
    for (int w = 0; w < warp; ++w) b += c->red[w], bn += c->redc[w];
    v = iv - v + b;
    n = in - n + bn;
}

// The same of a count alone, and of a mass alone with the total returned.
__device__ __forceinline__ uint32_t block_prefix_count(uint32_t n, UCtl* c) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const uint32_t in = warp_incl_scan_t(n, lane);
    __syncthreads();
    if (lane == 31) c->redc[warp] = in;
    __syncthreads();
    const uint32_t w = c->redc[lane & (UNW - 1)];
    return in - n + warp_sum_i(lane < warp ? int(w) : 0);
}
__device__ __forceinline__ unsigned long long block_prefix_mass(unsigned long long& v, UCtl* c) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const unsigned long long iv = warp_incl_scan_u64(v, lane);
    __syncthreads();
    if (lane == 31) c->red[warp] = iv;
    __syncthreads();
    unsigned long long b = 0, all = 0;
#pragma unroll
    for (int w = 0; w < UNW; ++w) {
        const unsigned long long x = c->red[w];
        if (w < warp) b += x;
        all += x;
    }
    v = iv - v + b;
    return all;
}

// The first bin at which the running count reaches k >= 1 (UB: never), in c->bin.  Block-wide.
__device__ __forceinline__ void find_count(const uint32_t* cnt, uint32_t k, UCtl* c) {
    constexpr int PER = UB / UNT;
    const int b0 = threadIdx.x * PER;
    uint32_t x[PER], n = 0;
#pragma unroll
    for (int i = 0; i < PER; ++i) n += x[i] = cnt[b0 + i];
    if (threadIdx.x == 0) c->bin = UB;
    uint32_t before = block_prefix_count(n, c);
    if (before < k && before + n >= k) {
#pragma unroll
        for (int i = 0; i < PER; ++i) {
            if (before < k && before + x[i] >= k) c->bin = b0 + i;
            before += x[i];
        }
    }
    __syncthreads();
}

// The first bin at which the running mass (by_mass) or count reaches target >= 1; the sums before it
// and in it go into the control words (bin UB when it is never reached).  Block-wide.
template <typename X>
__device__ __forceinline__ void find_bin(const X mass, const uint32_t* cnt, bool by_mass,
                                         unsigned long long target, UCtl* c) {
    constexpr int PER = UB / UNT;
    const int b0 = threadIdx.x * PER;
    unsigned long long v = 0;
    uint32_t n = 0;
#pragma unroll
    for (int i = 0; i < PER; ++i) {
        v += mass[b0 + i];
        n += cnt[b0 + i];
    }
    const unsigned long long own = by_mass ? v : n;
    block_prefix(v, n, c);
    if (threadIdx.x == 0) c->bin = UB;
    __syncthreads();
    const unsigned long long before = by_mass ? v : n;
    if (before < target && before + own >= target) {
        for (int i = 0; i < PER; ++i) {
            const unsigned long long mi = mass[b0 + i];
            const uint32_t ni = cnt[b0 + i];
            if ((by_mass ? v + mi : n + ni) >= target) {
                c->bin = b0 + i;
                c->above = v, c->above_cnt = n, c->in_mass = mi, c->in_cnt = ni;
                break;
            }
            v += mi, n += ni;
        }
    }
    __syncthreads();
}

// Masses of the bins: low words, then high words (each over all 32 banks).
struct Hist {
    uint32_t* lo;
    __device__ __forceinline__ unsigned long long operator[](int i) const { return (unsigned long long)lo[UB + i] << 32 | lo[i]; }
    __device__ __forceinline__ void set(int i, unsigned long long v) const { lo[i] = uint32_t(v), lo[UB + i] = uint32_t(v >> 32); }
    __device__ __forceinline__ void add(int i, unsigned long long v) const {
        const uint32_t w = uint32_t(v), old = atomicAdd(lo + i, w);
        const uint32_t h = uint32_t(v >> 32) + (old + w < old ? 1u : 0u);
        if (h) atomicAdd(lo + UB + i, h);
    }
    __device__ __forceinline__ Hist of(int rank) const { return Hist{peer(lo, rank)}; }
};

// A 64-bit add into a shared counter by 32-bit atomics: the low word's carry goes on.
__device__ __forceinline__ void add64(unsigned long long* p, unsigned long long v) {
    uint32_t* w = reinterpret_cast<uint32_t*>(p);
    const uint32_t lo = uint32_t(v), old = atomicAdd(w, lo);
    const uint32_t hi = uint32_t(v >> 32) + (old + lo < old ? 1u : 0u);
    if (hi) atomicAdd(w + 1, hi);
}

// The bin that the row's mass reaches `target` in, from exact masses.  Cluster-wide; over the histograms' memory.
// (Not inlined: hardly any row calls it.)
template <typename T>
__device__ __noinline__ int exact_bin(const URow<T> row, const Weigher wt, const Hist hist, const uint32_t* cnt, const uint32_t* segs,
                                      int s0, int s1, unsigned long long target, UCtl* c) {
    const int tid = threadIdx.x, lane = tid & 31, C = int(cluster_nctarank()), rank = int(cluster_ctarank());
    __syncthreads();
    for (int i = tid; i < UB; i += UNT) hist.set(i, 0);
    __syncthreads();
    for (int s = s0 + (tid >> 5); s < s1; s += UNW) {
        if (segs[s] <= KEY_NINF) continue;
        const uint4 v = row.load(s, lane);
#pragma unroll 1
        for (int e = 0; e < URow<T>::N; ++e) {
            int q;
            const unsigned long long w = wt.weight_of(element(v, e, T()), q);
            if (w) hist.add(q / Weigher::STEPS, w);
        }
    }
    // Every CTA sums its share of the bins over the cluster, then hands it to all.
    sync(C);
    const int n = UB / C;
    unsigned long long v[UB / UNT];
#pragma unroll
    for (int i = 0; i < UB / UNT; ++i) {
        v[i] = 0;
        if (tid + i * UNT < n)
            for (int q = 0; q < C; ++q) v[i] += hist.of(q)[rank * n + tid + i * UNT];
    }
    sync(C);
#pragma unroll
    for (int i = 0; i < UB / UNT; ++i)
        if (tid + i * UNT < n)
            for (int q = 0; q < C; ++q) hist.of(q).set(rank * n + tid + i * UNT, v[i]);
    sync(C);
    find_bin(hist, cnt, true, target, c);
    return c->bin;
}

template <typename T>
__global__ void __launch_bounds__(UNT, 2) uniform_kernel(const UniformArgs a) {
    using R = URow<T>;
    extern __shared__ __align__(16) unsigned char smem[];
    UCtl* c = reinterpret_cast<UCtl*>(smem + USmem::CTL);
    uint32_t* lkey = reinterpret_cast<uint32_t*>(smem + USmem::LKEY);
    int* lpos = reinterpret_cast<int*>(smem + USmem::LPOS);
    unsigned long long* lw = reinterpret_cast<unsigned long long*>(smem + USmem::LW);
    uint32_t* akey = reinterpret_cast<uint32_t*>(smem + USmem::AKEY);
    unsigned long long* aw = reinterpret_cast<unsigned long long*>(smem + USmem::AW);
    const Hist hist{reinterpret_cast<uint32_t*>(smem + USmem::HIST)};
    unsigned long long* smass = reinterpret_cast<unsigned long long*>(smem + USmem::HIST);  // [nsc], after the histograms
    uint32_t* tmass = reinterpret_cast<uint32_t*>(smass + UB);   // the cluster's masses, rounded, and counts
    uint32_t* hcnt = tmass + 2 * UB;
    uint32_t* tcnt = hcnt + UB;
    uint32_t* segs = reinterpret_cast<uint32_t*>(smem + USmem::seg_at(a.nsc));
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int C = int(cluster_nctarank()), rank = int(cluster_ctarank()), b = int(cluster_id_x());
    // The parameters were written before the scan began (it waits for its predecessors before
    // it lets this launch start), so they are read while it runs.
    const int r = a.indices ? a.indices[b] : b;
    const float u = a.u[b];
    const float temp = a.temperature ? a.temperature[b] : 1.f;
    const int k = a.top_k ? a.top_k[b] : 0;
    const float p = a.top_p ? a.top_p[b] : 1.f;
    const float mp = a.min_p ? a.min_p[b] : 0.f;
    if (tid < 256) c->tab[tid] = EXP2_256[tid];
    if (tid == 0) c->n = 0, c->nlive = 0, c->flag = 0, c->flag2 = 0;
    for (int i = tid; i < UB; i += UNT) hcnt[i] = 0;
    sync(C);  // every CTA of the cluster runs before another writes into its memory
    grid_dependency_wait();
    allow_dependents();

    // ---- the row's maximum
    bool bad = r < 0 || r >= a.batch_in || !(u >= 0.f && u < 1.f) || !(temp >= 1.17549435e-38f) || !(p == p) || !(mp <= 1.f);
    uint32_t kmax = 0;
    if (!bad) {
        const R row(a.x, a.stride, r, a.V);
#pragma unroll 4
        for (int s = tid; s < row.nseg; s += UNT) {
            const uint32_t sk = a.skey[int64_t(r) * a.ls + s];
            segs[s] = sk;
            kmax = max(kmax, sk);
        }
        kmax = warp_max_u(kmax);
        if (lane == 0) c->redc[warp] = kmax;
        __syncthreads();
        kmax = warp_max_u(c->redc[lane & (UNW - 1)]);
        bad = kmax >= KEY_PINF || kmax <= KEY_NINF;
    }
    if (bad) {  // the same in every thread of the cluster
        if (rank == 0 && tid == 0) a.out_token[b] = -1, a.out_valid[b] = 0;
        return;
    }
    const R row(a.x, a.stride, r, a.V);
    const Weigher wt(from_logit_key(kmax), temp, c->tab);
    const unsigned long long ONE = 1ull << 42;
    constexpr int LASTB = Weigher::LAST / Weigher::STEPS;
    const bool has_k = k > 0 && k < a.V, has_p = p < 1.f;
    const bool joint = a.order == FS_ORDER_JOINT || !has_k;  // top-p is measured against the whole row
    // min-p: w >= mp * max w; the integers are compared, rounded up.  floor_key: no element below it
    // passes (ln and the product within 2^-18 of their size).
    unsigned long long wmin = 1;
    uint32_t floor_key = KEY_NINF + 1;
    if (mp > 0.f) {
        bool cut = false;
        wmin = mp < 1.f ? mul_frac(mp, ONE, cut) : ONE;
        wmin = max(1ull, wmin + (cut ? 1 : 0));
        const float drop = temp * logf(mp);
        const float zf = wt.m + drop - 0x1p-18f * (fabsf(wt.m) + fabsf(drop));
        if (zf >= -3.402823466e38f) floor_key = max(floor_key, ukey(zf));
    }
    // This CTA's segments.
    const int per = (row.nseg + C - 1) / C;
    const int s0 = min(row.nseg, rank * per), s1 = min(row.nseg, s0 + per);
    // fn(z) over the elements of this CTA's segments whose maximum passes.
    auto each = [&](auto pass, auto fn) {
        for (int s = s0 + warp; s < s1; s += UNW * 2) {
            const bool one = pass(segs[s]), two = s + UNW < s1 && pass(segs[s + UNW]);
            uint4 v0, v1;
            if (one) v0 = row.load(s, lane);
            if (two) v1 = row.load(s + UNW, lane);
            float z[R::N];
            if (one) {
                unpack(v0, z, T());
#pragma unroll
                for (int e = 0; e < R::N; ++e) fn(z[e], s, e);
            }
            if (two) {
                unpack(v1, z, T());
#pragma unroll
                for (int e = 0; e < R::N; ++e) fn(z[e], s + UNW, e);
            }
        }
    };
    auto all = [](uint32_t) { return true; };
    // fn(z0, z1) over neighbouring elements of all of them.
    auto pairs = [&](auto fn) {
        for (int s = s0 + warp; s < s1; s += UNW * 2) {
            const bool more = s + UNW < s1;
            const uint4 v0 = row.load(s, lane);
            uint4 v1 = v0;
            if (more) v1 = row.load(s + UNW, lane);
            float z[R::N];
            unpack(v0, z, T());
#pragma unroll
            for (int e = 0; e < R::N; e += 2) fn(z[e], z[e + 1]);
            if (more) {
                unpack(v1, z, T());
#pragma unroll
                for (int e = 0; e < R::N; e += 2) fn(z[e], z[e + 1]);
            }
        }
    };
    // The row's mass from exact weights.  Cluster-wide.
    auto exact_mass = [&]() {
        unsigned long long v = 0, M = 0;
        pairs([&](float z0, float z1) {
            unsigned long long w[2];
            int q[2];
            wt.weights_of(z0, z1, w, q);
            v += w[0] + w[1];
        });
        v = block_sum(v, c);
        if (tid < C) peer(c->cmass, tid)[rank] = v;
        sync(C);
        for (int q = 0; q < C; ++q) M += c->cmass[q];
        return M;
    };

    // ---- small sets: everything in a list
    bool small = false;
    const bool try_k = has_k && k <= UCAP;
    if (try_k || (mp > 0.f && !(has_p && !joint))) {
        // zt: a bound that every element the decisions need reaches.  The bin of the k-th largest
        // segment maximum, its lower edge less the edge's rounding.
        float zt = -INFINITY;
        small = true;
        if (try_k) {
            for (int s = tid; s < row.nseg; s += UNT) atomicAdd(&hcnt[wt.bin_of(from_logit_key(segs[s]))], 1u);
            __syncthreads();
            find_count(hcnt, uint32_t(k), c);
            const int kb = c->bin;  // the last bin has next to no weight, and UB means fewer segments than k
            const float drop = wt.drop_of(kb);
            if (kb < LASTB) zt = wt.m - drop - 0x1p-18f * (fabsf(wt.m) + drop);
            small = kb < LASTB;
        }
        // (top-p inside the top k is measured against all of the top k, min-p or not)
        if (mp > 0.f && !(has_p && !joint)) {
            zt = fmaxf(zt, from_logit_key(floor_key));
            small = true;
        }
        if (small) {
            if (rank == 0) {
                // The live segments in order, then 64 of them at a time, four per warp: their elements at
                // or above zt, counted, placed by a prefix over the segments, written in index order.
                int* live = reinterpret_cast<int*>(hist.lo);
                const uint32_t kt = ukey(zt), zb = bound_of(zt, T());
                const int chunk = (row.nseg + UNT - 1) / UNT;
                const int f0 = min(row.nseg, tid * chunk), f1 = min(row.nseg, f0 + chunk);
                uint32_t nl = 0;
                for (int s = f0; s < f1; ++s) nl += segs[s] >= kt;
                uint32_t at = block_prefix_count(nl, c);
                if (tid == UNT - 1) c->nlive = int(at + nl);
                for (int s = f0; s < f1 && nl; ++s)
                    if (segs[s] >= kt) {
                        if (at < UCAP) live[at] = s;
                        ++at;
                    }
                __syncthreads();
                // each live segment holds a candidate, so more of them than UCAP are too many
                const int n_live = min(c->nlive, UCAP);
                int base = 0;
                for (int i0 = 0; i0 < n_live; i0 += 64) {
                    uint4 v[4];
                    uint32_t hit = 0, cnt[2] = {0, 0};   // four segments' hits; their counts, two to a word
#pragma unroll
                    for (int j = 0; j < 4; ++j)
                        if (i0 + warp * 4 + j < n_live) v[j] = row.load(live[i0 + warp * 4 + j], lane);
#pragma unroll
                    for (int j = 0; j < 4; ++j) {
                        if (i0 + warp * 4 + j < n_live) {
                            const uint32_t h = hits(v[j], zb, T());
                            hit |= h << (8 * j);
                            cnt[j >> 1] += __popc(h) << (16 * (j & 1));
                        }
                    }
                    const uint32_t in0 = warp_incl_scan_t(cnt[0], lane), in1 = warp_incl_scan_t(cnt[1], lane);
                    if (lane == 31) *reinterpret_cast<uint4*>(c->wcnt + warp * 4) =
                        make_uint4(in0 & 0xffff, in0 >> 16, in1 & 0xffff, in1 >> 16);
                    __syncthreads();
                    const int c0 = c->wcnt[lane * 2], c1 = c->wcnt[lane * 2 + 1];
                    const int incl = warp_incl_scan_i(c0 + c1, lane);
                    const int total = __shfl_sync(FULL, incl, 31);
                    // where the lane's elements of each segment go
                    const int b0 = base + __shfl_sync(FULL, incl - c0 - c1, warp * 2), b2 = base + __shfl_sync(FULL, incl - c0 - c1, warp * 2 + 1);
                    const int w0 = b0 + int((in0 - cnt[0]) & 0xffff), w1 = b0 + __shfl_sync(FULL, c0, warp * 2) + int((in0 - cnt[0]) >> 16);
                    const int w2 = b2 + int((in1 - cnt[1]) & 0xffff), w3 = b2 + __shfl_sync(FULL, c0, warp * 2 + 1) + int((in1 - cnt[1]) >> 16);
                    for (uint32_t left = hit; left; left &= left - 1) {
                        const int bit = __ffs(left) - 1, j = bit >> 3, e = bit & 7;
                        const int w = (j < 2 ? (j == 0 ? w0 : w1) : (j == 2 ? w2 : w3)) + __popc(hit >> (8 * j) & ((1u << e) - 1));
                        if (w < UCAP) {
                            const uint4 x = j < 2 ? (j == 0 ? v[0] : v[1]) : (j == 2 ? v[2] : v[3]);
                            lkey[w] = ukey(element(x, e, T()));
                            lpos[w] = live[i0 + warp * 4 + j] * R::SEG + lane * R::N + e;
                        }
                    }
                    base += total;
                    __syncthreads();
                }
                if (tid == 0) c->n = base;
                if (tid < C) *peer(&c->flag, tid) = c->nlive <= UCAP && base <= UCAP ? 1 : 0;
            }
            sync(C);
            small = c->flag != 0;
        }
    }
    if (small) {
        const bool whole = has_p && joint;   // M is needed
        float Mf = 0.f;
        unsigned long long M = 0;
        if (whole) {
            // float32, relative to the maximum.  Each exponent y is off by 4 2^-24 |y|, and most of
            // a row's mass lies above y = -log2(V) >= -21: 2^-18 of the mass; 2^y by 2^-22; at most 40 additions
            // in a row (a double takes the long runs): under 2^-17 together.
            double run = 0.0;
            const float cc = 1.44269504f / temp;
            if (a.ssum) {
                for (int s = tid; s < row.nseg; s += UNT) {
                    const float z = from_logit_key(segs[s]);
                    if (z > -INFINITY) run += double(a.ssum[int64_t(r) * a.ls + s] * exp2_approx((z - wt.m) * cc));
                }
            } else {
                float part = 0.f;
                each(all, [&](float z, int, int e) {
                    part += exp2_approx((z - wt.m) * cc);
                    if (e == R::N - 1) run += double(part), part = 0.f;
                });
            }
            float v = warp_sum(float(run));
            if (lane == 0) c->redc[warp] = __float_as_uint(v);
            __syncthreads();
            v = warp_sum(lane < UNW ? __uint_as_float(c->redc[lane]) : 0.f);
            if (!a.ssum) {
                if (tid < C) peer(c->cmass, tid)[rank] = __float_as_uint(v);
                sync(C);
                for (int q = 0; q < C; ++q) Mf += __uint_as_float(uint32_t(c->cmass[q]));
            } else {
                Mf = v;
            }
        }
        int n = 0, tpc = 1, per_thread = 1;
        if (rank == 0) {
            n = c->n;
            for (int i = tid; i < n; i += UNT) lw[i] = wt.weight_of(from_logit_key(lkey[i]));
            __syncthreads();
            per_thread = n <= 128 ? 1 : 4;
            while (tpc < (n <= 128 ? 8 : 32) && tpc * 2 * ((n + per_thread - 1) / per_thread) <= UNT) tpc *= 2;
        }
        // Four candidates a thread (one, up to 128), `tpc` threads for the same ones, each over its
        // share of the list.
        constexpr int PER = 4;
        const int sub = tid % tpc, i0 = tid / tpc * per_thread;
        unsigned long long above[PER] = {0, 0, 0, 0}, wi[PER] = {0, 0, 0, 0};
        bool keep[PER] = {false, false, false, false};
        auto compare = [&](auto count) {
            constexpr int N = decltype(count)::value;
            uint32_t ki[N];
            int cnt[N];
#pragma unroll
            for (int x = 0; x < N; ++x) {
                const bool in = i0 + x < n;
                wi[x] = in ? lw[i0 + x] : 0;
                ki[x] = in ? lkey[i0 + x] : 0xffffffffu;
                keep[x] = in;
                cnt[x] = 0;
            }
            if (!has_k && !has_p) return;
#pragma unroll 2
            for (int j = sub; j < n; j += tpc) {
                const uint32_t kj = lkey[j];
                const unsigned long long wj = lw[j];
#pragma unroll
                for (int x = 0; x < N; ++x)
                    if (kj > ki[x]) ++cnt[x], above[x] += wj;
            }
            for (int d = 1; d < tpc; d *= 2) {
#pragma unroll
                for (int x = 0; x < N; ++x) {
                    cnt[x] += __shfl_xor_sync(FULL, cnt[x], d);
                    above[x] += __shfl_xor_sync(FULL, above[x], d);
                }
            }
#pragma unroll
            for (int x = 0; x < N; ++x)
                if (has_k) keep[x] = keep[x] && cnt[x] < k;  // ties with the k-th are kept
        };
        bool exact = !whole;
        for (int turn = 0; turn < 2; ++turn) {
            bool unsure = false;
            if (rank == 0 && turn == 0) {
                if (per_thread == 1) compare(std::integral_constant<int, 1>());
                else compare(std::integral_constant<int, PER>());
            }
            if (rank == 0 && has_p && !whole) {
                unsigned long long F = 0;
#pragma unroll
                for (int x = 0; x < PER; ++x) F += keep[x] && sub == 0 ? wi[x] : 0;
                M = block_sum(F, c);
            }
            if (rank == 0 && has_p) {
                bool cut = false;
                unsigned long long G = 0;
                float lo = 0.f, hi = 0.f;
                if (exact) {
                    G = p > 0.f ? mul_frac(p, M, cut) : 0;
                    G = max(1ull, G + (cut ? 1 : 0));
                } else {
                    const float t = p > 0.f ? p * Mf * 0x1p42f : 0.f;
                    lo = t * (1.f - 0x1p-16f), hi = t * (1.f + 0x1p-16f);
                    unsure = !(Mf > 0.f && Mf < INFINITY);
                }
#pragma unroll
                for (int x = 0; x < PER; ++x) {
                    if (exact) {
                        keep[x] = keep[x] && above[x] < G;
                    } else if (keep[x] && wi[x] >= wmin) {
                        const float f = float(above[x]);
                        if (p > 0.f) unsure |= f >= lo && f <= hi;
                        else keep[x] = above[x] == 0;
                        if (p > 0.f && f > hi) keep[x] = false;
                    }
                }
            }
            if (exact) break;
            // A candidate too close to call: the row's mass is summed exactly.
            if (rank == 0) {
                unsure = __syncthreads_or(unsure);
                if (tid < C) *peer(&c->flag2, tid) = unsure ? 1 : 0;
            }
            sync(C);
            if (!c->flag2) break;
            M = exact_mass();
            exact = true;
        }
        if (rank != 0) return;
        // ---- the draw: candidates are in index order
        // (the threads that share candidates sit beside one another: the first of them holds them)
        unsigned long long own[PER], v = 0;
#pragma unroll
        for (int x = 0; x < PER; ++x) {
            own[x] = sub == 0 && keep[x] && wi[x] >= wmin ? wi[x] : 0;
            v += own[x];
        }
        const unsigned long long mine = v;
        const unsigned long long Z = block_prefix_mass(v, c);
        if (Z == 0) {
            if (tid == 0) a.out_token[b] = -1, a.out_valid[b] = 0;
            return;
        }
        bool cut;
        const unsigned long long t = u > 0.f ? mul_frac(u, Z, cut) : 0;
        if (v <= t && t - v < mine) {
#pragma unroll
            for (int x = 0; x < PER; ++x) {
                if (v <= t && t - v < own[x]) a.out_token[b] = lpos[i0 + x] - row.a0, a.out_valid[b] = 1;
                v += own[x];
            }
        }
        return;
    }

    // ---- other sets: thresholds from histograms
    uint32_t theta = floor_key;
    bool summed = false;   // the segments' masses are there
    if (has_k || has_p) {
        // Masses go into the bins as 32-bit words, in units of 2^-shift of an integer weight: at
        // most SEG times the segment maxima's weights, the row fits. (Adds that return nothing are
        // nearly free; 64-bit sums, whose carry needs the old value, cost 10 us of 60.)  They only
        // choose the bin: the masses above it and in it are summed exactly afterwards.
        float ml = 0.f;
        for (int s = tid; s < row.nseg; s += UNT)
            if (segs[s] > KEY_NINF) ml += exp2_approx((from_logit_key(segs[s]) - wt.m) * (1.44269504f / temp));
        ml = warp_sum(ml);
        __syncthreads();
        if (lane == 0) c->redc[warp] = __float_as_uint(ml);
        for (int i = tid; i < UB; i += UNT) hist.lo[i] = 0, hcnt[i] = 0;
        __syncthreads();
        ml = warp_sum(lane < UNW ? __uint_as_float(c->redc[lane]) : 0.f);
        const int shift = 11 + int(__float_as_uint(ml * (1.01f * R::SEG)) >> 23) - 126;  // 2^31 and its rounding
        const unsigned long long half = 1ull << shift >> 1;
        unsigned long long F = 0;
        pairs([&](float z0, float z1) {
            unsigned long long w[2];
            int q[2];
            wt.weights_of(z0, z1, w, q);
            F += w[0] + w[1];
#pragma unroll
            for (int x = 0; x < 2; ++x) {
                const uint32_t bin = uint32_t(q[x]) / Weigher::STEPS;
                if (w[x]) atomicAdd(hist.lo + bin, uint32_t((w[x] + half) >> shift));
                if (has_k) atomicAdd(hcnt + bin, 1u);
            }
        });
        F = block_sum(F, c);
        // The cluster's histograms summed into every CTA's totals, and the row's mass.
        if (tid < C) peer(c->cmass, tid)[rank] = F;
        sync(C);
        F = 0;
        for (int q = 0; q < C; ++q) F += c->cmass[q];
        {
            const int n = UB / C;
            for (int i = rank * n + tid; i < (rank + 1) * n && i <= LASTB; i += UNT) {
                uint32_t v = 0, m = 0;
                for (int q = 0; q < C; ++q) {
                    v += *peer(hist.lo + i, q);
                    if (has_k) m += *peer(hcnt + i, q);
                }
                for (int q = 0; q < C; ++q) {
                    *peer(tmass + i, q) = v;
                    if (has_k) *peer(tcnt + i, q) = m;
                }
            }
            for (int i = LASTB + 1 + tid; i < UB; i += UNT) tmass[i] = 0, tcnt[i] = 0;
            if (!has_k)
                for (int i = tid; i <= LASTB; i += UNT) tcnt[i] = 0;
        }
        sync(C);
        // The largest key whose elements at or above it reach `target` (count or mass); the mass at
        // or above it goes into `fmass`.  With `last`, the masses of this CTA's segments are
        // left in smass, of elements at or above that key and `also`.
        auto search = [&](bool by_mass, unsigned long long target, unsigned long long& fmass, bool last,
                          uint32_t also) -> uint32_t {
            find_bin(static_cast<const uint32_t*>(tmass), tcnt, by_mass, by_mass ? max(1ull, target >> shift) : target, c);
            int qb = c->bin;
            unsigned long long above = 0, above_t = c->above_cnt;
            // Where rounding put the border into another bin, the exact mass above the bin that was listed tells how far
            // the rounded masses are off there, and they are asked again; then the bin beside is taken.  After
            // that, and where they fall short of the target in a tail of weights that round to nothing, exact masses
            // choose the bin: four lists at most.  (64 rows of 256000 at top-p 0.999: 0.28 ms.  Moving on by one bin
            // a turn took up to 733 lists and 51 ms, and at 0.95, where some rows miss twice, 67.6 us instead of 64.5.)
            bool lost = by_mass && qb > LASTB - 1;
            for (int turn = 0; turn < 5; ++turn) {
                if (lost) qb = exact_bin<T>(row, wt, hist, hcnt, segs, s0, s1, target, c), lost = false;
                if (qb >= LASTB) return 0;  // reached only among elements of no weight or one unit
                __syncthreads();
                if (tid == 0) c->n = 0;
                if (last)
                    for (int i = tid; i < s1 - s0; i += UNT) smass[i] = 0;
                __syncthreads();
                // The bin's elements into this CTA's list; the weights of those above it summed.  Few lanes
                // hold an element at or above the bin (zl: its lower edge less the edge's rounding), so
                // each lane walks its own.
                const float drop = wt.drop_of(qb);
                const float zl = wt.m - drop - 0x1p-18f * (fabsf(wt.m) + drop);
                const uint32_t kz = zl == zl ? ukey(zl) : 0u, zb = bound_of(zl, T());
                unsigned long long over = 0, inside = 0;   // mass above the bin, in it
                auto walk = [&](int s, const uint4& v) {
                    uint32_t hit = kz ? hits(v, zb, T()) : (1u << R::N) - 1;
                    unsigned long long sum = 0;
                    while (hit) {
                        const int e = __ffs(hit) - 1;
                        hit &= hit - 1;
                        const float x = element(v, e, T());
                        int q;
                        const unsigned long long w = wt.weight_of(x, q);
                        q /= Weigher::STEPS;
                        if (q < qb) {
                            over += w;
                            if (ukey(x) >= also && w >= wmin) sum += w;
                        } else if (q == qb) {
                            inside += w;
                            const int at = atomicAdd(&c->n, 1);
                            if (at < UCAP) lkey[at] = ukey(x), lpos[at] = s - s0, lw[at] = w;
                        }
                    }
                    if (last) {
                        sum = warp_mass(sum);
                        if (lane == 0) smass[s - s0] = sum;
                    }
                };
                for (int s = s0 + warp; s < s1; s += UNW * 2) {
                    const bool one = segs[s] >= kz, two = s + UNW < s1 && segs[s + UNW] >= kz;
                    uint4 v0, v1;
                    if (one) v0 = row.load(s, lane);
                    if (two) v1 = row.load(s + UNW, lane);
                    if (one) walk(s, v0);
                    if (two) walk(s + UNW, v1);
                }
                over = block_sum(over, c);
                inside = block_sum(inside, c);
                const int ln = c->n;
                if (tid < C) peer(c->cn, tid)[rank] = ln, peer(c->cmass, tid)[rank] = over, peer(c->cin, tid)[rank] = inside;
                sync(C);
                int n = 0;
                above = 0;
                inside = 0;
                for (int q = 0; q < C; ++q) n += c->cn[q], above += c->cmass[q], inside += c->cin[q];
                fmass = above + inside;
                if (by_mass && (above >= target || fmass < target)) {
                    const int beside = qb + (above >= target ? -1 : 1);
                    sync(C);
                    if (turn == 0 && a.nsc <= UB) {   // (the masses of more segments lie over the bins)
                        const long long asked = (long long)c->above + ((long long)(target - above) >> shift);
                        find_bin(static_cast<const uint32_t*>(tmass), tcnt, true, (unsigned long long)max(1ll, asked), c);
                        lost = c->bin > LASTB - 1;
                        qb = c->bin == qb ? beside : c->bin;
                    } else {
                        lost = turn > 1;
                        qb = beside;
                    }
                    continue;
                }
                if (by_mass) above_t = above;
                if (n > UCAP) break;
                // every CTA gathers the whole list and decides
                int at = 0;
                for (int q = 0; q < C; ++q) {
                    for (int i = tid; i < c->cn[q]; i += UNT) akey[at + i] = *peer(lkey + i, q), aw[at + i] = *peer(lw + i, q);
                    at += c->cn[q];
                }
                __syncthreads();
                int tpc = 1;
                while (tpc < 32 && tpc * 2 * n <= UNT) tpc *= 2;
                uint32_t least = 0xffffffffu;
                unsigned long long kept = 0;
                for (int i0 = 0; i0 < n; i0 += UNT / tpc) {
                    const int i = i0 + tid / tpc;
                    const uint32_t ki = i < n ? akey[i] : 0xffffffffu;
                    int cnt = 0;
                    unsigned long long m = 0;
#pragma unroll 4
                    for (int j = tid % tpc; j < n; j += tpc)
                        if (akey[j] > ki) ++cnt, m += aw[j];
                    for (int d = 1; d < tpc; d *= 2) {
                        cnt += __shfl_xor_sync(FULL, cnt, d);
                        m += __shfl_xor_sync(FULL, m, d);
                    }
                    if (i < n && (by_mass ? above_t + m : above_t + cnt) < target) {
                        least = min(least, ki);
                        if (tid % tpc == 0) kept += aw[i];
                    }
                }
                fmass = above + block_sum(kept, c);
                least = warp_min_u(least);
                __syncthreads();
                if (lane == 0) c->redc[warp] = least;
                __syncthreads();
                least = warp_min_u(c->redc[lane & (UNW - 1)]);
                if (last) {
                    for (int i = tid; i < ln; i += UNT)
                        if (lkey[i] >= max(least, also) && lw[i] >= wmin) add64(smass + lpos[i], lw[i]);
                    summed = true;
                    __syncthreads();
                }
                sync(C);  // the lists have been read: they may be used again
                return least;
            }
            const float drop = wt.drop_of(qb);
            // Keys the bin can hold, with some slack for the rounding of its edges.
            const float lo = wt.m - drop, hi = qb > 0 ? wt.m - wt.drop_of(qb - 1) * (1.f - 1.f / 16.f / float(qb)) : wt.m;
            const float sl = 0x1p-18f * (fabsf(wt.m) + drop);
            uint32_t kl = max(KEY_NINF + 1, ukey(lo - sl == lo - sl ? fmaxf(lo - sl, -3.402823466e38f) : -3.402823466e38f));
            uint32_t kh = min(kmax, ukey(hi + sl == hi + sl ? fminf(hi + sl, 3.402823466e38f) : 3.402823466e38f));
            while (kh > kl) {
                const int bits = 32 - __clz(kh - kl);
                const int sh = bits > 11 ? bits - 11 : 0;
                __syncthreads();
                for (int i = tid; i < UB; i += UNT) hist.set(i, 0), hcnt[i] = 0;
                __syncthreads();
                each([&](uint32_t key) { return key >= kl; }, [&](float z, int, int) {
                    const uint32_t key = ukey(z);
                    if (key >= kl && key <= kh && wt.bin_of(z) == qb) {
                        const int q = int((kh - key) >> sh);
                        hist.add(q, wt.weight_of(z));
                        atomicAdd(hcnt + q, 1u);
                    }
                });
                // Every CTA sums its share of the bins over the cluster, then hands it to all.
                sync(C);
                const int n = UB / C;
                unsigned long long v[UB / UNT];
                uint32_t m[UB / UNT];
#pragma unroll
                for (int i = 0; i < UB / UNT; ++i) {
                    const int at = rank * n + tid + i * UNT;
                    v[i] = 0, m[i] = 0;
                    if (tid + i * UNT < n)
                        for (int q = 0; q < C; ++q) v[i] += hist.of(q)[at], m[i] += *peer(hcnt + at, q);
                }
                sync(C);
#pragma unroll
                for (int i = 0; i < UB / UNT; ++i) {
                    const int at = rank * n + tid + i * UNT;
                    if (tid + i * UNT < n)
                        for (int q = 0; q < C; ++q) hist.of(q).set(at, v[i]), *peer(hcnt + at, q) = m[i];
                }
                sync(C);
                find_bin(hist, hcnt, by_mass, target - above_t, c);
                const uint32_t q = uint32_t(c->bin);
                above += c->above;
                above_t += by_mass ? c->above : c->above_cnt;
                const uint32_t top = kh - (q << sh);
                kl = max(kl, sh ? (top - kl >= (1u << sh) ? top - (1u << sh) + 1 : kl) : top);
                kh = top;
                fmass = above + c->in_mass;
            }
            return kl;
        };
        unsigned long long none = 0;
        if (has_k) {
            unsigned long long fk = F;
            theta = max(theta, search(false, (unsigned long long)k, fk, !has_p, floor_key));
            if (!joint) F = fk;
        }
        if (has_p) {
            bool cut = false;
            unsigned long long G = p > 0.f ? mul_frac(p, F, cut) : 0;
            G = max(1ull, G + (cut ? 1 : 0));
            theta = max(theta, search(true, G, none, true, theta));
        }
        sync(C);  // every CTA has read the others' bins: the segments' masses may take their place
    }
    // ---- kept mass of every segment, then of every CTA
    unsigned long long own = 0;
    const uint32_t zb = bound_of(from_logit_key(theta), T());   // (theta is an element's or the floor's key)
    if (summed) {
        for (int i = tid; i < s1 - s0; i += UNT) own += smass[i];
    } else {
        for (int s = s0 + warp; s < s1; s += UNW) {
            unsigned long long v = 0;
            if (segs[s] >= theta) {
                const uint4 x = row.load(s, lane);
                for (uint32_t hit = hits(x, zb, T()); hit; hit &= hit - 1) {
                    const unsigned long long w = wt.weight_of(element(x, __ffs(hit) - 1, T()));
                    if (w >= wmin) v += w;
                }
                v = warp_mass(v);
            }
            if (lane == 0) {
                smass[s - s0] = v;
                own += v;
            }
        }
    }
    own = block_sum(own, c);
    if (tid < C) peer(c->cmass, tid)[rank] = own;
    sync(C);
    unsigned long long Z = 0, before = 0;
    for (int q = 0; q < C; ++q) {
        if (q < rank) before += c->cmass[q];
        Z += c->cmass[q];
    }
    if (Z == 0) {
        if (rank == 0 && tid == 0) a.out_token[b] = -1, a.out_valid[b] = 0;
        return;
    }
    bool cut;
    const unsigned long long t = u > 0.f ? mul_frac(u, Z, cut) : 0;
    if (t < before || t - before >= own) return;  // another CTA holds the token
    // ---- the segment, then the element
    const unsigned long long tl = t - before;
    const int ns = s1 - s0, each_t = (ns + UNT - 1) / UNT;
    unsigned long long v = 0;
    const int f0 = min(ns, tid * each_t), f1 = min(ns, f0 + each_t);
    for (int s = f0; s < f1; ++s) v += smass[s];
    const unsigned long long mine = v;
    block_prefix_mass(v, c);
    if (v <= tl && tl - v < mine) {
        for (int s = f0; s < f1; ++s) {
            if (tl - v < smass[s]) {
                c->seg = s0 + s;
                c->rest = tl - v;
                break;
            }
            v += smass[s];
        }
    }
    __syncthreads();
    if (warp == 0) {
        const int s = c->seg;
        const unsigned long long rest = c->rest;
        float z[R::N];
        unpack(row.load(s, lane), z, T());
        unsigned long long w[R::N], sum = 0;
#pragma unroll
        for (int e = 0; e < R::N; ++e) {
            w[e] = ukey(z[e]) >= theta ? wt.weight_of(z[e]) : 0;
            if (w[e] < wmin) w[e] = 0;
            sum += w[e];
        }
        unsigned long long at = warp_incl_scan_u64(sum, lane) - sum;
        if (at <= rest && rest - at < sum) {
            int tok = -1;
#pragma unroll
            for (int e = 0; e < R::N; ++e) {
                if (tok < 0 && rest - at < w[e]) tok = s * R::SEG + lane * R::N + e - row.a0;
                if (tok < 0) at += w[e];
            }
            a.out_token[b] = tok;
            a.out_valid[b] = 1;
        }
    }
}

// ------------------------------------------------------------------ host

static int row_segments(int vocab, int es) { return int((int64_t(vocab) + 16 / es - 1 + 512 / es - 1) / (512 / es)); }

template <typename T>
static fs_status run_uniform(UniformArgs& a, int C, int sms, size_t optin, void* stream) {
    const void* fn = reinterpret_cast<const void*>(uniform_kernel<T>);
    const fs_status st = prepare_kernel(fn);
    if (st != FS_OK) return st;
    a.nsc = (a.ls + C - 1) / C;
    const size_t smem = USmem::total(a.nsc, a.ls);
    if (smem > optin) return FS_ERR_UNSUPPORTED;
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.x = unsigned(C);
    attr[1].val.clusterDim.y = 1;
    attr[1].val.clusterDim.z = 1;
    cudaLaunchConfig_t cfg = {};
    cfg.stream = static_cast<cudaStream_t>(stream);
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    cfg.blockDim = dim3(256, 1, 1);
    const int64_t trips = int64_t(a.batch_in) * ((a.ls + USEG_TRIP - 1) / USEG_TRIP);
    cfg.gridDim = dim3(unsigned(std::max<int64_t>(1, std::min<int64_t>((trips + 7) / 8, int64_t(sms) * 8))), 1, 1);
    cudaError_t e = a.ssum ? cudaLaunchKernelEx(&cfg, seg_max_kernel<T, true>, a)
                           : cudaLaunchKernelEx(&cfg, seg_max_kernel<T, false>, a);
    if (e != cudaSuccess) return cuda_fail(e);
    cfg.numAttrs = 2;
    cfg.blockDim = dim3(UNT, 1, 1);
    cfg.gridDim = dim3(unsigned(a.nout) * unsigned(C), 1, 1);
    cfg.dynamicSmemBytes = smem;
    e = cudaLaunchKernelEx(&cfg, uniform_kernel<T>, a);
    return e == cudaSuccess ? FS_OK : cuda_fail(e);
}

}  // namespace fsd

extern "C" {

fs_status fs_from_uniforms_workspace_bytes(int32_t dtype, int32_t batch_in, int32_t vocab, size_t* bytes) {
    if (!bytes || batch_in < 0 || vocab < 1) return FS_ERR_INVALID_ARG;
    if (dtype != FS_F32 && dtype != FS_BF16 && dtype != FS_F16) return FS_ERR_INVALID_ARG;
    if (vocab > FS_MAX_VOCAB) return FS_ERR_UNSUPPORTED;
    *bytes = size_t(batch_in) * size_t(fsd::row_segments(vocab, dtype == FS_F32 ? 4 : 2)) * 8;
    return FS_OK;
}

fs_status fs_top_k_top_p_sampling_from_uniforms(const void* logits, int32_t dtype, int64_t row_stride, int32_t batch_in,
                                                int32_t vocab, const int32_t* indices, int32_t batch_out,
                                                const float* uniforms, const float* temperature, const int32_t* top_k,
                                                const float* top_p, const float* min_p, int32_t order,
                                                int32_t* out_token, uint8_t* out_valid, void* workspace,
                                                size_t workspace_bytes, void* stream) {
    using namespace fsd;
    size_t need = 0;
    const fs_status st = fs_from_uniforms_workspace_bytes(dtype, batch_in, vocab, &need);
    if (st != FS_OK) return st;
    if (batch_out < 0 || (!indices && batch_out != batch_in)) return FS_ERR_INVALID_ARG;
    if (order != FS_ORDER_TOP_K_FIRST && order != FS_ORDER_JOINT) return FS_ERR_INVALID_ARG;
    if (batch_in > 1 && row_stride < vocab) return FS_ERR_INVALID_ARG;
    if (batch_out == 0) return FS_OK;
    const int es = dtype == FS_F32 ? 4 : 2;
    if (!uniforms || !out_token || !out_valid || (batch_in > 0 && (!logits || !workspace))) return FS_ERR_INVALID_ARG;
    if (reinterpret_cast<uintptr_t>(logits) % es != 0 || reinterpret_cast<uintptr_t>(workspace) % 4 != 0)
        return FS_ERR_INVALID_ARG;
    if (workspace_bytes < need) {
        set_last_error("sampling from uniforms: the workspace is too small");
        return FS_ERR_INVALID_ARG;
    }
    UniformArgs a = {};
    a.x = logits;
    a.stride = row_stride;
    a.batch_in = batch_in;
    a.V = vocab;
    a.indices = indices;
    a.nout = batch_out;
    a.u = uniforms;
    a.temperature = temperature;
    a.top_k = top_k;
    a.top_p = top_p;
    a.min_p = min_p;
    a.order = order;
    a.out_token = out_token;
    a.out_valid = out_valid;
    a.skey = static_cast<uint32_t*>(workspace);
    a.ls = row_segments(vocab, es);
    // The total mass of a row goes with its segments' maxima where a small set is measured
    // against it and the row has one temperature.
    if (!indices && order == FS_ORDER_JOINT && top_p && (top_k || min_p))
        a.ssum = reinterpret_cast<float*>(a.skey + size_t(batch_in) * a.ls);
    // CTAs per row: one where a small set needs only the summary,
    // else as many as fill the GPU with two per SM; a power of two.  (By the arguments given: a row whose top_k
    // or min_p turns out to be off, or whose set is too large for the list, has one CTA too.)
    int C = 1, sms = 0;
    size_t optin = 0;
    const fs_status found = device_limits(sms, optin);
    if (found != FS_OK) return found;
    const bool whole = (!top_k && (top_p || !min_p)) || (order == FS_ORDER_JOINT && top_p && !a.ssum);
    if (whole)
        while (C < 8 && int64_t(batch_out) * C * 2 <= int64_t(sms) * 2 && a.ls >= C * 2 * 16) C *= 2;
    while (C < 8 && USmem::total((a.ls + C - 1) / C, a.ls) > (200u << 10)) C *= 2;
    if (int64_t(batch_out) * C > 0x7fffffffLL) return FS_ERR_UNSUPPORTED;
    switch (dtype) {
        case FS_F32: return run_uniform<float>(a, C, sms, optin, stream);
        case FS_BF16: return run_uniform<__nv_bfloat16>(a, C, sms, optin, stream);
        default: return run_uniform<__half>(a, C, sms, optin, stream);
    }
}

}  // extern "C"
