// Sampling with temperature, top-k, top-p and min-p from given random numbers (sm_103a).
//
// One number u in [0, 1) per output row decides its token.  With w_i = exp((z_i - m) / T),
// m the row's maximum, and S the kept set (every filter is a threshold on z), the token is
//   the first i of S, in index order, with  sum_{j in S, j <= i} w_j > u * sum_{j in S} w_j.
// Unlike the rejection sampler this needs the masses themselves, not only an accepted
// draw, and the decisions (which token the top-p mass ends on, which token u falls on)
// are borders between neighbours that may differ by 10^-6 of the row: a float32 sum would
// answer another token for flat rows.  So weights are 64-bit fixed-point integers,
// round(2^42 w) to within one unit and a relative 4e-11 (weight_of), and every sum and
// comparison is exact integer arithmetic.  Sums then do not depend on their order, the
// launch shape or atomics.
//
// Two launches.  seg_max_kernel streams every input row once, spread evenly over the GPU,
// and writes the largest order key of each segment (one 16-byte load per lane of a warp).
// uniform_kernel, one cluster of C CTAs per output row, reads those keys and then:
//   small top-k  segments whose maximum reaches the k-th largest segment maximum hold
//                every element of the top k; their elements at or above that bound (a
//                few dozen more than k) go into a list in shared memory, and every
//                decision is made there;
//   otherwise    a histogram of the weights over 2048 bins linear in m - z finds the bin
//                a threshold lies in, further histograms over the order keys inside it
//                find the exact key; one pass then leaves each segment's kept mass, and
//                one segment is read to find the token.
#include <algorithm>

#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include "fs_device.cuh"
#include "fs_host.h"

namespace fsd {

constexpr int UNT = 512;          // threads of uniform_kernel
constexpr int UNW = UNT / 32;
constexpr int UB = 2048;          // histogram bins
constexpr int UCAP = 512;         // candidates of the small top-k path
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
// Order key with -0 equal to +0.
__device__ __forceinline__ uint32_t ukey(float z) { return logit_key(z + 0.f); }

// ------------------------------------------------------------------ segment maxima

// Warp w of the grid takes trips of USEG_TRIP segments w, w + W, ...; bound by the HBM
// read.  A NaN marks its segment with the largest key.
template <typename T>
__global__ void __launch_bounds__(256) seg_max_kernel(const UniformArgs a) {
    using R = URow<T>;
    grid_dependency_wait();
    allow_dependents();
    const int lane = threadIdx.x & 31;
    const int trips = (a.ls + USEG_TRIP - 1) / USEG_TRIP;
    const int64_t total = int64_t(a.batch_in) * trips;
    for (int64_t w = int64_t(blockIdx.x) * 8 + (threadIdx.x >> 5); w < total; w += int64_t(gridDim.x) * 8) {
        const int r = int(w / trips), s0 = int(w - int64_t(r) * trips) * USEG_TRIP;
        const R row(a.x, a.stride, r, a.V);
        uint4 v[USEG_TRIP];
#pragma unroll
        for (int j = 0; j < USEG_TRIP; ++j)
            if (s0 + j < row.nseg) v[j] = row.load(s0 + j, lane);
#pragma unroll
        for (int j = 0; j < USEG_TRIP; ++j) {
            if (s0 + j >= row.nseg) continue;
            float z[R::N];
            unpack(v[j], z, T());
            uint32_t k = 0;
#pragma unroll
            for (int e = 0; e < R::N; ++e) k = max(k, z[e] == z[e] ? ukey(z[e]) : 0xffffffffu);
            k = warp_max_u(k);
            if (lane == 0) a.skey[int64_t(r) * a.ls + s0 + j] = k;
        }
    }
}

// ------------------------------------------------------------------ weights

// 2^(j / 32) * 2^42, rounded.
__constant__ unsigned long long EXP2_32[32] = {
    0x40000000000ull, 0x4166c34c561ull, 0x42d561b3e62ull, 0x444c0740497ull, 0x45cae0f1f54ull, 0x47521cc5a2eull,
    0x48e1e9b9d59ull, 0x4a7a77d47f8ull, 0x4c1bf828c6eull, 0x4dc69cdceaaull, 0x4f7a993048dull, 0x51382181862ull,
    0x52ff6b54d8bull, 0x54d0ad5a754ull, 0x56ac1f75215ull, 0x5891fac0e95ull, 0x5a827999fcfull, 0x5c7dd7a3b18ull,
    0x5e8451cfac0ull, 0x60962665334ull, 0x62b39508aa8ull, 0x64dcdec3371ull, 0x6712460a8fcull, 0x69540ec8f89ull,
    0x6ba27e656b5ull, 0x6dfddbcbed8ull, 0x70666f76155ull, 0x72dc8373be4ull, 0x75606373ee9ull, 0x77f25ccdee7ull,
    0x7a92be8a924ull, 0x7d41d96db91ull};

struct Weigher {
    float hm;          // m / 2
    float ch, cl;      // 2 log2(e) / T as a sum of two floats
    float m, inv_w;    // bins: (m - z) / 2 * inv_w, 2048 bins up to m - z = 30.5 T (weights there round to 0)
    const unsigned long long* tab;  // EXP2_32 in shared memory
    __device__ __forceinline__ Weigher(float m_, float T, const unsigned long long* t) : m(m_), tab(t) {
        hm = 0.5f * m_;
        const double c = 2.8853900817779268 / double(T);
        ch = float(c);
        cl = float(c - double(ch));
        inv_w = fminf(float(UB) / (15.25f * T), 3.0e38f);
    }
    // round(2^42 exp((z - m) / T)), z <= m.  The exponent (z - m) log2(e) / T as a sum of two
    // floats (halved operands, so that the difference cannot overflow; its rounding error
    // by the two-sum); split into n + j / 32 + r, |r| <= 1/64; 2^r - 1 as the product r ln 2 in two
    // floats plus a cubic remainder in one; then integers.  About 45 instructions.
    __device__ __forceinline__ unsigned long long weight_of(float z) const {
        const float h = 0.5f * z;
        const float d = __fsub_rn(h, hm), bb = __fsub_rn(d, h);
        const float dl = __fadd_rn(__fsub_rn(h, __fsub_rn(d, bb)), __fsub_rn(-hm, bb));
        const float yh = __fmul_rn(d, ch);
        if (!(yh > -44.f)) return 0;  // also -inf, whose product with a zero slope is NaN
        float yl = fmaf(d, ch, -yh);
        yl = fmaf(d, cl, yl);
        yl = fmaf(dl, ch, yl);
        const float t = fmaf(yh, 32.f, 12582912.f);  // + 1.5 * 2^23: the nearest integer in the low bits
        const int q = __float_as_int(t) - 0x4B400000;
        const float r0 = fmaf(__fsub_rn(t, 12582912.f), -0.03125f, yh);
        const float r = __fadd_rn(r0, yl), rl = __fsub_rn(yl, __fsub_rn(r, r0));
        constexpr float L = 0.693147182464599609375f, LL = -1.904654323148236017e-9f;  // ln 2
        const float sh = __fmul_rn(r, L);
        float sl = fmaf(r, L, -sh);
        sl = fmaf(r, LL, sl);
        sl = fmaf(rl, L, sl);
        const float c = fmaf(r, fmaf(r, 0.009618129107628477f, 0.05550410866482158f), 0.2402265069591007f);
        sl = fmaf(__fmul_rn(r, r), c, sl);
        // 2^r - 1 in units of 2^-36
        const int s = __float2int_rn(sh * 0x1p36f) + (__float_as_int(fmaf(sl, 0x1p36f, 12582912.f)) - 0x4B400000);
        const unsigned long long tj = tab[q & 31];
        const long long prod = (long long)int(tj >> 12) * s + (1 << 23);
        const unsigned long long v = tj + (unsigned long long)(prod >> 24);
        const int n = -(q >> 5);
        return (v + ((1ull << n) >> 1)) >> n;
    }
    // Bin of z: 0 the largest.  Each step is monotone in z, so a lower bin means larger z.
    __device__ __forceinline__ int bin_of(float z) const {
        return int(fminf(__fmul_rn(__fsub_rn(hm, 0.5f * z), inv_w), float(UB - 1)));
    }
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
    unsigned long long tab[32];
    unsigned long long red[UNW];
    uint32_t redc[UNW];
    unsigned long long cmass[MAX_CLUSTER];
    unsigned long long above, in_mass;  // find_bin's results
    uint32_t above_cnt, in_cnt;
    int bin;
    int n;               // candidates
    int nlive;
    unsigned long long fmass;
    int flag;
    int seg;
    unsigned long long rest;
};

struct USmem {
    static constexpr size_t CTL = 0;
    static constexpr size_t LKEY = align16(sizeof(UCtl));
    static constexpr size_t LPOS = LKEY + UCAP * 4;
    static constexpr size_t LW = LPOS + UCAP * 4;
    static constexpr size_t LK = LW + UCAP * 8;
    static constexpr size_t HIST = LK + UCAP * 8;     // masses, counts, their totals; later the segments' masses
    static constexpr size_t HIST_BYTES = size_t(UB) * 24;
    static __host__ __device__ size_t seg_at(int nsc) { return HIST + (size_t(nsc) * 8 > HIST_BYTES ? align16(size_t(nsc) * 8) : HIST_BYTES); }
    static __host__ __device__ size_t total(int nsc, int ls) { return seg_at(nsc) + align16(size_t(ls) * 4); }
};

template <typename X>
__device__ __forceinline__ X* peer(X* p, int rank) {
    return static_cast<X*>(__cluster_map_shared_rank(p, unsigned(rank)));
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

// The first bin at which the running mass (by_mass) or count reaches target >= 1; the sums before it
// and in it go into the control words (bin UB when it is never reached).  Block-wide.
__device__ __forceinline__ void find_bin(const unsigned long long* mass, const uint32_t* cnt, bool by_mass,
                                         unsigned long long target, UCtl* c) {
    constexpr int PER = UB / UNT;
    const int b0 = threadIdx.x * PER;
    unsigned long long v = 0;
    uint32_t n = 0;
#pragma unroll
    for (int i = 0; i < PER; ++i) {
        if (mass) v += mass[b0 + i];
        n += cnt[b0 + i];
    }
    const unsigned long long own = by_mass ? v : n;
    block_prefix(v, n, c);
    if (threadIdx.x == 0) c->bin = UB;
    __syncthreads();
    const unsigned long long before = by_mass ? v : n;
    if (before < target && before + own >= target) {
        for (int i = 0; i < PER; ++i) {
            const unsigned long long mi = mass ? mass[b0 + i] : 0;
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

// A 64-bit add into a shared counter by 32-bit atomics: the low word's carry goes on.
__device__ __forceinline__ void add64(unsigned long long* p, unsigned long long v) {
    uint32_t* w = reinterpret_cast<uint32_t*>(p);
    const uint32_t lo = uint32_t(v), old = atomicAdd(w, lo);
    const uint32_t hi = uint32_t(v >> 32) + (old + lo < old ? 1u : 0u);
    if (hi) atomicAdd(w + 1, hi);
}

template <typename T>
__global__ void __launch_bounds__(UNT, 2) uniform_kernel(const UniformArgs a) {
    using R = URow<T>;
    extern __shared__ __align__(16) unsigned char smem[];
    UCtl* c = reinterpret_cast<UCtl*>(smem + USmem::CTL);
    uint32_t* lkey = reinterpret_cast<uint32_t*>(smem + USmem::LKEY);
    int* lpos = reinterpret_cast<int*>(smem + USmem::LPOS);
    unsigned long long* lw = reinterpret_cast<unsigned long long*>(smem + USmem::LW);
    unsigned long long* lk = reinterpret_cast<unsigned long long*>(smem + USmem::LK);
    unsigned long long* hmass = reinterpret_cast<unsigned long long*>(smem + USmem::HIST);
    unsigned long long* tmass = hmass + UB;
    uint32_t* hcnt = reinterpret_cast<uint32_t*>(tmass + UB);
    uint32_t* tcnt = hcnt + UB;
    unsigned long long* smass = hmass;  // [nsc], after the histograms
    uint32_t* segs = reinterpret_cast<uint32_t*>(smem + USmem::seg_at(a.nsc));
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int C = int(cluster_nctarank()), rank = int(cluster_ctarank()), b = int(cluster_id_x());
    if (tid < 32) c->tab[tid] = EXP2_32[tid];
    if (tid == 0) c->n = 0, c->nlive = 0, c->flag = 0;
    cluster_sync();  // every CTA of the cluster runs before another writes into its memory
    grid_dependency_wait();
    allow_dependents();

    // ---- parameters; the row's maximum
    const int r = a.indices ? a.indices[b] : b;
    const float u = a.u[b];
    const float temp = a.temperature ? a.temperature[b] : 1.f;
    const int k = a.top_k ? a.top_k[b] : 0;
    const float p = a.top_p ? a.top_p[b] : 1.f;
    const float mp = a.min_p ? a.min_p[b] : 0.f;
    bool bad = r < 0 || r >= a.batch_in || !(u >= 0.f && u < 1.f) || !(temp >= 1.17549435e-38f) || !(p == p) || !(mp <= 1.f);
    uint32_t kmax = 0;
    if (!bad) {
        const R row(a.x, a.stride, r, a.V);
        for (int s = tid; s < row.nseg; s += UNT) {
            const uint32_t sk = a.skey[int64_t(r) * a.ls + s];
            segs[s] = sk;
            kmax = max(kmax, sk);
        }
        kmax = warp_max_u(kmax);
        if (lane == 0) c->redc[warp] = kmax;
        __syncthreads();
#pragma unroll
        for (int w = 0; w < UNW; ++w) kmax = max(kmax, c->redc[w]);
        bad = kmax >= KEY_PINF || kmax <= KEY_NINF;
    }
    if (bad) {  // the same in every thread of the cluster
        if (rank == 0 && tid == 0) a.out_token[b] = -1, a.out_valid[b] = 0;
        return;
    }
    __syncthreads();
    const R row(a.x, a.stride, r, a.V);
    const Weigher wt(from_logit_key(kmax), temp, c->tab);
    const unsigned long long ONE = 1ull << 42;
    const bool has_k = k > 0 && k < a.V, has_p = p < 1.f;
    // min-p: w >= mp * max w; the integers are compared, rounded up
    unsigned long long wmin = 1;
    if (mp > 0.f && mp < 1.f) {
        bool cut;
        wmin = mul_frac(mp, ONE, cut);
        wmin = max(1ull, wmin + (cut ? 1 : 0));
    } else if (mp >= 1.f) {
        wmin = ONE;
    }
    // This CTA's segments.
    const int per = (row.nseg + C - 1) / C;
    const int s0 = min(row.nseg, rank * per), s1 = min(row.nseg, s0 + per);
    // fn(z, position) over the elements of this CTA's segments.
    auto each = [&](auto fn) {
        for (int s = s0 + warp; s < s1; s += UNW * 2) {
            const bool two = s + UNW < s1;
            const uint4 v0 = row.load(s, lane);
            uint4 v1 = v0;
            if (two) v1 = row.load(s + UNW, lane);
            float z[R::N];
            unpack(v0, z, T());
#pragma unroll
            for (int e = 0; e < R::N; ++e) fn(z[e]);
            if (two) {
                unpack(v1, z, T());
#pragma unroll
                for (int e = 0; e < R::N; ++e) fn(z[e]);
            }
        }
    };
    auto clear = [&]() {
        for (int i = tid; i < UB; i += UNT) hmass[i] = 0, hcnt[i] = 0;
        __syncthreads();
    };
    // The cluster's histograms summed into every CTA's totals.
    auto totals = [&]() {
        cluster_sync();
        const int n = UB / C;
        for (int i = rank * n + tid; i < (rank + 1) * n; i += UNT) {
            unsigned long long v = 0;
            uint32_t m = 0;
            for (int q = 0; q < C; ++q) v += *peer(hmass + i, q), m += *peer(hcnt + i, q);
            for (int q = 0; q < C; ++q) *peer(tmass + i, q) = v, *peer(tcnt + i, q) = m;
        }
        cluster_sync();
    };

    // ---- the row's total mass, where top-p is measured against it
    const bool joint = a.order == FS_ORDER_JOINT || !has_k;
    // ---- small top-k: everything in a list
    bool small = false;
    if (has_k && k <= UCAP) {
        for (int i = tid; i < UB; i += UNT) hcnt[i] = 0;
        __syncthreads();
        for (int s = tid; s < row.nseg; s += UNT) atomicAdd(&hcnt[wt.bin_of(from_logit_key(segs[s]))], 1u);
        __syncthreads();
        find_bin(nullptr, hcnt, false, (unsigned long long)k, c);
        const int kb = c->bin;
        small = kb < UB - 1;  // the last bin has no weight, and UB means fewer segments than k
        if (small) {
            if (rank == 0) {
                // The live segments, one per warp and turn; elements in bins up to kb.
                int* live = reinterpret_cast<int*>(hmass);
                for (int s = tid; s < row.nseg; s += UNT)
                    if (wt.bin_of(from_logit_key(segs[s])) <= kb) {
                        const int at = atomicAdd(&c->nlive, 1);
                        if (at < UCAP) live[at] = s;
                    }
                __syncthreads();
                // each live segment holds a candidate, so more of them than UCAP are too many
                const int nl = min(c->nlive, UCAP);
                for (int i = warp; i < nl; i += UNW) {
                    float z[R::N];
                    unpack(row.load(live[i], lane), z, T());
#pragma unroll
                    for (int e = 0; e < R::N; ++e) {
                        if (wt.bin_of(z[e]) <= kb) {
                            const int at = atomicAdd(&c->n, 1);
                            if (at < UCAP) {
                                lkey[at] = ukey(z[e]);
                                lpos[at] = live[i] * R::SEG + lane * R::N + e;
                                lw[at] = wt.weight_of(z[e]);
                            }
                        }
                    }
                }
                __syncthreads();
                if (tid < C) *peer(&c->flag, tid) = c->nlive <= UCAP && c->n <= UCAP ? 1 : 0;
            }
            cluster_sync();
            small = c->flag != 0;
        }
    }
    unsigned long long M = 0;
    if (small && has_p && a.order == FS_ORDER_JOINT) {
        unsigned long long v = 0;
        each([&](float z) { v += wt.weight_of(z); });
        v = block_sum(v, c);
        if (tid < C) peer(c->cmass, tid)[rank] = v;
        cluster_sync();
        for (int q = 0; q < C; ++q) M += c->cmass[q];
    }
    if (small) {
        if (rank != 0) return;
        const int n = c->n;
        // Threads per candidate (a power of two, within a warp), each over its share of the list.
        int tpc = 1;
        while (tpc < 32 && tpc * 2 * n <= UNT) tpc *= 2;
        const int i = tid / tpc, sub = tid % tpc;
        const uint32_t ki = i < n ? lkey[i] : 0xffffffffu;
        int cnt = 0;
        unsigned long long above = 0;
        for (int j = sub; j < n; j += tpc)
            if (lkey[j] > ki) ++cnt, above += lw[j];
        for (int d = 1; d < tpc; d *= 2) {
            cnt += __shfl_xor_sync(FULL, cnt, d);
            above += __shfl_xor_sync(FULL, above, d);
        }
        bool keep = i < n && cnt < k;  // ties with the k-th are kept
        const unsigned long long wi = i < n ? lw[i] : 0;
        if (has_p) {
            const unsigned long long F = joint ? M : block_sum(keep && sub == 0 ? wi : 0, c);
            bool cut = false;
            unsigned long long G = p > 0.f ? mul_frac(p, F, cut) : 0;
            G = max(1ull, G + (cut ? 1 : 0));
            keep = keep && above < G;
        }
        keep = keep && wi >= wmin;
        const unsigned long long kept = keep ? wi : 0;
        if (i < n && sub == 0) lk[i] = kept;
        const unsigned long long Z = block_sum(sub == 0 ? kept : 0, c);
        bool cut;
        const unsigned long long t = u > 0.f ? mul_frac(u, Z, cut) : 0;
        unsigned long long incl = 0;
        const int pi = i < n ? lpos[i] : -1;
        for (int j = sub; j < n; j += tpc)
            if (lpos[j] <= pi) incl += lk[j];
        for (int d = 1; d < tpc; d *= 2) incl += __shfl_xor_sync(FULL, incl, d);
        if (keep && sub == 0 && incl > t && incl - kept <= t) a.out_token[b] = pi - row.a0, a.out_valid[b] = 1;
        if (Z == 0 && tid == 0) a.out_token[b] = -1, a.out_valid[b] = 0;
        return;
    }

    // ---- thresholds from histograms
    uint32_t theta = KEY_NINF + 1;
    const bool want_k = has_k;
    if (want_k || has_p) {
        clear();
        each([&](float z) {
            const int q = wt.bin_of(z);
            const unsigned long long w = wt.weight_of(z);
            if (w) add64(hmass + q, w);
            atomicAdd(hcnt + q, 1u);
        });
        totals();
        // The largest key whose elements at or above it reach `target` (count or mass); the mass at
        // or above it goes into `fmass`.  Keys are narrowed by histograms inside the bin.
        auto search = [&](bool by_mass, unsigned long long target, unsigned long long& fmass) -> uint32_t {
            find_bin(tmass, tcnt, by_mass, target, c);
            const int qb = c->bin;
            if (qb >= UB - 1) return 0;  // reached only among elements without weight
            unsigned long long above = c->above;
            unsigned long long above_t = by_mass ? c->above : c->above_cnt;
            fmass = above + c->in_mass;
            // Keys the bin can hold, with some slack for the rounding of its edges.
            const float wid = 2.f / wt.inv_w;
            const float lo = wt.m - float(qb + 1) * wid, hi = wt.m - float(qb) * wid;
            const float sl = 0x1p-20f * (fabsf(wt.m) + float(qb + 1) * wid);
            uint32_t kl = max(KEY_NINF + 1, ukey(lo - sl == lo - sl ? fmaxf(lo - sl, -3.402823466e38f) : -3.402823466e38f));
            uint32_t kh = min(kmax, ukey(hi + sl == hi + sl ? fminf(hi + sl, 3.402823466e38f) : 3.402823466e38f));
            while (kh > kl) {
                const int bits = 32 - __clz(kh - kl);
                const int sh = bits > 11 ? bits - 11 : 0;
                // the totals of the linear bins are needed again by a later search: own ones here
                __syncthreads();
                clear();
                each([&](float z) {
                    const uint32_t key = ukey(z);
                    if (key >= kl && key <= kh && wt.bin_of(z) == qb) {
                        const int q = int((kh - key) >> sh);
                        add64(hmass + q, wt.weight_of(z));
                        atomicAdd(hcnt + q, 1u);
                    }
                });
                // Summed into the leader's own bins first, then copied to every CTA.
                cluster_sync();
                const int n = UB / C;
                unsigned long long v[UB / UNT];
                uint32_t m[UB / UNT];
#pragma unroll
                for (int i = 0; i < UB / UNT; ++i) {
                    const int at = rank * n + tid + i * UNT;
                    v[i] = 0, m[i] = 0;
                    if (tid + i * UNT < n)
                        for (int q = 0; q < C; ++q) v[i] += *peer(hmass + at, q), m[i] += *peer(hcnt + at, q);
                }
                cluster_sync();
#pragma unroll
                for (int i = 0; i < UB / UNT; ++i) {
                    const int at = rank * n + tid + i * UNT;
                    if (tid + i * UNT < n)
                        for (int q = 0; q < C; ++q) *peer(hmass + at, q) = v[i], *peer(hcnt + at, q) = m[i];
                }
                cluster_sync();
                find_bin(hmass, hcnt, by_mass, target - above_t, c);
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
        unsigned long long F = 0, dummy = 0;
        for (int q = tid; q < UB; q += UNT) F += tmass[q];
        F = block_sum(F, c);
        if (want_k) {
            unsigned long long fk = F;
            theta = max(theta, search(false, (unsigned long long)k, fk));
            if (!joint) F = fk;
        }
        if (has_p) {
            bool cut = false;
            unsigned long long G = p > 0.f ? mul_frac(p, F, cut) : 0;
            G = max(1ull, G + (cut ? 1 : 0));
            theta = max(theta, search(true, G, dummy));
        }
        cluster_sync();  // every CTA has read the others' bins: the segments' masses may take their place
    }
    // ---- kept mass of every segment, then of every CTA
    unsigned long long own = 0;
    for (int s = s0 + warp; s < s1; s += UNW) {
        unsigned long long v = 0;
        if (segs[s] >= theta) {
            float z[R::N];
            unpack(row.load(s, lane), z, T());
#pragma unroll
            for (int e = 0; e < R::N; ++e) {
                if (ukey(z[e]) >= theta) {
                    const unsigned long long w = wt.weight_of(z[e]);
                    if (w >= wmin) v += w;
                }
            }
            v = warp_sum_u64(v);
        }
        if (lane == 0) smass[s - s0] = v;
        own += v;
    }
    own = block_sum(lane == 0 ? own : 0, c);
    if (tid < C) peer(c->cmass, tid)[rank] = own;
    cluster_sync();
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
    uint32_t none = 0;
    const int f0 = min(ns, tid * each_t), f1 = min(ns, f0 + each_t);
    for (int s = f0; s < f1; ++s) v += smass[s];
    const unsigned long long mine = v;
    block_prefix(v, none, c);
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
static fs_status run_uniform(UniformArgs& a, int C, void* stream) {
    int sms = 0;
    size_t optin = 0;
    fs_status st = device_limits(sms, optin);
    if (st != FS_OK) return st;
    const void* fn = reinterpret_cast<const void*>(uniform_kernel<T>);
    st = prepare_kernel(fn);
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
    cudaError_t e = cudaLaunchKernelEx(&cfg, seg_max_kernel<T>, a);
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
    *bytes = size_t(batch_in) * size_t(fsd::row_segments(vocab, dtype == FS_F32 ? 4 : 2)) * 4;
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
    // CTAs per row: one where the list path needs only the summary (top-k without a total mass),
    // else as many as fill the GPU with two per SM; a power of two.
    int C = 1;
    const bool whole = !top_k || (order == FS_ORDER_JOINT && top_p);
    if (whole)
        while (C < 8 && int64_t(batch_out) * C * 2 <= 304 && a.ls >= C * 2 * 16) C *= 2;
    while (C < 8 && USmem::total((a.ls + C - 1) / C, a.ls) > (200u << 10)) C *= 2;
    if (int64_t(batch_out) * C > 0x7fffffffLL) return FS_ERR_UNSUPPORTED;
    switch (dtype) {
        case FS_F32: return run_uniform<float>(a, C, stream);
        case FS_BF16: return run_uniform<__nv_bfloat16>(a, C, stream);
        default: return run_uniform<__half>(a, C, stream);
    }
}

}  // extern "C"
