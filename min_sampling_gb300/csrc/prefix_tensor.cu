// The shared prefix's part of attention on the 5th-generation tensor cores (sm_103a).
//
// One CTA per (query tile of a group, key/value head, range of keys).  The queries of all
// rows of a group that read one key/value head form the rows of two matrix products per
// tile of 128 keys: S = Q K^T, then O += P V with P = 2^(S - m).  S, P and O live in tensor
// memory: S (128 x 128 float32) is turned into P (16 bits) in place, and P feeds the second product from
// there.  Roles of the 16 warps:
//   warps 0-3, 4-7  softmax of tile 0 / tile 1, one thread per query: maximum, weights,
//                   sum; O is rescaled only when a maximum grows by more than 2^8 (P and the
//                   sum then stay within 2^8 of their range: exact in float32, no overflow in f16)
//   warps 8-11      keys and values: page look-ups and 16-byte asynchronous copies into
//                   a ring of swizzled tiles (any page size and strides)
//   warp 12         one thread issues the matrix instructions
// Two tiles are in flight so that one tile's softmax runs under the other's products:
//   SPLIT = false   256 queries, both tiles over the same keys
//   SPLIT = true    up to 128 queries, the tiles take alternate key tiles and are joined at
//                   the end
// Every wait on a barrier is bounded; one that runs out marks the CTA, which then drains
// its copies, frees its tensor memory and writes NaN.
#include "attention.cuh"

namespace fsd {

constexpr int TK = 128;          // keys per tile
constexpr int TNT = 512;         // threads
constexpr int LAG = 2;           // tiles of copies in flight behind the newest before one is handed over
constexpr uint32_t SPIN = 1u << 22;

template <int D, bool SPLIT>
struct TensorSmem {
    static constexpr int TILE = TK * D * 2;                  // 128 rows of queries, keys or values
    static constexpr int NQ = SPLIT ? 1 : 2;
    static constexpr int STAGES = D == 128 ? 7 - NQ : 8;
    static constexpr int KV = NQ * TILE;
    static constexpr int BARS = KV + STAGES * TILE;
    static constexpr int OUTS = BARS + 256;                  // the query rows' output rows
    static constexpr int OFFS = BARS - TILE;                 // their addresses, in the ring's last tile until it is loaded
    static constexpr int TOTAL = OUTS + NQ * TK * 4 + 1024;  // 1024: the base's alignment
};

// ------------------------------------------------------------------ barriers

__device__ __forceinline__ void bar_init(uint32_t bar, uint32_t count) {
    asm volatile("mbarrier.init.shared::cta.b64 [%0], %1;" ::"r"(bar), "r"(count) : "memory");
}
__device__ __forceinline__ void bar_arrive(uint32_t bar) {
    asm volatile("{ .reg .b64 t; mbarrier.arrive.shared::cta.b64 t, [%0]; }" ::"r"(bar) : "memory");
}
__device__ __forceinline__ bool bar_try(uint32_t bar, uint32_t parity) {
    uint32_t ok;
    asm volatile(
        "{ .reg .pred p; mbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2; selp.u32 %0, 1, 0, p; }"
        : "=r"(ok) : "r"(bar), "r"(parity) : "memory");
    return ok != 0;
}
// False when the wait ran out here or in another role of the CTA.
__device__ __forceinline__ bool bar_wait(uint32_t bar, uint32_t parity, volatile int* dead) {
    for (uint32_t i = 0; i < SPIN; ++i) {
        if (bar_try(bar, parity)) return true;
        if ((i & 63) == 63 && *dead) return false;
    }
    *dead = 1;
    return false;
}

// ------------------------------------------------------------------ tensor memory and matrix instructions

__device__ __forceinline__ void tmem_fence_before() { asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory"); }
__device__ __forceinline__ void tmem_fence_after() { asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory"); }
__device__ __forceinline__ void tmem_wait_ld() { asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory"); }
__device__ __forceinline__ void tmem_wait_st() { asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory"); }
__device__ __forceinline__ void proxy_fence() { asm volatile("fence.proxy.async.shared::cta;" ::: "memory"); }

#define R8(x, i) "=r"(x[i]), "=r"(x[i + 1]), "=r"(x[i + 2]), "=r"(x[i + 3]), "=r"(x[i + 4]), "=r"(x[i + 5]), "=r"(x[i + 6]), "=r"(x[i + 7])
#define W8(x, i) "r"(x[i]), "r"(x[i + 1]), "r"(x[i + 2]), "r"(x[i + 3]), "r"(x[i + 4]), "r"(x[i + 5]), "r"(x[i + 6]), "r"(x[i + 7])
// 32 columns of this thread's lane.
__device__ __forceinline__ void tmem_ld32(uint32_t (&x)[32], uint32_t addr) {
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x32.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16,%17,%18,%19,"
        "%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31}, [%32];"
        : R8(x, 0), R8(x, 8), R8(x, 16), R8(x, 24) : "r"(addr));
}
__device__ __forceinline__ void tmem_st32(uint32_t addr, const uint32_t (&x)[32]) {
    asm volatile(
        "tcgen05.st.sync.aligned.32x32b.x32.b32 [%32], {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16,%17,%18,"
        "%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31};"
        ::W8(x, 0), W8(x, 8), W8(x, 16), W8(x, 24), "r"(addr) : "memory");
}
__device__ __forceinline__ void tmem_st16(uint32_t addr, const uint32_t (&x)[16]) {
    asm volatile(
        "tcgen05.st.sync.aligned.32x32b.x16.b32 [%16], {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15};"
        ::W8(x, 0), W8(x, 8), "r"(addr) : "memory");
}
#undef R8
#undef W8

// The i-th run of N registers of an array.
template <int N, int K>
__device__ __forceinline__ uint32_t (&part(uint32_t (&x)[K], int i))[N] { return reinterpret_cast<uint32_t (&)[N]>(x[i * N]); }

// Shared-memory operand with 128-byte swizzle.  lead: byte stride between blocks of 64
// elements along the rows' contiguous direction (operands whose rows run along M or N only);
// groups of eight 128-byte rows are 1024 bytes apart.
__device__ __forceinline__ uint64_t operand(uint32_t addr, uint32_t lead) {
    return uint64_t((addr & 0x3ffff) >> 4) | uint64_t(lead >> 4) << 16 | uint64_t(1024 >> 4) << 32 | uint64_t(1) << 46 |
           uint64_t(2) << 61;
}
// Float32 accumulator, 128 rows, n columns; b_rows: B's rows run along N.
template <typename T>
constexpr uint32_t product(int n, bool b_rows) {
    const uint32_t f = sizeof(T) == 2 && std::is_same<T, __nv_bfloat16>::value ? 1u : 0u;
    return 1u << 4 | f << 7 | f << 10 | (b_rows ? 1u << 16 : 0u) | uint32_t(n / 8) << 17 | (128u / 16) << 24;
}
__device__ __forceinline__ void mma_smem(uint32_t d, uint64_t a, uint64_t b, uint32_t desc, bool add) {
    asm volatile("{ .reg .pred p; setp.ne.u32 p, %4, 0; tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p; }"
                 ::"r"(d), "l"(a), "l"(b), "r"(desc), "r"(uint32_t(add)) : "memory");
}
__device__ __forceinline__ void mma_tmem(uint32_t d, uint32_t a, uint64_t b, uint32_t desc, bool add) {
    asm volatile("{ .reg .pred p; setp.ne.u32 p, %4, 0; tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p; }"
                 ::"r"(d), "r"(a), "l"(b), "r"(desc), "r"(uint32_t(add)) : "memory");
}
// The barrier completes once every matrix instruction issued so far by this thread has.
__device__ __forceinline__ void mma_commit(uint32_t bar) {
    asm volatile("tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];" ::"r"(bar) : "memory");
}

// Byte offset of 16-byte chunk c of row r in a tile: blocks of 64 elements (128 bytes a row), chunks
// permuted by the row's index within eight.
__device__ __forceinline__ uint32_t tile_at(int r, int c) {
    return uint32_t((c >> 3) * (TK * 128) + r * 128 + (((c & 7) ^ (r & 7)) << 4));
}

// ------------------------------------------------------------------ the kernel

template <typename T, int D, bool SPLIT>
__global__ void __launch_bounds__(TNT, 1) prefix_tensor_kernel(const AttnArgs a) {
    using S = TensorSmem<D, SPLIT>;
    constexpr int ST = S::STAGES, DC = D / 8;
    constexpr int ROWS = SPLIT ? 128 : 256;
    extern __shared__ unsigned char raw[];
    const uint32_t base = (smem_u32(raw) + 1023) & ~1023u;
    unsigned char* mem = raw + (base - smem_u32(raw));
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    // barriers: full[ST], empty[ST], S[2], P[2], O[2]; the tensor memory's address, flags; the last barrier
    const uint32_t bars = base + S::BARS;
    const uint32_t full = bars, empty = bars + 8 * ST, sbar = bars + 16 * ST, pbar = sbar + 16, obar = sbar + 32, xbar = sbar + 64;
    volatile int* words = reinterpret_cast<volatile int*>(mem + S::BARS + 16 * ST + 48);
    volatile int* dead = words + 1;
    volatile int* poison = words + 2;
    grid_dependency_wait();
    allow_dependents();

    // ---- this CTA's queries and keys
    int item = blockIdx.x;
    const int tile = item % a.ptiles;
    item /= a.ptiles;
    const int head = item % a.Hkv, split = item / a.Hkv;
    const int2 gt = group_tile<ROWS>(a, tile, lane);
    if (gt.x < 0) return;
    const int b0 = group_begin(a, gt.x);
    const int per = a.Q * a.gs;
    const int M = (group_end(a, gt.x) - b0) * per, row0 = gt.y * ROWS;
    const int len = prefix_len(a, gt.x), step = range_len(len, a.SP);
    const int begin = split * step;
    if (begin >= len) return;
    const int end = min(len, begin + step);
    const int tiles = (end - begin + TK - 1) / TK;      // key tiles
    const int units = SPLIT ? tiles : 2 * tiles;         // (query tile, key tile) pairs: unit u is of tile u & 1
    const int* table = a.ptab + int64_t(gt.x) * a.pw;

    // Where each query row lies (and its part of the output goes), one thread per row.
    int64_t* q_off = reinterpret_cast<int64_t*>(mem + S::OFFS);
    int* o_row = reinterpret_cast<int*>(mem + S::OUTS);
    if (tid < ROWS) {
        const int g = row0 + tid;
        int64_t off = -1;
        int row = -1;
        if (g < M) {
            const int b = b0 + g / per, rem = g % per, qi = rem / a.gs, h = head * a.gs + rem % a.gs;
            off = b * a.qs[0] + qi * a.qs[1] + h * a.qs[2];
            row = (b * a.Q + qi) * a.Hq + h;
        }
        q_off[tid] = off;
        o_row[tid] = row;
    }
    if (tid == 0) {
        words[1] = 0, words[2] = 0;
        for (int i = 0; i < ST; ++i) bar_init(full + 8 * i, 128), bar_init(empty + 8 * i, 1);
        for (int i = 0; i < 2; ++i) bar_init(sbar + 8 * i, 1), bar_init(pbar + 8 * i, 128), bar_init(obar + 8 * i, 1);
        bar_init(xbar, 1);
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    }
    if (warp == 12) {
        asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], 512;" ::"r"(base + S::BARS + 16 * ST + 48) : "memory");
        asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
    }
    tmem_fence_before();
    __syncthreads();
    tmem_fence_after();
    const uint32_t tmem = uint32_t(words[0]);
    // columns: S of tile 0, S of tile 1, O of tile 0, O of tile 1
    const uint32_t s_at[2] = {tmem, tmem + 128}, o_at[2] = {tmem + 256, tmem + 256 + D};

    // Registers: 128 a thread at launch (512 threads); 176 for the softmax's two warpgroups and 80 for the
    // other two are the same total.
    if (warp >= 8 && warp < 12) {
        // ================================================ keys and values
        asm volatile("setmaxnreg.dec.sync.aligned.u32 80;");
        const int w = warp - 8;
        // Queries, in the group of copies before the first tile's.
#pragma unroll 4
        for (int i = tid - 256; i < ROWS * DC; i += 128) {
            const int r = i / DC, c = i % DC;
            const int64_t off = q_off[r];
            cp16(base + (r >> 7) * S::TILE + tile_at(r & 127, c), static_cast<const T*>(a.q) + (off < 0 ? 0 : off + c * 8), off >= 0);
        }
        cp_async_commit();
        asm volatile("bar.sync 2, 128;" ::: "memory");   // the addresses have been read
        // The page of this lane's key of tile t (32 keys a warp), -1 past the end, -2 for one that does not exist.
        auto page_of = [&](int t) {
            const int key = begin + t * TK + w * 32 + lane;
            if (t >= tiles || key >= end) return -1;
            const int page = table[a.page_shift >= 0 ? key >> a.page_shift : key / a.page_size];
            return page >= 0 && page < a.num_pages ? page : -2;
        };
        int count = 0;       // tiles of copies issued
        bool alive = true;
        auto hand_over = [&](int i) {   // copy tile i is there
            proxy_fence();
            bar_arrive(full + 8 * (i % ST));
        };
        auto load = [&](int t, bool value, int page) {
            if (!alive) return;
            const int st = count % ST;
            if (count >= ST && !__all_sync(FULL, bar_wait(empty + 8 * st, (count / ST - 1) & 1, dead))) {
                alive = false;
                return;
            }
            const int key = begin + t * TK + w * 32 + lane;
            const int64_t* str = value ? a.vc : a.kc;
            int64_t off = -1;
            if (page >= 0) {
                const int slot = a.page_shift >= 0 ? key & (a.page_size - 1) : key % a.page_size;
                off = page * str[0] + slot * str[1] + head * str[2];
            } else if (page == -2) {
                *poison = 1;
            }
            const T* src = static_cast<const T*>(value ? a.v : a.k);
            const uint32_t dst = base + S::KV + st * S::TILE;
            constexpr int RPI = 32 / DC;   // rows a warp copies at a time
#pragma unroll
            for (int i = 0; i < 32 / RPI; ++i) {
                const int r = i * RPI + lane / DC, c = lane % DC;
                const int64_t o = __shfl_sync(FULL, off, r);
                cp16(dst + tile_at(w * 32 + r, c), src + (o < 0 ? 0 : o + c * 8), o >= 0);
            }
            cp_async_commit();
            if (count >= LAG) {
                cp_async_wait<LAG>();
                hand_over(count - LAG);
            }
            ++count;
        };
        int pk = page_of(0);
        if (SPLIT) {
            // K0, K1, V0, K2, V1, K3, ...: the order in which the products first need them
            int p0 = pk, p1 = page_of(1);
            load(0, false, p0);
            if (tiles > 1) load(1, false, p1);
            for (int t = 0; t < tiles && alive; ++t) {
                const int p2 = page_of(t + 2);
                load(t, true, p0);
                if (t + 2 < tiles) load(t + 2, false, p2);
                p0 = p1, p1 = p2;
            }
        } else {
            for (int t = 0; t < tiles && alive; ++t) {
                const int next = page_of(t + 1);
                load(t, false, pk);
                load(t, true, pk);
                pk = next;
            }
        }
        cp_async_wait<0>();
        if (alive)
            for (int i = max(0, count - LAG); i < count; ++i) hand_over(i);
    } else if (warp >= 12) {
        // ================================================ matrix instructions
        asm volatile("setmaxnreg.dec.sync.aligned.u32 80;");
        if (warp == 12 && lane == 0) {
            constexpr uint32_t QK = product<T>(TK, false), PV = product<T>(D, true);
            int got = 0;      // copy tiles taken
            auto take = [&](int& st) {
                st = got % ST;
                const bool ok = bar_wait(full + 8 * st, (got / ST) & 1, dead);
                ++got;
                tmem_fence_after();
                return ok;
            };
            auto scores = [&](int t, int st) {
                const uint32_t q = base + (SPLIT ? 0 : t * S::TILE), k = base + S::KV + st * S::TILE;
#pragma unroll
                for (int i = 0; i < D / 16; ++i) {
                    const uint32_t at = (i >> 2) * (TK * 128) + (i & 3) * 32;
                    mma_smem(s_at[t], operand(q + at, 0), operand(k + at, 0), QK, i > 0);
                }
                mma_commit(sbar + 8 * t);
            };
            int kst = 0, vst = 0;
            bool ok = take(kst);
            if (ok) {
                scores(0, kst);
                if (SPLIT) {
                    mma_commit(empty + 8 * kst);
                    if (units > 1 && (ok = take(kst))) {
                        scores(1, kst);
                        mma_commit(empty + 8 * kst);
                    }
                } else {
                    scores(1, kst);
                    mma_commit(empty + 8 * kst);
                }
            }
            for (int u = 0; ok && u < units; ++u) {
                const int t = u & 1;
                if (SPLIT || t == 0) ok = take(vst);
                ok = ok && bar_wait(pbar + 8 * t, (u >> 1) & 1, dead);
                if (!ok) break;
                tmem_fence_after();
                const uint32_t v = base + S::KV + vst * S::TILE;
#pragma unroll
                for (int i = 0; i < TK / 16; ++i)
                    mma_tmem(o_at[t], s_at[t] + 8 * i, operand(v + i * 2048, TK * 128), PV, u > 1 || i > 0);
                if (SPLIT || t == 1) mma_commit(empty + 8 * vst);
                if (u + 2 < units) {
                    if (SPLIT || t == 0) ok = take(kst);
                    if (!ok) break;
                    scores(t, kst);
                    if (SPLIT || t == 1) mma_commit(empty + 8 * kst);
                } else {
                    mma_commit(obar + 8 * t);
                }
            }
            if (!ok) {   // what has been issued finishes before the tensor memory is freed
                *dead = 1;
                mma_commit(xbar);
                for (uint32_t i = 0; i < SPIN && !bar_try(xbar, 0); ++i) {}
            }
        }
        __syncwarp();
    } else {
        // ================================================ softmax
        asm volatile("setmaxnreg.inc.sync.aligned.u32 176;");
        const int t = warp >> 2, r = tid & 127;
        const uint32_t lanes = uint32_t(warp & 3) << 21;   // the warp's 32 lanes of tensor memory
        const int n = SPLIT ? (tiles + 1 - t) / 2 : tiles;
        float m = -INFINITY, l = 0.f;
        bool ok = true;
        for (int i = 0; i < n && ok; ++i) {
            const int valid = end - (begin + (SPLIT ? 2 * i + t : i) * TK);   // keys of this tile
            ok = __all_sync(FULL, bar_wait(sbar + 8 * t, i & 1, dead));
            if (!ok) break;
            tmem_fence_after();
            uint32_t x[TK];
#pragma unroll
            for (int c = 0; c < TK / 32; ++c) tmem_ld32(part<32>(x, c), s_at[t] + lanes + c * 32);
            tmem_wait_ld();
            float mul = a.scale;
            if (valid < TK) {   // scaled here, so that scores past the end are -infinity whatever the scale
                mul = 1.f;
#pragma unroll
                for (int e = 0; e < TK; ++e)
                    x[e] = e < valid ? __float_as_uint(__uint_as_float(x[e]) * a.scale) : 0xff800000u;
            }
            float mx = -INFINITY;
            if (mul < 0.f) {
#pragma unroll
                for (int e = 0; e < TK; ++e) mx = fmaxf(mx, -__uint_as_float(x[e]));
            } else {
                float m4[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
#pragma unroll
                for (int e = 0; e < TK; ++e) m4[e & 3] = fmaxf(m4[e & 3], __uint_as_float(x[e]));
                mx = fmaxf(fmaxf(m4[0], m4[1]), fmaxf(m4[2], m4[3]));
            }
            mx *= fabsf(mul);
            if (!(mx > -INFINITY)) mx = m;   // a scale of 0 times infinity, or nothing but NaN
            if (__any_sync(FULL, mx > m + 8.f)) {
                const float mn = fmaxf(m, mx);
                const float f = m == -INFINITY ? 0.f : exp2_fast(m - mn);
                m = mn;
                l *= f;
                if (i > 0) {
#pragma unroll
                    for (int c = 0; c < D / 32; ++c) {
                        uint32_t y[32];
                        tmem_ld32(y, o_at[t] + lanes + c * 32);
                        tmem_wait_ld();
#pragma unroll
                        for (int e = 0; e < 32; ++e) y[e] = __float_as_uint(__uint_as_float(y[e]) * f);
                        tmem_st32(o_at[t] + lanes + c * 32, y);
                    }
                }
            }
            const float ms = m == -INFINITY ? 0.f : m;
            float sum[2] = {0.f, 0.f};
#pragma unroll
            for (int e = 0; e < TK; e += 2) {
                float p0 = exp2_fast(fmaf(__uint_as_float(x[e]), mul, -ms));
                float p1 = exp2_fast(fmaf(__uint_as_float(x[e + 1]), mul, -ms));
                sum[0] += p0;
                sum[1] += p1;
                x[e / 2] = Mma<T>::pack(p0, p1);
            }
            l += sum[0] + sum[1];
            tmem_st32(s_at[t] + lanes, part<32>(x, 0));
            tmem_st32(s_at[t] + lanes + 32, part<32>(x, 1));
            tmem_wait_st();
            tmem_fence_before();
            bar_arrive(pbar + 8 * t);
        }
        // ---- this CTA's part
        if (ok && n > 0) ok = __all_sync(FULL, bar_wait(obar + 8 * t, 0, dead));
        // (the ring is written below: no product may read it any more)
        if (ok && units > 1) ok = __all_sync(FULL, bar_wait(obar + 8 * (1 - t), 0, dead));
        tmem_fence_after();
        const int64_t rows = int64_t(a.B) * a.Q * a.Hq;
        // joined with the other tile's through shared memory (the ring is done with)
        constexpr int PITCH = D + 4;
        float* other = reinterpret_cast<float*>(mem + S::KV);   // [128][PITCH], then maxima, sums (SPLIT); staged rows
        static_assert((SPLIT ? 128 * PITCH * 4 + 1024 : 256 * PITCH * 4) <= ST * S::TILE, "a tile's part fits in the ring");
        float f0 = 1.f, f1 = 0.f, ls = l;
        if (SPLIT && tiles > 1) {
            if (t == 1) {
                uint32_t x[32];
#pragma unroll
                for (int c = 0; c < D / 32; ++c) {
                    tmem_ld32(x, o_at[1] + lanes + c * 32);
                    tmem_wait_ld();
#pragma unroll
                    for (int e = 0; e < 32; e += 4)
                        *reinterpret_cast<uint4*>(other + r * PITCH + c * 32 + e) = make_uint4(x[e], x[e + 1], x[e + 2], x[e + 3]);
                }
                other[128 * PITCH + r] = m;
                other[128 * PITCH + 128 + r] = l;
            }
            asm volatile("bar.sync 1, 256;" ::: "memory");
            const float m1 = other[128 * PITCH + r], mj = fmaxf(m, m1), mz = mj == -INFINITY ? 0.f : mj;
            f0 = exp2_fast(m - mz), f1 = exp2_fast(m1 - mz);
            ls = l * f0 + other[128 * PITCH + 128 + r] * f1;
            m = mj;
        }
        if (!SPLIT || t == 0) {
            // (tensor memory is read by whole warps)
            const float bad = (*poison || !ok || *dead) ? __int_as_float(0x7fffffff) : 0.f;
            const float inv = (ls == 0.f ? 0.f : 1.f / ls) + bad;
            // Each warp's 32 rows through shared memory, so that a row is written as one line.
            float* mine = other + (SPLIT ? r : t * 128 + r) * PITCH;
#pragma unroll
            for (int c = 0; c < D / 32; ++c) {
                uint32_t x[32];
                tmem_ld32(x, o_at[t] + lanes + c * 32);
                tmem_wait_ld();
#pragma unroll
                for (int e = 0; e < 32; e += 4) {
                    float4 y = make_float4(__uint_as_float(x[e]), __uint_as_float(x[e + 1]), __uint_as_float(x[e + 2]),
                                           __uint_as_float(x[e + 3]));
                    float4* at = reinterpret_cast<float4*>(mine + c * 32 + e);
                    if (SPLIT && tiles > 1) {
                        const float4 z = *at;
                        y = make_float4(y.x * f0 + z.x * f1, y.y * f0 + z.y * f1, y.z * f0 + z.z * f1, y.w * f0 + z.w * f1);
                    }
                    *at = make_float4(y.x * inv, y.y * inv, y.z * inv, y.w * inv);
                }
            }
            const int own = o_row[SPLIT ? r : t * 128 + r];
            if (own >= 0) a.part_l[split * rows + own] = (ls == 0.f ? -INFINITY : m + log2f(ls)) + bad;
            __syncwarp();
            const float* first = mine - lane * PITCH;
#pragma unroll 4
            for (int i = 0; i < 32; ++i) {
                const int row = __shfl_sync(FULL, own, i);
                if (row < 0) break;
                if (lane < D / 4)
                    *reinterpret_cast<float4*>(a.part_o + (split * rows + row) * D + lane * 4) =
                        *reinterpret_cast<const float4*>(first + i * PITCH + lane * 4);
            }
        }
    }
    tmem_fence_before();
    __syncthreads();
    tmem_fence_after();
    if (warp == 12) asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, 512;" ::"r"(tmem) : "memory");
}

template <typename T, int D, bool SPLIT>
static fs_status launch(const AttnArgs& a, void* stream) {
    const void* fn = reinterpret_cast<const void*>(prefix_tensor_kernel<T, D, SPLIT>);
    const fs_status st = prepare_kernel(fn);
    if (st != FS_OK) return st;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(unsigned(int64_t(a.ptiles) * a.Hkv * a.SP), 1, 1);
    cfg.blockDim = dim3(TNT, 1, 1);
    cfg.dynamicSmemBytes = TensorSmem<D, SPLIT>::TOTAL;
    cfg.stream = static_cast<cudaStream_t>(stream);
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    const cudaError_t e = cudaLaunchKernelEx(&cfg, prefix_tensor_kernel<T, D, SPLIT>, a);
    return e == cudaSuccess ? FS_OK : cuda_fail(e);
}

template <typename T>
static fs_status launch_type(const AttnArgs& a, int head_dim, int tile, void* stream) {
    if (head_dim == 64) return tile == 128 ? launch<T, 64, true>(a, stream) : launch<T, 64, false>(a, stream);
    return tile == 128 ? launch<T, 128, true>(a, stream) : launch<T, 128, false>(a, stream);
}

fs_status launch_prefix_tensor(const AttnArgs& a, int dtype, int head_dim, int tile, void* stream) {
    return dtype == FS_BF16 ? launch_type<__nv_bfloat16>(a, head_dim, tile, stream)
                            : launch_type<__half>(a, head_dim, tile, stream);
}

}  // namespace fsd
