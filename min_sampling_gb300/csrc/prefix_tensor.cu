// The shared prefix's part of attention on the 5th-generation tensor cores (sm_103a).
//
// One CTA per (query tile of a group, key/value head, range of keys).  The queries of all
// rows of a group that read one key/value head form the rows of two matrix products per
// tile of 64 keys: S = Q K^T, then O += P V with P = 2^(S - m).  S, P and O live in tensor
// memory: S (128 x 64 float32) is turned into P (16 bits) in place, and P feeds the second product from
// there.  Roles of the 16 warps:
//   warps 0-3, 4-7  softmax of tile 0 / tile 1, one thread per query: maximum, weights,
//                   sum; O is rescaled only when a maximum grows by more than 2^GROWTH, which P and the
//                   sum then exceed 1 by (exact in float32; for f16 see Weights)
//   warps 8-11      keys and values: page look-ups and 16-byte asynchronous copies into
//                   a ring of swizzled tiles (any page size and strides)
//   warps 12, 13    issue the first and the second product
// Two query tiles of 128 are in flight, each with two S, so that the next scores are there when
// a tile's softmax asks for them: the softmax warps never wait for a product of their own.
// (With one S of 128 keys per tile, softmax and the products behind it ran one after the other:
// 5300 cycles for 256 queries and 128 keys; now about 4000.)
//   SPLIT = false   256 queries, both tiles over the same keys
//   SPLIT = true    up to 128 queries, the tiles take alternate key tiles and are joined at
//                   the end
// Measured, 8 key/value heads of 128 in bf16: 1024 queries a head over 16384 keys 69 us, 993 TFLOP/s (128
// CTAs; bound by the first product, whose 64 keys take 48 cycles of shared-memory reads an instruction,
// and the tiles' hand-overs); 64 queries over 65537 keys 52 us, 5.2 TB/s (bound by the reads).
// Every wait on a barrier is bounded; one that runs out marks the CTA, which then drains
// its copies, frees its tensor memory and writes NaN.
#include "attention.cuh"
#include "tensor_core.cuh"

namespace fsd {

constexpr int TM = 128;          // queries per tile
constexpr int TK = 64;           // keys per tile
constexpr int TNT = 512;         // threads

template <int D, bool SPLIT>
struct TensorSmem {
    static constexpr int QTILE = TM * D * 2, TILE = TK * D * 2;  // a tile of queries; of keys or values
    static constexpr int NQ = SPLIT ? 1 : 2;
    static constexpr int STAGES = SPLIT ? 12 : 10;
    static constexpr int KV = NQ * QTILE;
    static constexpr int BARS = KV + STAGES * TILE;
    static constexpr int OUTS = BARS + 384;                  // the query rows' output rows
    static constexpr int OFFS = BARS - TILE;                 // their addresses, in the ring's last tile until it is loaded
    static constexpr int TOTAL = OUTS + NQ * TM * 4 + 1024;  // 1024: the base's alignment
};

// ------------------------------------------------------------------ the order of the copies

// Keys of the first units, then values and keys in turn: the order in which the products first
// need them.  AHEAD: key tiles before the first values.
template <bool SPLIT>
struct CopyOrder {
    static constexpr int AHEAD = SPLIT ? 4 : 2;
};
// The key tile of copy c of 2 tiles, negated (less one) for its values.
template <bool SPLIT>
__device__ __forceinline__ int copy_tile(int c, int tiles) {
    const int ka = min(CopyOrder<SPLIT>::AHEAD, tiles), both = 2 * (tiles - ka);
    if (c < ka) return c;
    c -= ka;
    if (c < both) return c & 1 ? (c >> 1) + ka : -1 - (c >> 1);
    return -1 - (c - both / 2);
}
// The inverse: the copies of keys and of values of tile t.
template <bool SPLIT>
__device__ __forceinline__ int copy_of_keys(int t, int tiles) {
    const int ka = min(CopyOrder<SPLIT>::AHEAD, tiles);
    return t < ka ? t : ka + 2 * (t - ka) + 1;
}
template <bool SPLIT>
__device__ __forceinline__ int copy_of_values(int t, int tiles) {
    const int ka = min(CopyOrder<SPLIT>::AHEAD, tiles);
    return ka + (t < tiles - ka ? 2 * t : t + tiles - ka);
}

// ------------------------------------------------------------------ the kernel

template <typename T, int D, bool SPLIT>
__global__ void __launch_bounds__(TNT, 1) prefix_tensor_kernel(const AttnArgs a) {
    using S = TensorSmem<D, SPLIT>;
    using W = Weights<T>;
    constexpr int ST = S::STAGES, DC = D / 8;
    constexpr int ROWS = SPLIT ? 128 : 256;
    extern __shared__ unsigned char raw[];
    const uint32_t base = (smem_u32(raw) + 1023) & ~1023u;
    unsigned char* mem = raw + (base - smem_u32(raw));
    const int tid = threadIdx.x, warp = __shfl_sync(FULL, tid >> 5, 0), lane = tid & 31;
    // barriers: full[ST], empty[ST]; of each S: scores there, weights there, product P V done; the
    // queries; every product done (twice); then the tensor memory's address and the flags
    const uint32_t bars = base + S::BARS;
    const uint32_t full = bars, empty = full + 8 * ST, sbar = empty + 8 * ST, pbar = sbar + 32, vbar = pbar + 32;
    const uint32_t qbar = vbar + 32, xbar = qbar + 8, ybar = xbar + 8;
    constexpr int WORDS = S::BARS + 16 * ST + 128;
    static_assert(16 * ST + 128 + 12 <= 384, "the barriers fit");
    volatile int* words = reinterpret_cast<volatile int*>(mem + WORDS);
    volatile int* dead = words + 1;
    volatile int* poison = words + 2;
    grid_dependency_wait();
    allow_dependents();

    // ---- this CTA's queries and keys
    int item = blockIdx.x;
    const int tile = item % a.ptiles;
    item /= a.ptiles;
    const int head = item % a.Hkv, split = item / a.Hkv;
    const GroupTile gt = group_tile<ROWS>(a, tile, lane);
    if (gt.g < 0) return;
    const int per = a.Q * a.gs;
    const int M = (gt.b1 - gt.b0) * per, row0 = gt.tile * ROWS;
    const int step = range_len(gt.len, a.SP);
    const int begin = split * step;
    if (begin >= gt.len) return;
    const int end = min(gt.len, begin + step);
    const int tiles = (end - begin + TK - 1) / TK;      // key tiles
    const int units = SPLIT ? tiles : 2 * tiles;         // (query tile, key tile) pairs: unit u is of tile u & 1
    const int* table = a.ptab + int64_t(gt.g) * a.pw;

    // Where each query row lies (and its part of the output goes), one thread per row.
    int64_t* q_off = reinterpret_cast<int64_t*>(mem + S::OFFS);
    int* o_row = reinterpret_cast<int*>(mem + S::OUTS);
    if (tid < ROWS) {
        const int g = row0 + tid;
        int64_t off = NOWHERE;
        int row = -1;
        if (g < M) {
            const int b = gt.b0 + g / per, rem = g % per, qi = rem / a.gs, h = head * a.gs + rem % a.gs;
            off = b * a.qs[0] + qi * a.qs[1] + h * a.qs[2];
            row = (b * a.Q + qi) * a.Hq + h;
        }
        q_off[tid] = off;
        o_row[tid] = row;
    }
    if (warp == 13) {
        if (lane < ST) bar_init(full + 8 * lane, 1), bar_init(empty + 8 * lane, 1);
        if (lane < 4) bar_init(sbar + 8 * lane, 1), bar_init(pbar + 8 * lane, 128), bar_init(vbar + 8 * lane, 1);
        if (lane == 0) {
            words[1] = 0, words[2] = 0;
            bar_init(qbar, 256);
            bar_init(xbar, 1);
            bar_init(ybar, 1);
        }
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    }
    if (warp == 12) {
        asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], 512;" ::"r"(base + WORDS) : "memory");
        asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
    }
    tmem_fence_before();
    __syncthreads();
    tmem_fence_after();
    const uint32_t tmem = __shfl_sync(FULL, uint32_t(words[0]), 0);
    // columns: S of units u % 4 (tile u % 2), O of tile 0, O of tile 1
    const uint32_t o_at[2] = {tmem + 4 * TK, tmem + 4 * TK + D};

    // Registers: 128 a thread at launch (512 threads); 160 for the softmax's two warpgroups and 96 for the
    // other two are the same total.
    if (warp >= 8 && warp < 12) {
        // ================================================ keys and values
        asm volatile("setmaxnreg.dec.sync.aligned.u32 96;");
        // Each warp copies every fourth tile: the waits, the fence and the look-ups of a tile then cost
        // one warp, not four.  (All four on every tile: 940 cycles a tile of 16 KB.)
        const int w = warp - 8;
        // The pages of this lane's keys of a tile: keys lane and lane + 32; -1 past the end, -2 for one
        // that does not exist.
        auto page_of = [&](int key) {
            if (key >= end) return -1;
            const int page = table[a.page_shift >= 0 ? key >> a.page_shift : key / a.page_size];
            return page >= 0 && page < a.num_pages ? page : -2;
        };
        auto keys_of = [&](int c) {
            const int x = copy_tile<SPLIT>(c, tiles);
            return begin + (x < 0 ? -1 - x : x) * TK + lane;
        };
        int pg[2] = {-1, -1};
        if (w < 2 * tiles) pg[0] = page_of(keys_of(w)), pg[1] = page_of(keys_of(w) + 32);
        asm volatile("bar.sync 2, 384;" ::: "memory");   // the queries' addresses, in the ring, have been read
        int before = -1;     // the stage of the copies that are still to be handed over
        auto hand_over = [&]() {
            proxy_fence();
            __syncwarp();
            if (lane == 0) bar_arrive(full + 8 * before);
        };
        int st = w;
        uint32_t lap = 0;
#pragma unroll 1
        for (int c = w; c < 2 * tiles; c += 4) {
            const bool value = copy_tile<SPLIT>(c, tiles) < 0;
            const int key = keys_of(c);
            if (lap > 0 && !__all_sync(FULL, bar_wait(empty + 8 * st, (lap - 1) & 1, dead))) break;
            const int64_t* str = value ? a.vc : a.kc;
            const T* src = static_cast<const T*>(value ? a.v : a.k) + head * str[2];
            int64_t off[2];
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                off[h] = NOWHERE;
                if (pg[h] >= 0) {
                    const int slot = a.page_shift >= 0 ? (key + 32 * h) & (a.page_size - 1) : (key + 32 * h) % a.page_size;
                    off[h] = pg[h] * str[0] + slot * str[1];
                } else if (pg[h] == -2) {
                    *poison = 1;
                }
            }
            const uint32_t dst = base + S::KV + st * S::TILE;
            // eight lanes a row: a 128-byte line of each block of 64 elements
#pragma unroll
            for (int i = 0; i < TK / 4; ++i) {
                const int r = i * 4 + (lane >> 3), c8 = lane & 7;
                const int64_t o = __shfl_sync(FULL, off[i >> 3], r & 31);
                const bool on = o != NOWHERE;
                const T* from = src + (on ? o + c8 * 8 : 0);
#pragma unroll
                for (int h = 0; h < D / 64; ++h) cp16(dst + tile_at<TK>(r, c8 + 8 * h), from + (on ? 64 * h : 0), on);
            }
            cp_async_commit();
            if (c + 4 < 2 * tiles) pg[0] = page_of(keys_of(c + 4)), pg[1] = page_of(keys_of(c + 4) + 32);
            if (before >= 0) {
                cp_async_wait<1>();
                hand_over();
            }
            before = st;
            st += 4;
            if (st >= ST) st -= ST, ++lap;
        }
        cp_async_wait<0>();
        if (before >= 0 && !*dead) hand_over();
    } else if (warp >= 12) {
        // ================================================ matrix instructions
        asm volatile("setmaxnreg.dec.sync.aligned.u32 96;");
        // Two warps, one for each product: a unit's waits, commits and instructions take one warp
        // about as long as its products run.  A whole warp runs each loop, so that addresses and descriptors
        // stay in uniform registers; one elected lane issues.  (With one lane in a branch of its own each
        // instruction took about 120 cycles to issue.)
        const bool lead = elect();
        if (warp == 12) {
            // ---- scores.  A key tile is taken by the first unit that needs it and given back by the last.
            constexpr uint32_t QK = product<T>(TK, false);
            const uint32_t q_op = (base & 0x3ffff) >> 4, k_op = ((base + S::KV) & 0x3ffff) >> 4, hi = operand_high();
            bool ok = __all_sync(FULL, bar_wait(qbar, 0, dead));
            uint32_t kst = 0;
#pragma unroll 1
            for (int u = 0; u < units; ++u) {
                const int t = u & 1, buf = u & 3;   // buffer: tile t, half u / 2 % 2
                if (SPLIT || t == 0) {
                    const uint32_t c = copy_of_keys<SPLIT>(SPLIT ? u : u >> 1, tiles), lap = c / ST;
                    kst = c - lap * ST;
                    ok = ok && __all_sync(FULL, bar_wait(full + 8 * kst, lap & 1, dead));
                }
                if (u >= 4) ok = ok && __all_sync(FULL, bar_wait(vbar + 8 * buf, ((u >> 2) - 1) & 1, dead));
                if (!ok) break;
                tmem_fence_after();
                const uint32_t q = q_op + (SPLIT ? 0 : t * (S::QTILE >> 4)), k = k_op + kst * (S::TILE >> 4);
                const uint32_t d = tmem + buf * TK;
#pragma unroll
                for (int i = 0; i < D / 16; ++i)
                    mma_smem(lead, d, q + (((i >> 2) * (TM * 128) + (i & 3) * 32) >> 4), 0,
                             k + (((i >> 2) * (TK * 128) + (i & 3) * 32) >> 4), 0, hi, QK, i > 0);
                mma_commit(lead, sbar + 8 * buf);
                if (SPLIT || t == 1) mma_commit(lead, empty + 8 * kst);
            }
            if (!ok) {   // what has been issued finishes before the tensor memory is freed
                *dead = 1;
                mma_commit(lead, ybar);
                bar_drain(ybar);
            }
        } else if (warp == 13) {
            // ---- weights times values
            constexpr uint32_t PV = product<T>(D, true);
            const uint32_t v_op = ((base + S::KV) & 0x3ffff) >> 4, hi = operand_high();
            bool ok = true;
            uint32_t vst = 0;
#pragma unroll 1
            for (int u = 0; u < units; ++u) {
                const int t = u & 1, buf = u & 3;
                if (SPLIT || t == 0) {
                    const uint32_t c = copy_of_values<SPLIT>(SPLIT ? u : u >> 1, tiles), lap = c / ST;
                    vst = c - lap * ST;
                    ok = ok && __all_sync(FULL, bar_wait(full + 8 * vst, lap & 1, dead));
                }
                ok = ok && __all_sync(FULL, bar_wait(pbar + 8 * buf, (u >> 2) & 1, dead));
                if (!ok) break;
                tmem_fence_after();
                const uint32_t v = v_op + vst * (S::TILE >> 4);
                const uint32_t p = tmem + buf * TK, o = tmem + 4 * TK + t * D;
                const bool add = u > 1;
#pragma unroll
                for (int i = 0; i < TK / 16; ++i) mma_tmem(lead, o, p + 8 * i, v + i * (2048 >> 4), TK * 128, hi, PV, add || i > 0);
                mma_commit(lead, vbar + 8 * buf);
                if (SPLIT || t == 1) mma_commit(lead, empty + 8 * vst);
            }
            mma_commit(lead, xbar);   // every product is done
            if (!ok) {
                *dead = 1;
                bar_drain(xbar);
            }
        }
        __syncwarp();
    } else {
        // ================================================ softmax
        asm volatile("setmaxnreg.inc.sync.aligned.u32 160;");
        // Queries first, by all 256 threads.
#pragma unroll 4
        for (int i = tid; i < ROWS * DC; i += 256) {
            const int r = i / DC, c = i % DC;
            const int64_t off = q_off[r];
            const bool on = off != NOWHERE;
            cp16(base + (r >> 7) * S::QTILE + tile_at<TM>(r & 127, c), static_cast<const T*>(a.q) + (on ? off + c * 8 : 0), on);
        }
        cp_async_commit();
        asm volatile("bar.sync 2, 384;" ::: "memory");   // the addresses have been read
        cp_async_wait<0>();
        proxy_fence();
        bar_arrive(qbar);

        const int t = warp >> 2, r = tid & 127;
        const uint32_t lanes = uint32_t(warp & 3) << 21;   // the warp's 32 lanes of tensor memory
        const int n = SPLIT ? (tiles + 1 - t) / 2 : tiles;
        float m = -INFINITY, l = 0.f;
        bool ok = true, huge = false;
#pragma unroll 1
        for (int i = 0; i < n && ok; ++i) {
            const int valid = end - (begin + (SPLIT ? 2 * i + t : i) * TK);   // keys of this tile
            const int buf = t + 2 * (i & 1);
            const uint32_t sc = tmem + buf * TK + lanes;
            ok = __all_sync(FULL, bar_wait(sbar + 8 * buf, (i >> 1) & 1, dead));
            if (!ok) break;
            tmem_fence_after();
            uint32_t x[TK];
#pragma unroll
            for (int c = 0; c < TK / 32; ++c) tmem_ld32(part<32>(x, c), sc + c * 32);
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
            if (__any_sync(FULL, mx - m > W::GROWTH)) {   // (the difference is exact where it decides; m + 8 may round to m)
                const float mn = fmaxf(m, mx);
                const float f = m == -INFINITY ? 0.f : exp2_fast(m - mn);
                m = mn;
                l *= f;
                huge = __any_sync(FULL, fabsf(m) > 0x1p20f);
                if (i > 0) {
                    // the last product of this tile (the one before was done before these scores were)
                    ok = __all_sync(FULL, bar_wait(vbar + 8 * (buf ^ 2), ((i - 1) >> 1) & 1, dead));
                    if (!ok) break;
                    tmem_fence_after();
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
            float off = W::SHIFT - ms;
            // A maximum is a rounded product and a weight's exponent below is not: beyond 2^20 their difference, up to
            // 2^-25 of the maximum, would count in the exponent (at 2^31 it is 2^6 and more).
            if (huge) {
#pragma unroll
                for (int e = 0; e < TK; ++e) x[e] = __float_as_uint(__fmul_rn(__uint_as_float(x[e]), mul) - ms);
                mul = 1.f;
                off = W::SHIFT;
            }
            float sum[2] = {0.f, 0.f};
#pragma unroll
            for (int e = 0; e < TK; e += 2) {
                float p0 = exp2_fast(fmaf(__uint_as_float(x[e]), mul, off));
                float p1 = exp2_fast(fmaf(__uint_as_float(x[e + 1]), mul, off));
                sum[0] += p0;
                sum[1] += p1;
                x[e / 2] = Mma<T>::pack(p0, p1);
            }
            l += sum[0] + sum[1];
            tmem_st32(sc, part<32>(x, 0));
            tmem_wait_st();
            tmem_fence_before();
            bar_arrive(pbar + 8 * buf);
        }
        // ---- this CTA's part, once every product of both tiles is done (the ring is written below)
        ok = ok && __all_sync(FULL, bar_wait(xbar, 0, dead));
        tmem_fence_after();
        const int64_t rows = int64_t(a.B) * a.Q * a.Hq;
        // SPLIT: joined with the other tile's through shared memory
        constexpr int PITCH = D + 4;
        float* other = reinterpret_cast<float*>(mem + S::KV);   // [128][PITCH], then maxima, sums (SPLIT); staged rows
        static_assert((SPLIT ? 128 * PITCH * 4 + 1024 : 256 * PITCH * 4) <= ST * S::TILE, "a tile's part fits in the ring");
        float f0 = 1.f, f1 = 0.f, ls = l;
        if (SPLIT && tiles > 1) {
            if (t == 1) {
#pragma unroll 1
                for (int c = 0; c < D / 32; ++c) {
                    uint32_t x[32];
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
            // Each row through shared memory, from where one bulk copy writes it.
            float* mine = other + (SPLIT ? r : t * 128 + r) * PITCH;
#pragma unroll 1
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
            if (own >= 0) {
                proxy_fence();
                asm volatile("cp.async.bulk.global.shared::cta.bulk_group [%0], [%1], %2;"
                             ::"l"(a.part_o + (split * rows + own) * D), "r"(smem_u32(mine)), "r"(D * 4) : "memory");
                asm volatile("cp.async.bulk.commit_group;" ::: "memory");
                a.part_l[split * rows + own] = (ls == 0.f ? -INFINITY : m + (log2f(ls) - W::SHIFT)) + bad;
                asm volatile("cp.async.bulk.wait_group 0;" ::: "memory");
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
