// Attention of chunks of new tokens on the 5th-generation tensor cores (sm_103a): requests with more query
// rows per key/value head than a tile of chunk_rows_kernel holds.
//
// A tile of up to 256 query rows (two tiles of 128) runs over its keys, 128 at a time:
//   S = Q K^T,  P = 2^(S - m),  O += P V.
// S, P and O live in tensor memory (S 128 x 128 float32 and O 128 x D for each of the two tiles, all
// of the 512 columns); S is turned into P (16 bits) in place, and P feeds the second product from there.
// Roles of the 16 warps:
//   warps 0-3, 4-7  softmax of tile 0 / tile 1, one thread per row: maximum, weights, sum; O is rescaled
//                   only when a maximum grows by more than 2^GROWTH; at the end the row's output
//   warps 8-11      keys and values: page look-ups and 16-byte asynchronous copies into a ring of
//                   swizzled tiles (any page size and strides)
//   warps 12, 13    issue the first and the second product
// While one tile's softmax runs, the tensor cores have the other tile's products. (Keys 128 at a time and
// not 64: the first product reads both operands from shared memory, at 64 keys 48 cycles an instruction of
// 32, at 128 as many as it takes.)
//
// One CTA per SM takes an equal run of units (key tiles) of the launch's line of work, see chunk_attention.cu; all
// roles walk the run's tiles at their own pace, so keys of the next tile are on their way while one is finished.
// Every wait on a barrier is bounded; one that runs out marks the CTA, which then drains its copies
// and products, frees its tensor memory and writes NaN.
#include "chunk.cuh"
#include "tensor_core.cuh"

namespace fsd {

constexpr int CM = 128;         // query rows of a tile of one warpgroup
constexpr int CK = 128;         // keys per tile
constexpr int CNT = 512;        // threads

template <int D>
struct ChunkTensorSmem {
    static constexpr int QTILE = CM * D * 2, TILE = CK * D * 2;
    static constexpr int STAGES = D == 128 ? 5 : 11;
    static constexpr int KV = 2 * QTILE;
    static constexpr int BARS = KV + STAGES * TILE;
    static constexpr int WORDS = BARS + 16 * STAGES + 12 * 8;
    static constexpr int TOTAL = WORDS + 32 + 1024;   // 1024: the base's alignment
};

// Two floats at a time.
__device__ __forceinline__ void fma_pair(float& x, float& y, float mul, float add) {
    asm("{ .reg .b64 a, b, c; mov.b64 a, {%0, %1}; mov.b64 b, {%2, %2}; mov.b64 c, {%3, %3};"
        " fma.rn.f32x2 a, a, b, c; mov.b64 {%0, %1}, a; }" : "+f"(x), "+f"(y) : "f"(mul), "f"(add));
}
__device__ __forceinline__ void add_pair(float& x, float& y, float a, float b) {
    asm("{ .reg .b64 a, b; mov.b64 a, {%0, %1}; mov.b64 b, {%2, %3}; add.rn.f32x2 a, a, b; mov.b64 {%0, %1}, a; }"
        : "+f"(x), "+f"(y) : "f"(a), "f"(b));
}

// ------------------------------------------------------------------ a run's tiles

// The part of a query tile that lies in a CTA's run: key tiles i0 .. i1 - 1 of one key/value head.
struct Segment {
    Request x;
    KeyTiles<CK> kt;
    int64_t end;            // the query tile's last unit, all heads, plus one
    int r, row0, head, i0, i1, M;
    __device__ __forceinline__ Segment(const ChunkArgs& a, int tile, int64_t unit, int64_t last)
        : Segment(a, a.t_items[tile], unit, last) {}
    __device__ __forceinline__ Segment(const ChunkArgs& a, int4 it, int64_t unit, int64_t last)
        : x(request(a, it.x)), kt(a, x.pos(a, it.y), x.pos(a, min(it.y + MANY, x.rows(a)) - 1)), r(it.x), row0(it.y), M(x.rows(a)) {
        const int64_t before = (int64_t(it.w) << 32 | uint32_t(it.z)) * a.Hkv, rel = unit - before;
        end = before + int64_t(kt.n) * a.Hkv;
        head = int(rel / kt.n);
        i0 = int(rel - int64_t(head) * kt.n);
        i1 = int(min(int64_t(kt.n), i0 + (last - unit)));
    }
    __device__ __forceinline__ int tiles() const { return i1 - i0; }
    __device__ __forceinline__ bool two() const { return M - row0 > CM; }   // rows for the second tile
    // Key tile of which some token of the query tile does not see all the keys that are loaded.
    __device__ __forceinline__ bool partial(const ChunkArgs& a, int k0) const {
        const int p_lo = x.pos(a, row0), p_hi = x.pos(a, min(row0 + MANY, M) - 1);
        return p_lo != p_hi && (k0 + CK > p_lo + 1 || (p_hi - k0 >= a.window && k0 + CK > a.sinks));
    }
};

// Copies of a segment of n key tiles, in the order in which the products need them: keys one tile ahead
// of values.  The key tile of copy c, negated (less one) for its values; and the inverse.
__device__ __forceinline__ int copy_of(int c, int n) {
    if (c == 0) return 0;
    if (c == 2 * n - 1) return -n;
    return c & 1 ? (c + 1) >> 1 : -(c >> 1);
}
__device__ __forceinline__ int keys_copy(int i) { return i == 0 ? 0 : 2 * i - 1; }
__device__ __forceinline__ int values_copy(int i, int n) { return i == n - 1 ? 2 * n - 1 : 2 * i + 2; }

// ------------------------------------------------------------------ the kernel

template <typename T, int D>
__global__ void __launch_bounds__(CNT, 1) chunk_tensor_kernel(const ChunkArgs a) {
    using S = ChunkTensorSmem<D>;
    using W = Weights<T>;
    constexpr int ST = S::STAGES, DC = D / 8;
    extern __shared__ unsigned char raw[];
    const uint32_t base = (smem_u32(raw) + 1023) & ~1023u;
    unsigned char* mem = raw + (base - smem_u32(raw));
    const int tid = threadIdx.x, warp = __shfl_sync(FULL, tid >> 5, 0), lane = tid & 31;
    // barriers: full[ST], empty[ST]; of each tile: queries there, scores there, weights there (in two
    // halves), product P V done; of each product, all done when a wait ran out.  Then the tensor memory's
    // address, a flag and, for four segments, whose values had infinities taken out
    const uint32_t full = base + S::BARS, empty = full + 8 * ST, qbar = empty + 8 * ST, sbar = qbar + 16, pbar = sbar + 16,
                   vbar = pbar + 32, xbar = vbar + 16;
    volatile int* words = reinterpret_cast<volatile int*>(mem + S::WORDS);
    volatile int* dead = words + 1;
    volatile int* odd = words + 2;      // [4]
    grid_dependency_wait();
    allow_dependents();

    // ---- this CTA's run of units
    const int n_tiles = a.t_plan[0];
    const int64_t total = (int64_t(a.t_plan[2]) << 32 | uint32_t(a.t_plan[1])) * a.Hkv;
    const int64_t run = max(int64_t(a.t_least), (total + a.t_grid - 1) / a.t_grid);
    const int64_t unit = min(blockIdx.x * run, total), last = min(unit + run, total);
    if (tid == 0) a.t_split[blockIdx.x] = make_int4(0, 0, 0, 0);
    if (unit >= last) return;
    for (int i = tid; i < n_tiles; i += CNT) {
        const int4 it = a.t_items[i];
        const int64_t before = (int64_t(it.w) << 32 | uint32_t(it.z)) * a.Hkv;
        int64_t next = total;
        if (i + 1 < n_tiles) {
            const int4 up = a.t_items[i + 1];
            next = (int64_t(up.w) << 32 | uint32_t(up.z)) * a.Hkv;
        }
        if (before <= unit && unit < next) words[6] = i;
    }
    if (warp == 13) {
        if (lane < ST) bar_init(full + 8 * lane, 1), bar_init(empty + 8 * lane, 1);
        if (lane < 2) bar_init(qbar + 8 * lane, 128), bar_init(sbar + 8 * lane, 1), bar_init(vbar + 8 * lane, 1), bar_init(xbar + 8 * lane, 1);
        if (lane < 4) bar_init(pbar + 8 * lane, 128), odd[lane] = 0;
        if (lane == 0) *dead = 0;
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    }
    if (warp == 12) {
        asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], 512;" ::"r"(base + S::WORDS) : "memory");
        asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
    }
    tmem_fence_before();
    __syncthreads();
    tmem_fence_after();
    const uint32_t tmem = __shfl_sync(FULL, uint32_t(words[0]), 0);
    int tile = __shfl_sync(FULL, words[6], 0);

    // Registers: 128 a thread at launch (512 threads); 200 for the softmax's two warpgroups and 56 for the
    // other two are the same total.
    if (warp >= 8 && warp < 12) {
        // ================================================ keys and values
        asm volatile("setmaxnreg.dec.sync.aligned.u32 56;");
        // Each warp copies every fourth tile: its waits, fence and look-ups cost one warp.
        const int w = warp - 8;
        uint32_t seq = 0;        // copies before the segment
        int before = -1;         // the stage of the copies that are still to be handed over
        int st = w;
        uint32_t lap = 0;
        bool ok = true;
        int segment = 0;
        bool check = false;      // the copies to be handed over are values that not every query sees: looked through
        int check_segment = 0;
        auto hand_over = [&]() {
            if (check) {
                unsigned char* tb = mem + S::KV + before * S::TILE;
                __syncwarp();
                bool any = false;
#pragma unroll 4
                for (int i = lane; i < CK * DC; i += 32) any |= odd_words<T>(*reinterpret_cast<const uint4*>(tb + i * 16));
                if (__any_sync(FULL, any)) {
                    for (int i = lane; i < CK * DC; i += 32) {
                        uint4* p = reinterpret_cast<uint4*>(tb + i * 16);
                        *p = even_words<T>(*p);
                    }
                    odd[check_segment & 3] = check_segment + 1;
                }
            }
            proxy_fence();
            __syncwarp();
            if (lane == 0) bar_arrive(full + 8 * before);
        };
#pragma unroll 1
        for (int64_t u = unit; u < last && ok; ++segment) {
            const Segment sg(a, tile, u, last);
            const int n = sg.tiles();
            const int* table = a.table + int64_t(sg.r) * a.width;
            // The page of a key; -1 for one that no query of the tile sees, -2 for one that does not exist.
            auto page_of = [&](int key) {
                if (!sg.kt.seen(key)) return -1;
                const int page = table[a.page_shift >= 0 ? key >> a.page_shift : key / a.page_size];
                return page >= 0 && page < a.num_pages ? page : -2;
            };
            auto first_key = [&](int c) {
                const int i = copy_of(c, n);
                return sg.kt.at(sg.i0 + (i < 0 ? -1 - i : i));
            };
            int pg[CK / 32];
            int c = int((w - seq) & 3);
            auto look_up = [&](int c) {
                if (c >= 2 * n) return;
                const int key = first_key(c) + lane;
#pragma unroll
                for (int h = 0; h < CK / 32; ++h) pg[h] = page_of(key + 32 * h);
            };
            look_up(c);
#pragma unroll 1
            for (; c < 2 * n; c += 4) {
                const bool value = copy_of(c, n) < 0;
                const int k0 = first_key(c);
                if (lap > 0) {
                    // (what this warp has copied may be what the stage waits for)
                    if (before >= 0 && !__all_sync(FULL, bar_test(empty + 8 * st, (lap - 1) & 1))) {
                        cp_async_wait<0>();
                        hand_over();
                        before = -1;
                    }
                    if (!__all_sync(FULL, bar_wait(empty + 8 * st, (lap - 1) & 1, dead))) {
                        ok = false;
                        break;
                    }
                }
                const int64_t* str = value ? a.vc : a.kc;
                const T* src = static_cast<const T*>(value ? a.v : a.k) + sg.head * str[2];
                const uint32_t dst = base + S::KV + st * S::TILE;
                bool missing = false;
#pragma unroll
                for (int h = 0; h < CK / 32; ++h) {
                    int64_t off = NOWHERE;
                    if (pg[h] >= 0) {
                        const int key = k0 + lane + 32 * h;
                        const int slot = a.page_shift >= 0 ? key & (a.page_size - 1) : key % a.page_size;
                        off = pg[h] * str[0] + slot * str[1];
                    }
                    missing |= pg[h] == -2;
                    // eight lanes a row: a 128-byte line of each block of 64 elements
#pragma unroll
                    for (int i = 0; i < 8; ++i) {
                        const int r = i * 4 + (lane >> 3), c8 = lane & 7;
                        const int64_t o = __shfl_sync(FULL, off, r);
                        const bool on = o != NOWHERE;
                        const T* from = src + (on ? o + c8 * 8 : 0);
#pragma unroll
                        for (int b = 0; b < D / 64; ++b) cp16(dst + tile_at<CK>(r + 32 * h, c8 + 8 * b), from + (on ? 64 * b : 0), on);
                    }
                }
                cp_async_commit();
                if (!value && __any_sync(FULL, missing)) {   // such keys are NaN, and so is every query that sees one
                    cp_async_wait<0>();
                    __syncwarp();
#pragma unroll
                    for (int h = 0; h < CK / 32; ++h)
                        if (pg[h] == -2)
                            for (int e = 0; e < DC; ++e)
                                *reinterpret_cast<uint4*>(mem + (dst - base) + tile_at<CK>(lane + 32 * h, e)) =
                                    make_uint4(0x7fff7fffu, 0x7fff7fffu, 0x7fff7fffu, 0x7fff7fffu);
                }
                look_up(c + 4);
                if (before >= 0) {
                    cp_async_wait<1>();
                    hand_over();
                }
                before = st;
                check = value && sg.partial(a, k0);
                check_segment = segment;
                st += 4;
                if (st >= ST) st -= ST, ++lap;
            }
            // Handed over before the next tile's lengths and pages are read.
            if (before >= 0) {
                cp_async_wait<0>();
                hand_over();
                before = -1;
            }
            seq += 2 * n;
            u += n;
            if (u >= sg.end) ++tile;
        }
        cp_async_wait<0>();
    } else if (warp >= 12) {
        // ================================================ matrix instructions
        asm volatile("setmaxnreg.dec.sync.aligned.u32 56;");
        // Two warps, one for each product.  A whole warp runs each loop, so that addresses and descriptors
        // stay in uniform registers; one elected lane issues.
        const bool lead = elect();
        if (warp == 12) {
            // ---- scores
            constexpr uint32_t QK = product<T>(CK, false);
            const uint32_t q_op = (base & 0x3ffff) >> 4, k_op = ((base + S::KV) & 0x3ffff) >> 4, hi = operand_high();
            bool ok = true;
            uint32_t seq = 0, segs[2] = {0, 0}, done[2] = {0, 0};   // copies; segments and products of each tile
#pragma unroll 1
            for (int64_t u = unit; u < last && ok;) {
                const Segment sg(a, tile, u, last);
                const int n = sg.tiles();
                const bool two = sg.two();
#pragma unroll 1
                for (int i = 0; i < n && ok; ++i) {
                    const uint32_t c = seq + keys_copy(i), lap = c / ST, kst = c - lap * ST;
                    ok = __all_sync(FULL, bar_wait(full + 8 * kst, lap & 1, dead));
#pragma unroll
                    for (int t = 0; t < 2; ++t) {
                        if (t == 1 && !two) break;
                        if (i == 0) ok = ok && __all_sync(FULL, bar_wait(qbar + 8 * t, segs[t]++ & 1, dead));
                        // the weights of the product before, in the same columns, have been read
                        if (done[t] > 0) ok = ok && __all_sync(FULL, bar_wait(vbar + 8 * t, (done[t] - 1) & 1, dead));
                        if (!ok) break;
                        ++done[t];
                        tmem_fence_after();
                        const uint32_t q = q_op + t * (S::QTILE >> 4), k = k_op + kst * (S::TILE >> 4);
#pragma unroll
                        for (int s = 0; s < D / 16; ++s)
                            mma_smem(lead, tmem + t * CK, q + (((s >> 2) * (CM * 128) + (s & 3) * 32) >> 4), 0,
                                     k + (((s >> 2) * (CK * 128) + (s & 3) * 32) >> 4), 0, hi, QK, s > 0);
                        mma_commit(lead, sbar + 8 * t);
                    }
                    if (ok) mma_commit(lead, empty + 8 * kst);
                }
                seq += 2 * n;
                u += n;
                if (u >= sg.end) ++tile;
            }
            if (!ok) {   // what has been issued finishes before the tensor memory is freed
                *dead = 1;
                mma_commit(lead, xbar + 0);
                for (uint32_t i = 0; i < SPIN && !bar_try(xbar + 0, 0); ++i) {}
            }
        } else if (warp == 13) {
            // ---- weights times values
            constexpr uint32_t PV = product<T>(D, true);
            const uint32_t v_op = ((base + S::KV) & 0x3ffff) >> 4, hi = operand_high();
            bool ok = true;
            uint32_t seq = 0, done[2] = {0, 0};
#pragma unroll 1
            for (int64_t u = unit; u < last && ok;) {
                const Segment sg(a, tile, u, last);
                const int n = sg.tiles();
                const bool two = sg.two();
#pragma unroll 1
                for (int i = 0; i < n && ok; ++i) {
                    const uint32_t c = seq + values_copy(i, n), lap = c / ST, vst = c - lap * ST;
                    ok = __all_sync(FULL, bar_wait(full + 8 * vst, lap & 1, dead));
                    const uint32_t v = v_op + vst * (S::TILE >> 4);
#pragma unroll
                    for (int t = 0; t < 2; ++t) {
                        if (t == 1 && !two) break;
                        const uint32_t p = tmem + t * CK, o = tmem + 2 * CK + t * D;
#pragma unroll
                        for (int h = 0; h < 2; ++h) {
                            ok = ok && __all_sync(FULL, bar_wait(pbar + 16 * t + 8 * h, done[t] & 1, dead));
                            if (!ok) break;
                            tmem_fence_after();
#pragma unroll
                            for (int s = 4 * h; s < 4 * h + 4; ++s)
                                mma_tmem(lead, o, p + 8 * s, v + s * (2048 >> 4), CK * 128, hi, PV, i > 0 || s > 0);
                        }
                        if (!ok) break;
                        ++done[t];
                        mma_commit(lead, vbar + 8 * t);
                    }
                    if (ok) mma_commit(lead, empty + 8 * vst);
                }
                seq += 2 * n;
                u += n;
                if (u >= sg.end) ++tile;
            }
            if (!ok) {   // what has been issued finishes before the tensor memory is freed
                *dead = 1;
                mma_commit(lead, xbar + 8);
                for (uint32_t i = 0; i < SPIN && !bar_try(xbar + 8, 0); ++i) {}
            }
        }
        __syncwarp();
    } else {
        // ================================================ softmax
        asm volatile("setmaxnreg.inc.sync.aligned.u32 200;");
        const int t = warp >> 2, r = tid & 127;
        const uint32_t lanes = uint32_t(warp & 3) << 21;   // the warp's 32 lanes of tensor memory
        const uint32_t sc = tmem + t * CK + lanes, oc = tmem + 2 * CK + t * D + lanes;
        bool ok = true;
        uint32_t done = 0;      // products of this tile
        int segment = 0;
#pragma unroll 1
        for (int64_t u = unit; u < last; ++segment) {
            float m = -INFINITY, l = 0.f;
            bool active;
            int n, pos, t_lo, t_hi, few, skip, i0;      // (no more than this stays in registers beside a row's scores)
            {
                const Segment sg(a, tile, u, last);
                n = sg.tiles();
                active = ok && (t == 0 || sg.two());
                few = sg.kt.few, skip = sg.kt.skip, i0 = sg.i0;
                pos = sg.x.pos(a, min(sg.row0 + t * CM + r, sg.M - 1));
                // positions of this tile's first and last token
                t_lo = sg.x.pos(a, sg.row0 + t * CM), t_hi = sg.x.pos(a, min(sg.row0 + (t + 1) * CM, sg.M) - 1);
                if (active) {
                    // The queries of this tile, by its 128 threads (the product that read the ones before is done).
#pragma unroll 4
                    for (int i = r; i < CM * DC; i += 128) {
                        const int q = i / DC, c = i % DC, qr = sg.row0 + t * CM + q;
                        const bool there = qr < sg.M;
                        const int j = there ? qr / a.gs : 0, h = sg.head * a.gs + (there ? qr % a.gs : 0);
                        cp16(base + t * S::QTILE + tile_at<CM>(q, c),
                             static_cast<const T*>(a.q) + (sg.x.q0 + j) * a.qs[0] + h * a.qs[1] + c * 8, there);
                    }
                    cp_async_commit();
                    cp_async_wait<0>();
                    proxy_fence();
                    bar_arrive(qbar + 8 * t);
                }
            }
            if (active) {
                bool huge = false;
#pragma unroll 1
                for (int i = 0; i < n; ++i) {
                    const int at = i0 + i, k0 = (at < few ? at : at - few + skip) * CK;
                    ok = __all_sync(FULL, bar_wait(sbar + 8 * t, done & 1, dead));
                    if (!ok) break;
                    ++done;
                    tmem_fence_after();
                    uint32_t x[CK];
#pragma unroll
                    for (int c = 0; c < CK / 32; ++c) tmem_ld32(part<32>(x, c), sc + c * 32);
                    tmem_wait_ld();
                    float mul = a.scale;
                    if (mul < 0.f) {
                        mul = -mul;
#pragma unroll
                        for (int e = 0; e < CK; ++e) x[e] ^= 0x80000000u;
                    }
                    // Scaled here where some keys are not seen, so that their scores are -infinity whatever the scale.
                    const bool edge = t_hi - k0 >= a.window;
                    if (k0 + CK > t_lo + 1 || edge) {
                        const int lim = pos + 1 - k0;
#pragma unroll
                        for (int e = 0; e < CK; ++e)
                            x[e] = e < lim ? __float_as_uint(__uint_as_float(x[e]) * mul) : 0xff800000u;
                        if (edge) {
                            const int low = pos - a.window + 1 - k0, few = a.sinks - k0;
#pragma unroll
                            for (int e = 0; e < CK; ++e)
                                if (e < low && e >= few) x[e] = 0xff800000u;
                        }
                        mul = 1.f;
                    }
                    float m4[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
#pragma unroll
                    for (int e = 0; e < CK; e += 2)
                        m4[(e >> 1) & 3] = fmaxf(m4[(e >> 1) & 3], fmaxf(__uint_as_float(x[e]), __uint_as_float(x[e + 1])));
                    float mx = fmaxf(fmaxf(m4[0], m4[1]), fmaxf(m4[2], m4[3])) * mul;
                    if (!(mx > -INFINITY)) mx = m;   // a scale of 0 times infinity, or nothing but NaN
                    if (__any_sync(FULL, mx - m > W::GROWTH)) {   // (the difference is exact where it decides)
                        const float mn = fmaxf(m, mx);
                        const float f = m == -INFINITY ? 0.f : exp2_fast(m - mn);
                        m = mn;
                        l *= f;
                        huge = __any_sync(FULL, fabsf(m) > 0x1p20f);
                        if (i > 0) {
                            // (the last product of this tile was done before these scores were begun)
#pragma unroll
                            for (int c = 0; c < D / 16; ++c) {
                                uint32_t y[16];
                                tmem_ld16(y, oc + c * 16);
                                tmem_wait_ld();
#pragma unroll
                                for (int e = 0; e < 16; ++e) y[e] = __float_as_uint(__uint_as_float(y[e]) * f);
                                tmem_st16(oc + c * 16, y);
                            }
                        }
                    }
                    const float ms = m == -INFINITY ? 0.f : m;
                    float off = W::SHIFT - ms;
                    // A maximum is a rounded product and a weight's exponent below is not: beyond 2^20 their difference, up
                    // to 2^-25 of the maximum, would count in the exponent (at 2^31 it is 2^6 and more).
                    if (huge) {
#pragma unroll
                        for (int e = 0; e < CK; ++e) x[e] = __float_as_uint(__fmul_rn(__uint_as_float(x[e]), mul) - ms);
                        mul = 1.f;
                        off = W::SHIFT;
                    }
                    float s0 = 0.f, s1 = 0.f;
#pragma unroll
                    for (int h = 0; h < 2; ++h) {
#pragma unroll
                        for (int e = 64 * h; e < 64 * h + 64; e += 2) {
                            float p0 = __uint_as_float(x[e]), p1 = __uint_as_float(x[e + 1]);
                            fma_pair(p0, p1, mul, off);
                            p0 = exp2_fast(p0), p1 = exp2_fast(p1);
                            add_pair(s0, s1, p0, p1);
                            x[e / 2] = Mma<T>::pack(p0, p1);
                        }
                        tmem_st32(sc + 32 * h, part<32>(x, h));
                        tmem_wait_st();
                        tmem_fence_before();
                        bar_arrive(pbar + 16 * t + 8 * h);
                    }
                    l += s0 + s1;
                }
                // ---- the row's output, once the last product is done
                ok = ok && __all_sync(FULL, bar_wait(vbar + 8 * t, (done - 1) & 1, dead));
                tmem_fence_after();
            }
            const Segment sg(a, tile, u, last);
            const int row = sg.row0 + t * CM + r;
            const bool on = row < sg.M;
            if (t == 0 || sg.two()) {
                const float bad = (!ok || *dead) ? __int_as_float(0x7fffffff) : 0.f;
                const float inv = (l == 0.f ? 0.f : 1.f / l) + bad;
                const float lse = (l == 0.f ? -INFINITY : m + (log2f(l) - W::SHIFT)) + bad;
                const bool whole = sg.i0 == 0 && sg.i1 == sg.kt.n;
                const bool fix = odd[segment & 3] == segment + 1;
                const int j = on ? row / a.gs : 0, h = sg.head * a.gs + (on ? row % a.gs : 0);
                T* out = static_cast<T*>(a.out) + (sg.x.q0 + j) * a.os[0] + h * a.os[1];
                const int64_t at = int64_t(2 * blockIdx.x + (sg.i0 == 0)) * MANY + t * CM + r;
#pragma unroll 1
                for (int c = 0; c < D / 32; ++c) {
                    uint32_t y[32];
                    tmem_ld32(y, oc + c * 32);
                    tmem_wait_ld();
#pragma unroll
                    for (int e = 0; e < 32; ++e) y[e] = __float_as_uint(__uint_as_float(y[e]) * inv);
                    if (on && fix) {   // (their weights are positive: exp(s - m) > 0)
                        for (int i = 0; i < n; ++i) {
                            const int k0 = sg.kt.at(sg.i0 + i);
                            if (!sg.partial(a, k0)) continue;
#pragma unroll
                            for (int e = 0; e < 32; e += 4) {
                                float4 z = make_float4(__uint_as_float(y[e]), __uint_as_float(y[e + 1]), __uint_as_float(y[e + 2]),
                                                       __uint_as_float(y[e + 3]));
                                add_odd<T>(a, a.table + int64_t(sg.r) * a.width, pos, k0, CK, sg.head, c * 32 + e, z);
                                y[e] = __float_as_uint(z.x), y[e + 1] = __float_as_uint(z.y);
                                y[e + 2] = __float_as_uint(z.z), y[e + 3] = __float_as_uint(z.w);
                            }
                        }
                    }
                    if (on && whole) {
                        auto two = [&](int e) { return Mma<T>::pack(__uint_as_float(y[e]), __uint_as_float(y[e + 1])); };
#pragma unroll
                        for (int e = 0; e < 32; e += 8)
                            *reinterpret_cast<uint4*>(out + c * 32 + e) = make_uint4(two(e), two(e + 2), two(e + 4), two(e + 6));
                    } else if (on) {
#pragma unroll
                        for (int e = 0; e < 32; e += 4)
                            *reinterpret_cast<uint4*>(a.t_part_o + at * D + c * 32 + e) = make_uint4(y[e], y[e + 1], y[e + 2], y[e + 3]);
                    }
                    __syncwarp();   // (tensor memory is read by whole warps)
                }
                if (on) {
                    if (!whole) a.t_part_l[at] = lse;
                    else if (a.lse) a.lse[int64_t(sg.x.q0 + j) * a.Hq + h] = lse * 0.693147180559945309f;
                }
                if (!whole && sg.i0 == 0 && tid == 0)   // this CTA has the tile's first part and says how many CTAs have one
                    a.t_split[blockIdx.x] = make_int4(sg.r, sg.head, sg.row0, int((u + sg.kt.n - 1) / run) - int(blockIdx.x) + 1);
                tmem_fence_before();   // the reads above, before the next product into the same columns
            }
            u += n;
            if (u >= sg.end) ++tile;
        }
    }
    tmem_fence_before();
    __syncthreads();
    tmem_fence_after();
    if (warp == 12) asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, 512;" ::"r"(tmem) : "memory");
}

template <typename T, int D>
static fs_status launch(const ChunkArgs& a, void* stream) {
    const void* fn = reinterpret_cast<const void*>(chunk_tensor_kernel<T, D>);
    const fs_status st = prepare_kernel(fn);
    if (st != FS_OK) return st;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(unsigned(a.t_grid), 1, 1);
    cfg.blockDim = dim3(CNT, 1, 1);
    cfg.dynamicSmemBytes = ChunkTensorSmem<D>::TOTAL;
    cfg.stream = static_cast<cudaStream_t>(stream);
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    const cudaError_t e = cudaLaunchKernelEx(&cfg, chunk_tensor_kernel<T, D>, a);
    return e == cudaSuccess ? FS_OK : cuda_fail(e);
}

fs_status launch_chunk_tensor(const ChunkArgs& a, int dtype, int head_dim, void* stream) {
    if (dtype == FS_BF16) return head_dim == 64 ? launch<__nv_bfloat16, 64>(a, stream) : launch<__nv_bfloat16, 128>(a, stream);
    return head_dim == 64 ? launch<__half, 64>(a, stream) : launch<__half, 128>(a, stream);
}

}  // namespace fsd
