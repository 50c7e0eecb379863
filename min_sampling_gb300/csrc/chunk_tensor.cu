// Attention of chunks of new tokens on the 5th-generation tensor cores (sm_103a): requests with more query
// rows per key/value head than a tile of chunk_few_kernel holds.
//
// A tile of up to 256 query rows (two tiles of 128) runs over its keys, 128 at a time:
//   S = Q K^T,  P = 2^(S - m),  O += P V.
// S, P and O live in tensor memory (S 128 x 128 float32 and O 128 x D for each of the two tiles, all
// of the 512 columns; heads of 64 leave room for a third S, so that scores are there when a softmax asks for them: 2150 cycles
// for 256 rows and 128 keys, 2600 without); S is turned into P (16 bits) in place, and P feeds the second product from there.
// Roles of the 16 warps:
//   warps 0-3, 4-7  softmax of tile 0 / tile 1, one thread per row: maximum, weights, sum; O is rescaled
//                   only when a maximum grows by more than 2^GROWTH; at the end the row's output
//   warps 8, 9      keys, half a tile each; warps 10, 11 values: page look-ups and copies into a ring of swizzled tiles
//   warp 12         issues the products, PV and then the next S that goes into the same columns: in order, so that
//                   the weights have been read when the scores behind them are written
//   warp 13         looks values through that not every query sees, see below
//   warp 14         what the next tiles are, into a ring that all roles read
//   warp 15         queries of the next tile, as soon as the last product that reads the old ones is done
// While one tile's softmax runs, the tensor cores have the other tile's products. (Keys 128 at a time and
// not 64: the first product reads both operands from shared memory, at 64 keys 48 cycles an instruction of
// 32, at 128 as many as it takes.)
//
// Copies: see chunk_copy.cuh; without maps (GATHER = false) 16-byte asynchronous copies.
//
// A row's 128 scores are read once and stay in registers from the maximum to the weights.  What few tiles need
// (keys not seen, negative scales, huge scores) is done to the scores in tensor memory, in loops over 32 of them: unrolled
// between the maximum and the weights, it took as long in tiles that skip it (the maximum 570 cycles, now 260), for
// the instruction cache holds neither.  Of a tile's weights three quarters are announced first, so that the
// product that reads the last quarter is 128 cycles and not 256.
//
// Measured, bf16, 32 heads over 8 of 128: a prompt of 8190 tokens 420 to 426 us, 1.3 PFLOP/s, two thirds of the rate of the largest
// library product. For 256 rows and 128 keys the products take 2048 cycles, a tile's scores 1570 (load 330, maximum
// 260, weights 980) and then its products and the hand-overs, together 2860: that chain bounds it, and where 16-token
// pages are read by all SMs at once 400 cycles of waiting for keys and values.  Heads of 64: 2150 cycles, the weights', of two
// tiles at a time.  A tile's end (64 KB written by 256 threads, 32 bytes a store and clock) takes as long as t_start units.
//
// One CTA per SM takes an equal run of units (key tiles) of the launch's line of work, see many_run; all
// roles walk the run's tiles at their own pace, so keys of the next tile are on their way while one is finished.
// Every wait on a barrier is bounded; one that runs out marks the CTA, which then drains its copies
// and products, frees its tensor memory and writes NaN for all rows of its run.
#include "chunk_copy.cuh"

namespace fsd {

constexpr int CM = 128;         // query rows of a tile of one warpgroup
constexpr int CK = 128;         // keys per tile
constexpr int CNT = 512;        // threads
constexpr int ROLES = 8;        // the first warp that is not the softmax's
constexpr int AHEAD = 4;        // tiles that are described ahead

// The part of a query tile that lies in a CTA's run: n key tiles (0: no more), i0 on, of one key/value head.
struct Segment {
    int n, r, row0, head, i0, M;
    int whole, parts;           // all of the tile's keys; the CTAs that have a part of it (of its first part)
    Request x;
    KeyTiles<CK> kt;
    int p_lo, p_hi;             // positions of the first and last token
    __device__ __forceinline__ bool two() const { return M - row0 > CM; }   // rows for the second tile
    __device__ __forceinline__ bool partial(const ChunkArgs& a, int k0) const { return partial_keys(a, p_lo, p_hi, k0, CK); }
};

// A CTA's way along its run.  Warp-collective.
struct ManyLine {
    int r, row0;
    int64_t u, before;
    __device__ __forceinline__ explicit ManyLine(const ManyRun& run) : r(run.r), row0(run.row0), u(run.first), before(run.before) {}
    // The segment that the next unit lies in; n = 0: none.
    __device__ __forceinline__ Segment next(const ChunkArgs& a, const ManyRun& run, int cta, int lane) {
        const int64_t last = run.last;
        Segment sg;
        sg.n = 0;
        if (u >= last) return sg;
        sg.r = r, sg.row0 = row0;
        sg.x = request<true>(a, r);
        sg.M = sg.x.rows(a);
        const ManyTile tile(a, sg.x, row0);
        const int each = tile.units;
        sg.p_lo = tile.p_lo, sg.p_hi = tile.p_hi, sg.kt = tile.kt;
        sg.head = int((u - before) / each);
        const int64_t from = before + int64_t(sg.head) * each;     // of this head
        sg.i0 = tile.tiles(u - from);
        sg.n = tile.tiles(min(int64_t(each), last - from)) - sg.i0;
        sg.whole = sg.n == sg.kt.n;
        sg.parts = sg.whole || sg.i0 > 0 ? 0 : run.owner(from + each - 1) - cta + 1;
        u = min(from + each, last);
        if (u < last && u >= before + int64_t(each) * a.Hkv) {
            before += int64_t(each) * a.Hkv;
            row0 += MANY;
            if (row0 >= sg.M) {     // the next request with more than FEW rows
                row0 = 0;
                for (unsigned hit = 0; hit == 0;) {
                    const int k = r + 1 + lane;
                    hit = __ballot_sync(FULL, k < a.R && request<true>(a, min(k, a.R - 1)).rows(a) > a.rows_upto);
                    r += hit ? __ffs(int(hit)) : 32;
                    if (!hit && r >= a.R - 1) {     // (none is left: not with the lengths that the run was cut by)
                        u = last;
                        break;
                    }
                }
            }
        }
        // (a run that ends within a tile's start leaves all of it to the next)
        if (sg.n <= 0) sg.n = 0;
        return sg;
    }
};

template <int D>
struct ChunkTensorSmem {
    static constexpr int QTILE = CM * D * 2, TILE = CK * D * 2;
    static constexpr int STAGES = D == 128 ? 5 : 11;
    static constexpr int KV = 2 * QTILE;
    static constexpr int BARS = KV + STAGES * TILE;
    static constexpr int NBARS = 3 * STAGES + 22 + 2 * AHEAD;
    static constexpr int SEGS = BARS + NBARS * 8;
    static constexpr int WORDS = SEGS + AHEAD * int(sizeof(Segment));
    static constexpr int RUN = (WORDS + 160 + 7) / 8 * 8;
    static constexpr int TOTAL = RUN + int(sizeof(ManyRun));
    static_assert(TOTAL <= 227 * 1024, "shared memory");
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

template <int N> using Int = std::integral_constant<int, N>;
__device__ __forceinline__ void max3(float& m, float x, float y) {    // (NaN loses)
    asm("max.f32 %0, %0, %1, %2;" : "+f"(m) : "f"(x), "f"(y));
}

__device__ __forceinline__ void store32(void* p, const uint32_t (&x)[8]) {
    asm volatile("st.global.v8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};"
                 ::"l"(p), "r"(x[0]), "r"(x[1]), "r"(x[2]), "r"(x[3]), "r"(x[4]), "r"(x[5]), "r"(x[6]), "r"(x[7]) : "memory");
}

// Copies of a segment of n key tiles, in the order in which the products need them: keys one tile ahead
// of values.
__device__ __forceinline__ int keys_copy(int i) { return i == 0 ? 0 : 2 * i - 1; }
__device__ __forceinline__ int values_copy(int i, int n) { return i == n - 1 ? 2 * n - 1 : 2 * i + 2; }

// ------------------------------------------------------------------ the kernel

template <typename T, int D, bool GATHER>
__global__ void __launch_bounds__(CNT, 1) chunk_tensor_kernel(const __grid_constant__ ChunkArgs a, const __grid_constant__ ChunkMaps maps) {
    using S = ChunkTensorSmem<D>;
    using W = Weights<T>;
    constexpr int ST = S::STAGES, DC = D / 8;
    extern __shared__ __align__(1024) unsigned char mem[];
    const uint32_t base = smem_u32(mem);
    const int tid = threadIdx.x, warp = __shfl_sync(FULL, tid >> 5, 0), lane = tid & 31;
    // barriers: full[ST], empty[ST]; of each tile: queries there, queries done with, scores there [2], weights there
    // (in two parts) [2][2], product P V done [2]; of each product, all done when a wait ran out; landed, but still to be
    // looked through [ST]; segments there, done with [AHEAD].  (Two by turns where scores are two units ahead of a product.)  Then the segments, the tensor memory's address, a
    // flag, whose values had infinities taken out (four segments), which half key tiles miss pages (of sixteen tiles).
    const uint32_t full = base + S::BARS, empty = full + 8 * ST, qbar = empty + 8 * ST, qfree = qbar + 16, sbar = qfree + 16,
                   pbar = sbar + 32, vbar = pbar + 64, xbar = vbar + 32, land = xbar + 16, segbar = land + 8 * ST, segfree = segbar + 8 * AHEAD;
    volatile int* words = reinterpret_cast<volatile int*>(mem + S::WORDS);
    volatile int* dead = words + 1;
    volatile int* odd = words + 2;      // [4]
    volatile int* missing = words + 8;  // [16][2]
    Segment* segs = reinterpret_cast<Segment*>(mem + S::SEGS);
    // Heads of 64 leave room for a third S: the scores of unit c (2 i + t, key tile i of query tile t of a segment) lie in S
    // c % 3, and are written once the weights of unit c - 3 have been read: while the softmax of both tiles has work.
    // Heads of 128 have one S for each tile.
    constexpr bool DEEP = D == 64;
    auto s_col = [](uint32_t b) { return b == 2 ? 384u : b * CK; };   // O lies between the second and the third
    // of tile t's u-th key tile since the start: where its barriers are, and the parity to wait for
    auto turn = [](int t, uint32_t u) { return DEEP ? 2 * t + (u & 1) : uint32_t(t); };
    auto phase = [](uint32_t u) { return DEEP ? u >> 1 & 1 : u & 1; };
    // (set up while the launch before runs)
    if (warp == ROLES + 5) {
        if (lane < ST) bar_init(full + 8 * lane, 2), bar_init(empty + 8 * lane, 1), bar_init(land + 8 * lane, 2);
        if (lane < 2) bar_init(qbar + 8 * lane, 1), bar_init(qfree + 8 * lane, 1), bar_init(xbar + 8 * lane, 1);
        if (lane < 4) bar_init(sbar + 8 * lane, 1), bar_init(vbar + 8 * lane, 1);
        if (lane < 8) bar_init(pbar + 8 * lane, 128);
        // (a segment is read by four copying warps, the one that issues products, the one that looks values through, the
        // queries' and eight of the softmax)
        if (lane < AHEAD) odd[lane] = 0, bar_init(segbar + 8 * lane, 1), bar_init(segfree + 8 * lane, 15);
        if (lane == 0) *dead = 0;
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    }
    if (warp == ROLES + 4) {
        asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], 512;" ::"r"(base + S::WORDS) : "memory");
        asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
    }
    grid_dependency_wait();
    allow_dependents();

    // ---- this CTA's run of units (the ring's memory is free for the search: the fence orders it before the copies)
    const ManyRun& run = *reinterpret_cast<ManyRun*>(mem + S::RUN);
    const bool any = many_run<CNT>(a, int(blockIdx.x), reinterpret_cast<int64_t*>(mem + S::KV), *reinterpret_cast<ManyRun*>(mem + S::RUN));
    if (tid == 0) a.t_split[blockIdx.x] = make_int4(0, 0, 0, 0);
    proxy_fence();
    tmem_fence_before();
    __syncthreads();
    tmem_fence_after();
    const uint32_t tmem = __shfl_sync(FULL, uint32_t(words[0]), 0);
    if (!any) {
        if (warp == ROLES + 4) asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, 512;" ::"r"(tmem) : "memory");
        return;
    }

    // The s-th segment, once it is described; and given back, by each warp.
    auto next_segment = [&](uint32_t s, bool& ok) -> const Segment& {
        ok = ok && __all_sync(FULL, bar_wait(segbar + 8 * (s % AHEAD), (s / AHEAD) & 1, dead, a.patience));
        return segs[s % AHEAD];
    };
    auto give_back = [&](uint32_t s) {
        __syncwarp();
        if (lane == 0) bar_arrive(segfree + 8 * (s % AHEAD));
    };

    // Every role's end.  Copies that one which gave up has in flight land (a microsecond or two) before their memory is anyone
    // else's.
    auto all_done = [&]() {
        for (int i = 0; *dead && i < 1000; ++i) __nanosleep(1000);
        tmem_fence_before();
        asm volatile("bar.sync 1, %0;" ::"n"(CNT) : "memory");
        tmem_fence_after();
    };

    // Registers: 128 a thread at launch (512 threads); 200 for the softmax's two warpgroups and 56 for the other
    // two are the same total.
    if (warp >= ROLES) {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 56;");
    if (warp < ROLES + 4) {
        // ================================================ keys (two warps) and values (two), half a tile each
        const bool value = warp >= ROLES + 2;
        const int half = warp & 1, row = half * 64 + (lane & 15) * 4;
        const int64_t* str = value ? a.vc : a.kc;
        uint32_t seq = 0, unit = 0;   // copies and key tiles before the segment
        bool ok = true;
        for (uint32_t s = 0;; ++s) {
            const Segment& sg = next_segment(s, ok);
            if (!ok) break;
            const int n = sg.n, i0 = sg.i0, head = sg.head;
            if (n == 0) break;
            const KeyTiles<CK> kt = sg.kt;
            const int* table = a.table + int64_t(sg.r) * a.width;
            Pages pages;
            auto look_up = [&](int i) {
                if (i < n) pages.look_up<true>(a, table, kt.at(i0 + i) + row);
            };
            look_up(0);
#pragma unroll 1
            for (int i = 0; i < n; ++i) {
                const int k0 = kt.at(i0 + i);
                const uint32_t c = seq + (value ? values_copy(i, n) : keys_copy(i)), lap = c / ST, st = c - lap * ST;
                if (lap > 0 && !__all_sync(FULL, bar_wait(empty + 8 * st, (lap - 1) & 1, dead, a.patience))) {
                    ok = false;
                    break;
                }
                const bool gone = pages.resolve(a, kt, k0 + row);
                if (!value) {
                    const int any = __any_sync(FULL, gone);
                    if (lane == 0) missing[2 * ((unit + i) & 15) + half] = any;
                }
                const uint32_t dst = base + S::KV + st * S::TILE;
                // (values that not every query sees are looked through first)
                const uint32_t bar = (value && sg.partial(a, k0) ? land : full) + 8 * st;
                if (GATHER) {
                    if (lane == 0) bar_expect(bar, 64 * D * 2);
                    __syncwarp();
                    copy_rows<D>(a, value ? maps.v : maps.k, pages, k0 + half * 64, head, dst + half * 8192, CK * 128, bar, lane);
                } else {
                    const T* src = static_cast<const T*>(value ? a.v : a.k) + head * str[2];
#pragma unroll
                    for (int j = 0; j < 4; ++j) {
                        const int key = k0 + row + j, slot = a.page_shift >= 0 ? key & (a.page_size - 1) : key % a.page_size;
                        const int64_t off = pages.at[j] >= 0 ? pages.at[j] * str[0] + slot * str[1] : NOWHERE;
                        // four rows at a time (of quads 4 q .. 4 q + 3), eight lanes a 128-byte line
#pragma unroll
                        for (int q = 0; q < 4; ++q) {
                            const int from = q * 4 + (lane >> 3), r = half * 64 + from * 4 + j;
                            const int64_t o = __shfl_sync(FULL, off, from);
                            const bool on = o != NOWHERE;
#pragma unroll
                            for (int b = 0; b < D / 64; ++b)
                                cp16(dst + tile_at<CK>(r, (lane & 7) + 8 * b), src + (on ? o + (lane & 7) * 8 + 64 * b : 0), on);
                        }
                    }
                    cp_async_commit();
                    cp_async_wait<0>();
                }
                look_up(i + 1);
                if (!GATHER) {
                    proxy_fence();
                    __syncwarp();
                    if (lane == 0) bar_arrive(bar);
                }
            }
            if (!ok) break;
            seq += 2 * n;
            unit += n;
            give_back(s);
        }
        if (!ok) *dead = 1;
    } else if (warp == ROLES + 4) {
        // ================================================ products
        // (The whole warp runs the loop and one elected lane issues; lengths are made uniform by reductions, so that
        // operands and descriptors are computed in uniform registers.  Where the compiler cannot see that they
        // are, it moves every one over for every instruction: 80 cycles each, of the 64 that it takes.)
        const bool lead = elect();
        constexpr uint32_t QK = product<T>(CK, false), PV = product<T>(D, true);
        const uint32_t q_op = (base & 0x3ffff) >> 4, k_op = ((base + S::KV) & 0x3ffff) >> 4, hi = operand_high();
        const uint32_t tm = __reduce_max_sync(FULL, tmem);
        bool ok = true;
        uint32_t at = 0, lap = 0;       // the next copy's stage in the ring, and its parity
        uint32_t uses[2] = {0, 0}, made[2] = {0, 0}, done[2] = {0, 0};   // segments, modulo 2; key tiles' scores; products P V
        for (uint32_t s = 0;; ++s) {
            const Segment& sg = next_segment(s, ok);
            if (!ok) break;
            const uint32_t n = __reduce_max_sync(FULL, uint32_t(sg.n)), tiles = __reduce_max_sync(FULL, sg.two() ? 2u : 1u);
            if (n == 0) break;
            give_back(s);
            auto wait = [&](uint32_t bar, uint32_t parity) { ok = ok && __all_sync(FULL, bar_wait(bar, parity, dead, a.patience)); };
            auto scores = [&](bool last, int t, uint32_t st, uint32_t b) {
                const uint32_t q = q_op + t * (S::QTILE >> 4), k = k_op + st * (S::TILE >> 4);
#pragma unroll
                for (int d = 0; d < D / 16; ++d)
                    mma_smem(lead, tm + s_col(b), q + (((d >> 2) * (CM * 128) + (d & 3) * 32) >> 4), 0,
                             k + (((d >> 2) * (CK * 128) + (d & 3) * 32) >> 4), 0, hi, QK, d > 0);
                mma_commit(lead, sbar + 8 * turn(t, made[t]++));
                if (last) mma_commit(lead, qfree + 8 * t);
                if (t + 1 == int(tiles)) mma_commit(lead, empty + 8 * st);
            };
            auto weighted = [&](bool add, int t, uint32_t st, uint32_t b) {
                const uint32_t p = tm + s_col(b), o = tm + 2 * CK + t * D, v = k_op + st * (S::TILE >> 4);
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                    wait(pbar + 16 * turn(t, done[t]) + 8 * h, phase(done[t]));
                    tmem_fence_after();
                    if (ok) {
#pragma unroll
                        for (int k = 6 * h; k < 6 + 2 * h; ++k)
                            mma_tmem(lead, o, p + 8 * k, v + k * (2048 >> 4), CK * 128, hi, PV, add || k > 0);
                    }
                }
                if (DEEP) mma_commit(lead, vbar + 8 * turn(t, done[t]));
                ++done[t];
                if (t + 1 == int(tiles)) mma_commit(lead, empty + 8 * st);
            };
            auto forward = [&](uint32_t& pos, uint32_t& par) { par ^= pos + 1 == ST ? 1 : 0, pos = pos + 1 == ST ? 0 : pos + 1; };
            // (the segment before is done with the tiles' columns: its last weights have been issued for)
            wait(full + 8 * at, lap);
#pragma unroll
            for (int t = 0; t < 2; ++t)
                if (t < int(tiles)) {
                    wait(qbar + 8 * t, uses[t]);
                    uses[t] ^= 1;
                    tmem_fence_after();
                    if (ok) scores(n == 1, t, at, t);
                }
            forward(at, lap);
            if constexpr (DEEP) {
                uint32_t kst = 0, b = 0;    // the keys of the second tile's next scores; the S of this unit's first tile
                auto ahead = [&](uint32_t j, uint32_t b) {      // the first tile's scores of key tile j
                    if (j >= n) return;
                    kst = at;
                    wait(full + 8 * at, lap);
                    forward(at, lap);
                    tmem_fence_after();
                    if (ok) scores(j + 1 == n, 0, kst, b);
                };
                ahead(1, 2);
#pragma unroll 1
                for (uint32_t i = 0; i < n && ok; ++i) {
                    const uint32_t vst = at, b1 = b == 2 ? 0 : b + 1;
                    wait(full + 8 * vst, lap);
                    forward(at, lap);
                    weighted(i > 0, 0, vst, b);
                    if (tiles == 2) {
                        if (i + 1 < n && ok) scores(i + 2 == n, 1, kst, b);
                        weighted(i > 0, 1, vst, b1);
                    }
                    ahead(i + 2, b1);
                    b = b1 == 2 ? 0 : b1 + 1;
                }
            } else {
#pragma unroll 1
                for (uint32_t i = 0; i < n && ok; ++i) {
                    // the next keys, then these values; the last values alone
                    const bool more = i + 1 < n;
                    const uint32_t kst = at, kpar = lap;
                    if (more) forward(at, lap);
                    const uint32_t vst = at, vpar = lap;
                    forward(at, lap);
                    wait(full + 8 * vst, vpar);
                    weighted(i > 0, 0, vst, 0);
                    if (more) {
                        wait(full + 8 * kst, kpar);
                        tmem_fence_after();
                        if (ok) scores(i + 2 == n, 0, kst, 0);
                    } else {
                        mma_commit(lead, vbar);
                    }
                    if (tiles == 2) {
                        weighted(i > 0, 1, vst, 1);
                        if (more) {
                            if (ok) scores(i + 2 == n, 1, kst, 1);
                        } else {
                            mma_commit(lead, vbar + 8);
                        }
                    }
                }
            }
            if (!ok) break;
        }
        if (!ok) {   // what has been issued finishes before the tensor memory is freed
            *dead = 1;
            mma_commit(lead, xbar);
            bar_drain(xbar);
        }
        __syncwarp();
    } else if (warp == ROLES + 5) {
        // ================================================ values that not every query sees
        // A value that only some of the tokens see may be infinite or NaN, which a weight of zero does not cancel: such values
        // are taken out of the tile, and added at the end to the outputs of the queries that see them.
        uint32_t seq = 0, uses = 0;     // copies before the segment; each stage's parity
        bool ok = true;
        for (uint32_t s = 0;; ++s) {
            const Segment& sg = next_segment(s, ok);
            if (!ok || sg.n == 0) break;
            const int n = sg.n;
#pragma unroll 1
            for (int i = 0; i < n && ok; ++i) {
                if (!sg.partial(a, sg.kt.at(sg.i0 + i))) continue;
                const uint32_t st = (seq + values_copy(i, n)) % ST;
                ok = __all_sync(FULL, bar_wait(land + 8 * st, uses >> st & 1, dead, a.patience));
                if (!ok) break;
                uses ^= 1u << st;
                uint4* tile = reinterpret_cast<uint4*>(mem + S::KV + st * S::TILE);
                bool any = false;
#pragma unroll 8
                for (int e = lane; e < CK * DC; e += 32) any |= odd_words<T>(tile[e]);
                if (__any_sync(FULL, any)) {
                    for (int e = lane; e < CK * DC; e += 32) tile[e] = even_words<T>(tile[e]);
                    odd[s & 3] = int(s) + 1;
                }
                proxy_fence();
                __syncwarp();
                if (lane < 2) bar_arrive(full + 8 * st);
            }
            if (!ok) break;
            seq += 2 * n;
            give_back(s);
        }
        if (!ok) *dead = 1;
    } else if (warp == ROLES + 6) {
        // ================================================ what the next tiles are
        ManyLine line(run);
        bool ok = true;
        for (uint32_t s = 0; ok; ++s) {
            if (s >= AHEAD) ok = __all_sync(FULL, bar_wait_exactly(segfree + 8 * (s % AHEAD), (s / AHEAD - 1) & 1, dead, a.patience));
            if (!ok) break;
            const Segment sg = line.next(a, run, int(blockIdx.x), lane);
            if (lane == 0) segs[s % AHEAD] = sg;
            __syncwarp();
            if (lane == 0) bar_arrive(segbar + 8 * (s % AHEAD));
            if (sg.n == 0) break;
        }
        // A CTA that gave up: what has been written of its run's rows is not told apart from what has not.
        all_done();
        if (*dead) {
            line = ManyLine(run);
            for (Segment sg = line.next(a, run, int(blockIdx.x), lane); sg.n > 0; sg = line.next(a, run, int(blockIdx.x), lane))
                lost_tile<T, D, MANY>(a, sg, a.t_part_l, a.t_split, int(blockIdx.x), lane);
        }
        return;
    } else if (warp == ROLES + 7) {
        // ================================================ queries
        bool ok = true;
        uint32_t uses[2] = {0, 0};
        for (uint32_t s = 0;; ++s) {
            const Segment& sg = next_segment(s, ok);
            if (!ok || sg.n == 0) break;
#pragma unroll
            for (int t = 0; t < 2; ++t) {
                if (t == 1 && !sg.two()) break;
                if (uses[t] > 0) ok = ok && __all_sync(FULL, bar_wait(qfree + 8 * t, (uses[t] - 1) & 1, dead, a.patience));
                if (!ok) break;
                ++uses[t];
                const int row0 = sg.row0 + t * CM;
                if (GATHER && maps.qrows) {   // (rows behind the request's are computed, and not written)
                    if (lane == 0) {
                        bar_expect(qbar + 8 * t, CM * D * 2);
#pragma unroll
                        for (int b = 0; b < D / 64; ++b)
                            copy_box(base + t * S::QTILE + b * (CM * 128), &maps.q.boxes, b * 64, sg.head * a.gs, sg.x.q0 + row0 / a.gs,
                                     qbar + 8 * t);
                    }
                } else if (GATHER) {
                    int rows[4];
#pragma unroll
                    for (int j = 0; j < 4; ++j) {
                        const int row = row0 + lane * 4 + j, tok = row / a.gs;
                        rows[j] = row < sg.M ? (sg.x.q0 + tok) * maps.q.step[0] + (sg.head * a.gs + row - tok * a.gs) * maps.q.step[1] : -1;
                    }
                    if (lane == 0) bar_expect(qbar + 8 * t, CM * D * 2);
                    __syncwarp();
#pragma unroll
                    for (int b = 0; b < D / 64; ++b)
                        gather4(base + t * S::QTILE + b * (CM * 128) + lane * 512, &maps.q.rows, b * 64, rows, qbar + 8 * t);
                } else {
#pragma unroll 4
                    for (int i = lane; i < CM * DC; i += 32) {
                        const int q = i / DC, c = i % DC, row = row0 + q;
                        const bool there = row < sg.M;
                        const int tok = there ? row / a.gs : 0, h = sg.head * a.gs + (there ? row % a.gs : 0);
                        cp16(base + t * S::QTILE + tile_at<CM>(q, c),
                             static_cast<const T*>(a.q) + (sg.x.q0 + tok) * a.qs[0] + h * a.qs[1] + c * 8, there);
                    }
                    cp_async_commit();
                    cp_async_wait<0>();
                    proxy_fence();
                    __syncwarp();
                    if (lane == 0) bar_arrive(qbar + 8 * t);
                }
            }
            if (!ok) break;
            give_back(s);
        }
        if (!ok) *dead = 1;
    }
    } else {
        // ================================================ softmax
        asm volatile("setmaxnreg.inc.sync.aligned.u32 200;");
        const int t = warp >> 2, r = tid & 127;
        const uint32_t lanes = uint32_t(warp & 3) << 21;   // the warp's 32 lanes of tensor memory
        const uint32_t oc = tmem + 2 * CK + t * D + lanes;
        bool ok = true;
        uint32_t done = 0, unit = 0, ends = 0;      // scores of this tile; key tiles of segments before; segments of this tile
#pragma unroll 1
        for (uint32_t s = 0; ok; ++s) {
            const Segment& sg = next_segment(s, ok);
            if (!ok || sg.n == 0) break;
            const int n = sg.n, row = sg.row0 + t * CM + r;
            if (t == 0 || sg.two()) {
                const bool on = row < sg.M;
                const int pos = sg.x.pos(a, min(row, sg.M - 1));
                // positions of this tile's first and last token
                const int t_lo = sg.x.pos(a, sg.row0 + t * CM), t_hi = sg.x.pos(a, min(sg.row0 + (t + 1) * CM, sg.M) - 1);
                const int few = sg.kt.few, skip = sg.kt.skip, i0 = sg.i0;
                float m = -INFINITY, l = 0.f;
#pragma unroll 1
                for (int i = 0; i < n; ++i) {
                    const int at = i0 + i, k0 = (at < few ? at : at - few + skip) * CK;
                    const uint32_t turns = turn(t, done), sc = tmem + lanes + s_col(DEEP ? uint32_t(2 * i + t) % 3 : uint32_t(t));
                    ok = __all_sync(FULL, bar_wait(sbar + 8 * turns, phase(done), dead, a.patience));
                    if (!ok) break;
                    ++done;
                    tmem_fence_after();
                    float mul = a.scale;
                    const bool edge = t_hi - k0 >= a.window, gone = missing[2 * ((unit + i) & 15)] | missing[2 * ((unit + i) & 15) + 1];
                    const bool some = k0 + CK > t_lo + 1 || edge;   // not every row sees all of the keys
                    const int lim = pos + 1 - k0, low = edge ? pos - a.window + 1 - k0 : 0, first = a.sinks - k0;
                    if (some || gone || !(mul > 0.f)) {
                        // Scores of keys not seen become -infinity, whatever the scale; a key whose page does not exist is NaN.
                        // (In tensor memory, 32 at a time: unrolled over all the scores in registers, this code stood
                        // between the maximum's and the weights', and was as slow where it ran.)
                        const bool rare = gone || !(mul > 0.f);
                        const float f = rare ? mul : 1.f;
                        if (rare) mul = 1.f;
#pragma unroll 1
                        for (int c = 0; c < CK; c += 32) {
                            uint32_t x[32];
                            tmem_ld32(x, sc + c);
                            // the keys of these 32 that the row sees: below `lim`, and from `low` on or below `first`
                            auto below = [](int n) { return n <= 0 ? 0u : n >= 32 ? 0xffffffffu : (1u << n) - 1; };
                            const uint32_t see = below(lim - c) & (~below(low - c) | below(first - c));
                            const uint32_t lost = gone ? missing_pages<true>(a, sg.r, k0 + c) : 0u;
                            tmem_wait_ld();
                            keep32(x);
#pragma unroll
                            for (int e = 0; e < 32; ++e) x[e] = see >> e & 1 ? __float_as_uint(__uint_as_float(x[e]) * f) : 0xff800000u;
                            if (lost & see) {
#pragma unroll
                                for (int e = 0; e < 32; ++e)
                                    if (lost & see & 1u << e) x[e] = 0x7fffffffu;
                            }
                            tmem_st32(sc + c, x);
                        }
                        tmem_wait_st();
                    }
                    // The second half of the scores is on its way while the first half's maximum is taken.
                    uint32_t x[CK];
                    auto load = [&](int i) { tmem_ld32(part<32>(x, i), sc + 32 * i); };
                    load(0), load(1);
                    tmem_wait_ld();
                    load(2), load(3);
                    float m4[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
#pragma unroll
                    for (int e = 0; e < CK; e += 2) {
                        if (e == CK / 2) {
                            tmem_wait_ld();
                            keep32(part<32>(x, 2));
                            keep32(part<32>(x, 3));
                        }
                        max3(m4[(e >> 1) & 3], __uint_as_float(x[e]), __uint_as_float(x[e + 1]));
                    }
                    float mx = fmaxf(fmaxf(m4[0], m4[1]), fmaxf(m4[2], m4[3]));
                    mx *= mul;
                    // A scale of 0 times infinity, or nothing but NaN.  Rows behind the request's have the queries of whatever
                    // request comes next (with its outputs, where those are written over them): without a maximum they have no
                    // part in the votes below, which decide how the warp's other rows are rounded.
                    if (!on || !(mx > -INFINITY)) mx = m;
                    if (__any_sync(FULL, mx - m > W::GROWTH)) {   // (the difference is exact where it decides)
                        const float mn = fmaxf(m, mx);
                        const float f = m == -INFINITY ? 0.f : exp2_fast(m - mn);
                        m = mn;
                        l *= f;
                        if (i > 0) {
                            // (with one S the last product of this tile was done before these scores were begun)
                            if (DEEP) {
                                ok = __all_sync(FULL, bar_wait(vbar + 8 * turn(t, done), phase(done - 2), dead, a.patience));
                                if (!ok) break;
                                tmem_fence_after();
                            }
#pragma unroll 1
                            for (int c = 0; c < D; c += 16) {
                                uint32_t y[16];
                                tmem_ld16(y, oc + c);
                                tmem_wait_ld();
#pragma unroll
                                for (int e = 0; e < 16; ++e) y[e] = __float_as_uint(__uint_as_float(y[e]) * f);
                                tmem_st16(oc + c, y);
                            }
                        }
                    }
                    const float ms = m == -INFINITY ? 0.f : m;
                    float off = W::SHIFT - ms;
                    // A maximum is a rounded product and a weight's exponent below is not: beyond 2^20 their difference, up
                    // to 2^-25 of the maximum, would count in the exponent (at 2^31 it is 2^6 and more).
                    if (__any_sync(FULL, fabsf(m) > 0x1p20f && m > -INFINITY)) {
#pragma unroll 1
                        for (int c = 0; c < CK; c += 32) {
                            uint32_t y[32];
                            tmem_ld32(y, sc + c);
                            tmem_wait_ld();
#pragma unroll
                            for (int e = 0; e < 32; ++e) y[e] = __float_as_uint(__fmul_rn(__uint_as_float(y[e]), mul) - ms);
                            tmem_st32(sc + c, y);
                        }
                        tmem_wait_st();
                        load(0), load(1), load(2), load(3);
                        tmem_wait_ld();
                        mul = 1.f;
                        off = W::SHIFT;
                    }
                    // ---- weights
                    float s0 = 0.f, s1 = 0.f, s2 = 0.f, s3 = 0.f;
                    // (three quarters of them first: the products that read those are done when the last quarter is there)
                    auto weigh = [&](auto from, auto to) {
#pragma unroll
                        for (int e = from; e < to; e += 4) {
                            float p0 = __uint_as_float(x[e]), p1 = __uint_as_float(x[e + 1]), p2 = __uint_as_float(x[e + 2]),
                                  p3 = __uint_as_float(x[e + 3]);
                            fma_pair(p0, p1, mul, off);
                            fma_pair(p2, p3, mul, off);
                            p0 = exp2_fast(p0), p1 = exp2_fast(p1), p2 = exp2_fast(p2), p3 = exp2_fast(p3);
                            add_pair(s0, s1, p0, p1);
                            add_pair(s2, s3, p2, p3);
                            x[e / 2] = Mma<T>::pack(p0, p1);
                            x[e / 2 + 1] = Mma<T>::pack(p2, p3);
                        }
                    };
                    auto there = [&](int h) {
                        tmem_wait_st();
                        tmem_fence_before();
                        bar_arrive(pbar + 16 * turns + 8 * h);
                    };
                    weigh(Int<0>(), Int<96>());
                    tmem_st32(sc, part<32>(x, 0));
                    tmem_st16(sc + 32, part<16>(x, 2));
                    weigh(Int<96>(), Int<112>());
                    there(0);
                    weigh(Int<112>(), Int<128>());
                    tmem_st16(sc + 48, part<16>(x, 3));
                    there(1);
                    l += (s0 + s1) + (s2 + s3);
                }
                // ---- the row's output, once the last product is done
                const uint32_t end = DEEP ? done - 1 : ends++;
                ok = ok && __all_sync(FULL, bar_wait(vbar + 8 * turn(t, end), phase(end), dead, a.patience));
                if (!ok) break;
                tmem_fence_after();
                const float inv = l == 0.f ? 0.f : 1.f / l;
                const float lse = l == 0.f ? -INFINITY : m + (log2f(l) - W::SHIFT);
                const bool whole = sg.whole, fix = odd[s & 3] == int(s) + 1;
                const int j = on ? row / a.gs : 0, h = sg.head * a.gs + (on ? row - j * a.gs : 0);
                T* out = static_cast<T*>(a.out) + (sg.x.q0 + j) * a.os[0] + h * a.os[1];
                const int64_t slot = int64_t(2 * blockIdx.x + (i0 == 0)) * MANY + t * CM + r;
#pragma unroll 1
                for (int c = 0; c < D; c += 32) {
                    uint32_t y[32];
                    tmem_ld32(y, oc + c);
                    tmem_wait_ld();
#pragma unroll
                    for (int e = 0; e < 32; ++e) y[e] = __float_as_uint(__uint_as_float(y[e]) * inv);
                    if (on && fix) {   // (their weights are positive: exp(s - m) > 0)
                        for (int i = 0; i < n; ++i) {
                            const int k0 = sg.kt.at(i0 + i);
                            if (!sg.partial(a, k0)) continue;
#pragma unroll
                            for (int e = 0; e < 32; e += 4) {
                                float4 z = make_float4(__uint_as_float(y[e]), __uint_as_float(y[e + 1]), __uint_as_float(y[e + 2]),
                                                       __uint_as_float(y[e + 3]));
                                add_odd<T, true>(a, a.table + int64_t(sg.r) * a.width, pos, k0, CK, sg.head, c + e, z);
                                y[e] = __float_as_uint(z.x), y[e + 1] = __float_as_uint(z.y);
                                y[e + 2] = __float_as_uint(z.z), y[e + 3] = __float_as_uint(z.w);
                            }
                        }
                    }
                    // 32 bytes a store, a whole sector, where the rows are aligned to it: 64 KB of 16-byte stores take 4000 cycles.
                    if (on && whole) {
                        auto two = [&](int e) { return Mma<T>::pack(__uint_as_float(y[e]), __uint_as_float(y[e + 1])); };
#pragma unroll
                        for (int e = 0; e < 32; e += 2) y[e / 2] = two(e);
                        if (a.out_32) {
                            store32(out + c, part<8>(y, 0));
                            store32(out + c + 16, part<8>(y, 1));
                        } else {
#pragma unroll
                            for (int e = 0; e < 16; e += 4) *reinterpret_cast<uint4*>(out + c + 2 * e) = make_uint4(y[e], y[e + 1], y[e + 2], y[e + 3]);
                        }
                    } else if (on) {
#pragma unroll
                        for (int e = 0; e < 4; ++e) store32(a.t_part_o + slot * D + c + 8 * e, part<8>(y, e));
                    }
                    __syncwarp();   // (tensor memory is read by whole warps)
                }
                if (on) {
                    if (!whole) a.t_part_l[slot] = make_float2(m, l * exp2f(-W::SHIFT));
                    else if (a.lse) a.lse[int64_t(sg.x.q0 + j) * a.Hq + h] = lse * 0.693147180559945309f;
                }
                // The CTA that has a tile's first part says how many CTAs have one.
                if (sg.parts > 0 && tid == 0) a.t_split[blockIdx.x] = make_int4(sg.r, sg.head, sg.row0, sg.parts);
                tmem_fence_before();   // the reads above, before the next product into the same columns
            }
            unit += n;
            give_back(s);
        }
    }
    all_done();
    if (warp == ROLES + 4) asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, 512;" ::"r"(tmem) : "memory");
}

// ------------------------------------------------------------------ host

template <typename T, int D, bool GATHER>
static fs_status launch(const ChunkArgs& a, const ChunkMaps& maps, void* stream) {
    const fs_status st = prepare_kernel(reinterpret_cast<const void*>(chunk_tensor_kernel<T, D, GATHER>));
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
    const cudaError_t e = cudaLaunchKernelEx(&cfg, chunk_tensor_kernel<T, D, GATHER>, a, maps);
    return e == cudaSuccess ? FS_OK : cuda_fail(e);
}

template <typename T>
static fs_status launch_type(const ChunkArgs& a, const ChunkMaps* maps, int head_dim, void* stream) {
    static const ChunkMaps none = {};
    if (maps) return head_dim == 64 ? launch<T, 64, true>(a, *maps, stream) : launch<T, 128, true>(a, *maps, stream);
    return head_dim == 64 ? launch<T, 64, false>(a, none, stream) : launch<T, 128, false>(a, none, stream);
}

fs_status launch_chunk_tensor(const ChunkArgs& a, const ChunkMaps* maps, int dtype, int head_dim, void* stream) {
    return dtype == FS_BF16 ? launch_type<__nv_bfloat16>(a, maps, head_dim, stream) : launch_type<__half>(a, maps, head_dim, stream);
}

}  // namespace fsd
