// Attention of single tokens, and of a few, over a paged cache (sm_103a): requests of up to 16 query rows per
// key/value head.
//
// Bound by the reads of keys and values.  One warp describes the run's tiles and copies them, 64 keys and their values at
// a time, into a ring that is as deep as shared memory allows (two CTAs on an SM, 192 KB on their way); four
// warps take 16 of the 64 keys each (mma.sync) with a running maximum, sum and output of their own, joined at the
// tile's end.  Nothing but the ring's barriers ties them together, so the reads go on over the ends of tiles and
// requests.  64 requests of up to 8192 tokens, 8 heads of 128: 175 us, 6.2 TB/s (with copies by the four
// warps themselves, a tile ahead and a barrier each, 250 us).
// Every wait on a barrier is bounded; one that runs out marks the CTA, which then writes NaN for all rows of its run.
#include "chunk_copy.cuh"

#include "fragments.cuh"

namespace fsd {

constexpr int FK = 64;          // keys per tile
constexpr int FNT = 160;        // threads
constexpr int FAHEAD = 2;       // tiles that are described ahead

// The part of a tile that lies in a CTA's run: n key tiles (0: no more), i0 on, of one key/value head.
struct FewSegment {
    int n, r, row0, head, i0, M;
    int whole, parts;           // all of the tile's keys; the CTAs that have a part of it (of its first part)
    Request x;
    KeyTiles<FK> kt;
    int p_lo, p_hi;             // positions of the first and last token
};

// A CTA's way along its run.
struct FewLine {
    Place pl;
    Request x;
    int64_t unit;
    __device__ __forceinline__ FewLine(const ChunkArgs& a, const Run& run) : pl(run.place), x{}, unit(run.first) {
        if (run.first < run.last) x = request<false>(a, pl.r);     // (there may be no requests at all)
    }
    // The segment that the next unit lies in; n = 0: none.
    __device__ __forceinline__ FewSegment next(const ChunkArgs& a, const Run& run, int cta) {
        FewSegment sg;
        sg.n = 0;
        if (unit >= run.last) return sg;
        while (unit >= pl.before + pl.units * a.Hkv) {
            pl.before += pl.units * a.Hkv;
            x = request<false>(a, ++pl.r);
            pl.units = units_of<FEW, FK>(a, x);
        }
        sg.r = pl.r, sg.x = x;
        sg.head = int((unit - pl.before) / pl.units);
        sg.M = x.rows(a);
        int64_t from = pl.before + int64_t(sg.head) * pl.units;   // the tile's first unit
        sg.row0 = 0;
        for (;; from += sg.kt.n + FEW_START, sg.row0 += FEW) {
            sg.p_lo = x.pos(a, sg.row0), sg.p_hi = x.pos(a, min(sg.row0 + FEW, sg.M) - 1);
            sg.kt = KeyTiles<FK>(a, sg.p_lo, sg.p_hi);
            if (unit < from + sg.kt.n + FEW_START) break;
        }
        const int each = sg.kt.n + FEW_START;
        sg.i0 = int(max(unit - from - FEW_START, int64_t(0)));
        sg.n = max(int(min(int64_t(each), run.last - from)) - FEW_START - sg.i0, 0);
        sg.whole = sg.n == sg.kt.n;
        sg.parts = sg.whole || sg.i0 > 0 ? 0 : int((from + each - 1) / run.length) - cta + 1;
        unit = min(from + each, run.last);
        return sg;      // (a run that ends within a tile's FEW_START leaves all of it to the next)
    }
};

template <int D>
struct FewSmem {
    static constexpr int TILE = FK * D * 2;
    static constexpr int STAGES = D == 64 ? 6 : 3;
    static constexpr int QTILE = FEW * D * 2;
    static constexpr int Q = STAGES * 2 * TILE;                 // [FAHEAD]
    static constexpr int MERGE = Q + FAHEAD * QTILE;            // [4 warps][4 rows][D] float32
    static constexpr int STATS = MERGE + 16 * D * 4;            // [4 warps][FEW] maxima, then sums
    static constexpr int BARS = STATS + 4 * FEW * 8;
    static constexpr int NBARS = 2 * STAGES + 3 * FAHEAD;
    static constexpr int SEGS = BARS + NBARS * 8;
    static constexpr int WORDS = SEGS + FAHEAD * int(sizeof(FewSegment));   // flag, the warps' flags [4], pages missing [STAGES]
    static constexpr int TOTAL = (WORDS + 20 + STAGES * 4 + 7) / 8 * 8;
    static_assert(D == 256 ? TOTAL <= 227 * 1024 : TOTAL <= 113 * 1024, "one or two CTAs on an SM");
};

template <typename T, int D>
__global__ void __launch_bounds__(FNT) chunk_few_kernel(const __grid_constant__ ChunkArgs a, const __grid_constant__ ChunkMaps maps) {
    using S = FewSmem<D>;
    constexpr int ST = S::STAGES, DC = D / 8;
    constexpr float UP = std::is_same<T, __half>::value ? 32768.f : 1.f;   // the weights' factor in the product
    extern __shared__ __align__(1024) unsigned char mem[];
    const uint32_t base = smem_u32(mem);
    const int tid = threadIdx.x, warp = __shfl_sync(FULL, tid >> 5, 0), lane = tid & 31;
    // barriers: full[ST], empty[ST]; queries there, segments there, done with [FAHEAD]
    const uint32_t full = base + S::BARS, empty = full + 8 * ST, qbar = empty + 8 * ST, segbar = qbar + 8 * FAHEAD,
                   segfree = segbar + 8 * FAHEAD;
    FewSegment* segs = reinterpret_cast<FewSegment*>(mem + S::SEGS);
    volatile int* dead = reinterpret_cast<volatile int*>(mem + S::WORDS);
    volatile int* gone = dead + 1;      // [4], a warp whose wait ran out
    volatile int* missing = dead + 5;   // [ST]
    int64_t* words = reinterpret_cast<int64_t*>(mem + S::MERGE);     // while the run is looked up
    const int cta = int(blockIdx.x);
    if (!few_starts(a)) return;
    const Run run = run_of<FNT, FEW, FK>(a, cta, words);
    if (tid == 0) {
        a.split[cta] = make_int4(0, 0, 0, 0);
        for (int i = 0; i < ST; ++i) bar_init(full + 8 * i, 1), bar_init(empty + 8 * i, 4);
        for (int i = 0; i < FAHEAD; ++i) bar_init(qbar + 8 * i, 1), bar_init(segbar + 8 * i, 1), bar_init(segfree + 8 * i, 4);
        *dead = 0;
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    }
    if (a.zero_rest) zero_rest<T, D>(a, cta, FNT);
    __syncthreads();

    // Every role's end.  Copies that one which gave up has in flight land (a microsecond or two) before their memory is anyone
    // else's.
    auto all_done = [&]() {
        for (int i = 0; *dead && i < 1000; ++i) __nanosleep(1000);
        asm volatile("bar.sync 2, %0;" ::"n"(FNT) : "memory");
    };
    if (warp == 4) {
        // ================================================ what the next tiles are, and their copies
        FewLine line(a, run);
        uint32_t c = 0;         // key tiles before
        bool ok = true;
        for (uint32_t s = 0;; ++s) {
            const uint32_t slot = s % FAHEAD;
            if (s >= FAHEAD) ok = __all_sync(FULL, bar_wait_exactly(segfree + 8 * slot, (s / FAHEAD - 1) & 1, dead, a.patience));
            if (!ok) break;
            const FewSegment sg = line.next(a, run, cta);
            if (lane == 0) segs[slot] = sg;
            if (sg.n > 0) {
                // queries: rows 4 q .. 4 q + 3 by lane (q, block)
                int rows[4];
                const int q = lane & 3, b = lane >> 2;
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    const int row = sg.row0 + q * 4 + j, tok = row / a.gs;
                    rows[j] = row < sg.M ? (sg.x.q0 + tok) * maps.q.step[0] + (sg.head * a.gs + row - tok * a.gs) * maps.q.step[1] : -1;
                }
                if (lane == 0) bar_expect(qbar + 8 * slot, S::QTILE);
                __syncwarp();
                if (b < D / 64) gather4(base + S::Q + slot * S::QTILE + b * (FEW * 128) + q * 512, &maps.q.rows, b * 64, rows, qbar + 8 * slot);
            }
            __syncwarp();
            if (lane == 0) bar_arrive(segbar + 8 * slot);
            if (sg.n == 0) break;
            const int* table = a.table + int64_t(sg.r) * a.width;
            Pages pages;
            const int row = (lane & 15) * 4;
            pages.look_up<false>(a, table, sg.kt.at(sg.i0) + row);
#pragma unroll 1
            for (int i = 0; i < sg.n; ++i, ++c) {
                const uint32_t lap = c / ST, st = c - lap * ST;
                const int k0 = sg.kt.at(sg.i0 + i);
                Pages now = pages;
                if (i + 1 < sg.n) pages.look_up<false>(a, table, sg.kt.at(sg.i0 + i + 1) + row);
                if (lap > 0) ok = __all_sync(FULL, bar_wait(empty + 8 * st, (lap - 1) & 1, dead, a.patience));
                if (!ok) break;
                const int any = __any_sync(FULL, now.resolve(a, sg.kt, k0 + row));
                if (lane == 0) {
                    missing[st] = any;
                    bar_expect(full + 8 * st, 2 * S::TILE);
                }
                __syncwarp();
                const uint32_t dst = base + st * 2 * S::TILE;
                copy_rows<D>(a, maps.k, now, k0, sg.head, dst, FK * 128, full + 8 * st, lane);
                copy_rows<D>(a, maps.v, now, k0, sg.head, dst + S::TILE, FK * 128, full + 8 * st, lane);
            }
            if (!ok) break;
        }
        if (!ok) *dead = 1;
        all_done();
        if (*dead) {    // what has been written of the run's rows is not told apart from what has not
            line = FewLine(a, run);
            for (FewSegment sg = line.next(a, run, cta); sg.n > 0; sg = line.next(a, run, cta))
                lost_tile<T, D, FEW>(a, sg, a.part_l, a.split, cta, lane);
        }
        return;
    } else {
        // ================================================ 16 keys of each tile a warp
        uint32_t c = 0;
        const int kr = warp * 16;   // this warp's keys of a tile
        float* stats = reinterpret_cast<float*>(mem + S::STATS);
        float* merge = reinterpret_cast<float*>(mem + S::MERGE);
        for (uint32_t s = 0;; ++s) {
            const uint32_t slot = s % FAHEAD;
            bool ok = __all_sync(FULL, bar_wait(segbar + 8 * slot, (s / FAHEAD) & 1, dead, a.patience));
            const FewSegment& sg = segs[slot];
            const int n = ok ? sg.n : 0;
            float o[D / 8][4];
            float mrow[2] = {-INFINITY, -INFINITY}, lrow[2] = {0.f, 0.f};
            int pos[2] = {0, 0};
            bool odd_seen = false;
#pragma unroll
            for (int f = 0; f < D / 8; ++f)
#pragma unroll
                for (int e = 0; e < 4; ++e) o[f][e] = 0.f;
            const uint32_t qs = base + S::Q + slot * S::QTILE;
            uint32_t qf[D <= 128 ? D / 16 : 1][4];
            if (n > 0) {
                ok = __all_sync(FULL, bar_wait(qbar + 8 * slot, (s / FAHEAD) & 1, dead, a.patience));
                if constexpr (D <= 128) {
#pragma unroll
                    for (int kk = 0; kk < D / 16; ++kk) ldsm4(qf[kk], qs + tile_at<FEW>(lane & 15, kk * 2 + (lane >> 4)));
                }
#pragma unroll
                for (int j = 0; j < 2; ++j) pos[j] = sg.x.pos(a, min(sg.row0 + j * 8 + (lane >> 2), sg.M - 1));
            }
#pragma unroll 1
            for (int i = 0; i < n && ok; ++i, ++c) {
                const uint32_t lap = c / ST, st = c - lap * ST;
                const int k0 = sg.kt.at(sg.i0 + i);
                ok = __all_sync(FULL, bar_wait(full + 8 * st, lap & 1, dead, a.patience));
                if (!ok) break;
                const uint32_t ks = base + st * 2 * S::TILE, vs = ks + S::TILE;
                // A value that only some of the tokens see may be infinite or NaN, which a weight of zero does not
                // cancel: such values are taken out of the tile, and added at the end to the outputs of the
                // queries that see them.
                if (partial_keys(a, sg.p_lo, sg.p_hi, k0, FK)) {
                    bool odd = false;
#pragma unroll 1
                    for (int e = lane; e < 16 * DC; e += 32) {
                        uint4* p = reinterpret_cast<uint4*>(mem + (vs - base) + tile_at<FK>(kr + e / DC, e % DC));
                        if (odd_words<T>(*p)) *p = even_words<T>(*p), odd = true;
                    }
                    if (__any_sync(FULL, odd)) {
                        odd_seen = true;
                        proxy_fence();   // (the next copy into this stage comes behind these writes)
                        __syncwarp();
                    }
                }
                float sc[2][4];
#pragma unroll
                for (int f = 0; f < 2; ++f)
#pragma unroll
                    for (int e = 0; e < 4; ++e) sc[f][e] = 0.f;
#pragma unroll
                for (int kk = 0; kk < D / 16; ++kk) {
                    uint32_t bf[4], af[4];
                    ldsm4(bf, ks + tile_at<FK>(kr + ((lane >> 4) << 3) + (lane & 7), kk * 2 + ((lane >> 3) & 1)));
                    if constexpr (D <= 128) {
#pragma unroll
                        for (int e = 0; e < 4; ++e) af[e] = qf[kk][e];
                    } else {
                        ldsm4(af, qs + tile_at<FEW>(lane & 15, kk * 2 + (lane >> 4)));
                    }
                    Mma<T>::run(sc[0], af, bf[0], bf[1]);
                    Mma<T>::run(sc[1], af, bf[2], bf[3]);
                }
                // ---- running maximum, weights and sum
                const int kbase = k0 + kr + (lane & 3) * 2;
                const bool edge = sg.p_hi - k0 >= a.window;   // (uniform) below some token's window
                const unsigned bits = missing[st] ? missing_pages<false>(a, sg.r, k0 + kr) : 0u;
                uint32_t pf[4];
#pragma unroll
                for (int j = 0; j < 2; ++j) {
                    const int lim = pos[j] + 1 - kbase, low = edge ? pos[j] - a.window + 1 - kbase : INT32_MIN, few = a.sinks - kbase;
                    float mx = -INFINITY;
#pragma unroll
                    for (int f = 0; f < 2; ++f)
#pragma unroll
                        for (int e = 0; e < 2; ++e) {
                            float& y = sc[f][j * 2 + e];
                            const int k = f * 8 + e;
                            const bool see = k < lim && (k >= low || k < few);
                            y = see ? y * a.scale : -INFINITY;
                            if (bits && see && bits >> ((lane & 3) * 2 + k) & 1) y = __int_as_float(0x7fffffff);
                            mx = fmaxf(mx, y);
                        }
                    mx = fmaxf(mx, __shfl_xor_sync(FULL, mx, 1));
                    mx = fmaxf(mx, __shfl_xor_sync(FULL, mx, 2));
                    const float mn = fmaxf(mrow[j], mx);
                    const float ms = mn == -INFINITY ? 0.f : mn;
                    const float alpha = exp2_fast(mrow[j] - ms);
                    mrow[j] = mn;
                    float sum = 0.f;
#pragma unroll
                    for (int f = 0; f < 2; ++f)
#pragma unroll
                        for (int e = 0; e < 2; ++e) {
                            float& y = sc[f][j * 2 + e];
                            y = exp2_fast(y - ms);
                            sum += y;
                        }
                    lrow[j] = lrow[j] * alpha + sum;
                    if (__any_sync(FULL, alpha != 1.f)) {
#pragma unroll
                        for (int f = 0; f < D / 8; ++f) {
                            o[f][j * 2] *= alpha;
                            o[f][j * 2 + 1] *= alpha;
                        }
                    }
                }
                // The weights enter the product in 16 bits, as the matrix instruction takes them, each off by half a
                // step of the type; their sum stays in 32.  In f16 they are 2^15 larger: half a step down to 2^-29 of
                // the maximum, 2^-40 of it below.
#pragma unroll
                for (int f = 0; f < 2; ++f)
#pragma unroll
                    for (int j = 0; j < 2; ++j) pf[2 * f + j] = Mma<T>::pack(sc[f][2 * j] * UP, sc[f][2 * j + 1] * UP);
                // ---- values
#pragma unroll
                for (int d = 0; d < D / 16; ++d) {
                    uint32_t bf[4];
                    ldsm4_t(bf, vs + tile_at<FK>(kr + (((lane >> 3) & 1) << 3) + (lane & 7), d * 2 + (lane >> 4)));
                    Mma<T>::run(o[2 * d], pf, bf[0], bf[1]);
                    Mma<T>::run(o[2 * d + 1], pf, bf[2], bf[3]);
                }
                __syncwarp();
                if (lane == 0) bar_arrive(empty + 8 * st);
            }
            // ---- the warps' parts joined, four rows at a time
#pragma unroll
            for (int j = 0; j < 2; ++j) {
                float l = lrow[j];
                l += __shfl_xor_sync(FULL, l, 1);
                l += __shfl_xor_sync(FULL, l, 2);
                if ((lane & 3) == 0) {
                    stats[warp * FEW + j * 8 + (lane >> 2)] = mrow[j];
                    stats[4 * FEW + warp * FEW + j * 8 + (lane >> 2)] = l;
                }
            }
            const int odd_any = __any_sync(FULL, odd_seen);
            if (lane == 0) gone[warp] = ok ? odd_any : 2;
            asm volatile("bar.sync 1, 128;" ::: "memory");
            const int f0 = gone[0], f1 = gone[1], f2 = gone[2], f3 = gone[3];
            // All four leave here and nowhere else, at a run's end or when one of them has given up (*dead is set): a warp that saw
            // the end and left by itself would be waited for by one whose wait for the same segment ran out.
            if (n == 0 || f0 == 2 || f1 == 2 || f2 == 2 || f3 == 2) break;
            const bool fix = (f0 | f1 | f2 | f3) != 0;
            float scale[2];
#pragma unroll
            for (int j = 0; j < 2; ++j) {
                float m = -INFINITY;
#pragma unroll
                for (int w = 0; w < 4; ++w) m = fmaxf(m, stats[w * FEW + j * 8 + (lane >> 2)]);
                scale[j] = exp2_fast(mrow[j] - (m == -INFINITY ? 0.f : m)) * (1.f / UP);
            }
            const int rows = min(FEW, sg.M - sg.row0);
            const bool whole = sg.whole;
            const int part = 2 * cta + (sg.i0 == 0);   // (a run has two parts at most, one of them from a tile's start)
#pragma unroll
            for (int g = 0; g < FEW / 4; ++g) {
                if (4 * g >= rows) break;
#pragma unroll
                for (int j = 0; j < 2; ++j)
                    if (j == g / 2 && (lane >> 4) == (g & 1)) {
#pragma unroll
                        for (int f = 0; f < D / 8; ++f)
                            *reinterpret_cast<float2*>(merge + (warp * 4 + (lane >> 2 & 3)) * D + f * 8 + (lane & 3) * 2) =
                                make_float2(o[f][j * 2] * scale[j], o[f][j * 2 + 1] * scale[j]);
                    }
                asm volatile("bar.sync 1, 128;" ::: "memory");
                for (int i = tid; i < D; i += 128) {    // a row's four neighbouring elements each
                    const int r = 4 * g + i / (D / 4), d = i % (D / 4) * 4;
                    if (r >= rows) continue;
                    float m = -INFINITY, l = 0.f;
#pragma unroll
                    for (int w = 0; w < 4; ++w) m = fmaxf(m, stats[w * FEW + r]);
                    const float ms = m == -INFINITY ? 0.f : m;
                    float4 y = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
                    for (int w = 0; w < 4; ++w) {
                        l += exp2_fast(stats[w * FEW + r] - ms) * stats[4 * FEW + w * FEW + r];
                        const float4 z = *reinterpret_cast<const float4*>(merge + (w * 4 + (r & 3)) * D + d);
                        y = make_float4(y.x + z.x, y.y + z.y, y.z + z.z, y.w + z.w);
                    }
                    const float inv = l == 0.f ? 0.f : 1.f / l;
                    const float lse = l == 0.f ? -INFINITY : m + log2f(l);
                    y = make_float4(y.x * inv, y.y * inv, y.z * inv, y.w * inv);
                    const int row = sg.row0 + r;
                    if (fix) {   // (their weights are positive: exp(s - m) > 0)
                        const int* table = a.table + int64_t(sg.r) * a.width;
                        const int p = sg.x.pos(a, row);
                        for (int t = 0; t < n; ++t) {
                            const int k0 = sg.kt.at(sg.i0 + t);
                            if (partial_keys(a, sg.p_lo, sg.p_hi, k0, FK)) add_odd<T, false>(a, table, p, k0, FK, sg.head, d, y);
                        }
                    }
                    const int j = row / a.gs, h = sg.head * a.gs + row - j * a.gs;
                    if (whole) {
                        T* out = static_cast<T*>(a.out) + (sg.x.q0 + j) * a.os[0] + h * a.os[1] + d;
                        *reinterpret_cast<uint2*>(out) = make_uint2(Mma<T>::pack(y.x, y.y), Mma<T>::pack(y.z, y.w));
                        if (d == 0 && a.lse) a.lse[int64_t(sg.x.q0 + j) * a.Hq + h] = lse * 0.693147180559945309f;
                    } else {
                        const int64_t at = int64_t(part) * FEW + r;
                        *reinterpret_cast<float4*>(a.part_o + at * D + d) = y;
                        if (d == 0) a.part_l[at] = make_float2(m, l);
                    }
                }
                asm volatile("bar.sync 1, 128;" ::: "memory");
            }
            if (sg.parts > 0 && tid == 0)   // this CTA has the tile's first part and says how many CTAs have one
                a.split[cta] = make_int4(sg.r, sg.head, sg.row0, sg.parts);
            __syncwarp();
            if (lane == 0) bar_arrive(segfree + 8 * slot);
        }
    }
    all_done();
}

template <typename T, int D>
static fs_status launch(const ChunkArgs& a, const ChunkMaps& maps, void* stream) {
    const fs_status st = prepare_kernel(reinterpret_cast<const void*>(chunk_few_kernel<T, D>));
    if (st != FS_OK) return st;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(unsigned(a.grid + (a.t_grid > 0)), 1, 1);
    cfg.blockDim = dim3(FNT, 1, 1);
    cfg.dynamicSmemBytes = FewSmem<D>::TOTAL;
    cfg.stream = static_cast<cudaStream_t>(stream);
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    const cudaError_t e = cudaLaunchKernelEx(&cfg, chunk_few_kernel<T, D>, a, maps);
    return e == cudaSuccess ? FS_OK : cuda_fail(e);
}

template <typename T>
static fs_status launch_type(const ChunkArgs& a, const ChunkMaps& maps, int head_dim, void* stream) {
    return head_dim == 64    ? launch<T, 64>(a, maps, stream)
           : head_dim == 128 ? launch<T, 128>(a, maps, stream)
                             : launch<T, 256>(a, maps, stream);
}

fs_status launch_chunk_few(const ChunkArgs& a, const ChunkMaps& maps, int dtype, int head_dim, void* stream) {
    return dtype == FS_BF16 ? launch_type<__nv_bfloat16>(a, maps, head_dim, stream) : launch_type<__half>(a, maps, head_dim, stream);
}

}  // namespace fsd
