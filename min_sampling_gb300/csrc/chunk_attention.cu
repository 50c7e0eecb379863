// Attention of chunks of new tokens over a paged key/value cache (sm_103a).
//
// Request r has nq queries, its last nq tokens of len.  The query at position p sees the keys k <= p
// with k > p - window or k < sinks:
//   out = softmax(scale * q K^T) V  over those keys.
// The queries of all heads that share a key/value head are the rows of one matrix, so that a key is
// read once for all of them: nq * (heads / key-value heads) rows, in tiles.
//
// The work of a launch is one line of units, (request, key/value head, query tile, key tile), cut into
// equal runs, one for each CTA, whatever the mix of lengths.  A CTA takes the tiles in its run one after the
// other; a tile that lies in one run is written at once, the parts of one that is cut are joined by
// their maxima and sums in a fixed order (join_chunk_kernel; no atomics):
//   m = max_i m_i,  l = sum_i 2^(m_i - m) l_i,  out = sum_i 2^(m_i - m) l_i out_i / l.
//
// Three launches: chunk_tensor.cu, requests of more than 16 rows, on the 5th-generation tensor cores; chunk_few.cu, requests of
// up to 16 rows, single tokens above all; the parts joined.  The first two have lines of their own and do not wait for each other:
// the SMs that are done with the first take the second's CTAs.  (The other way round, and one CTA planning
// for all, 5 us more for two chunks of 1021 tokens behind 16384 and 47 single tokens, of 465. On SMs
// of their own beside the first they slowed its CTAs on the neighbouring SMs by a sixth: 35 us more.)
// chunk_rows_kernel (mma.sync) has many rows of heads of 256, and a few where the caches' strides have no map for the copy engine.
#include "chunk.cuh"

#include <atomic>
#include <numeric>
#include <type_traits>

#include "chunk_copy.cuh"
#include "fragments.cuh"

namespace fsd {

constexpr int CSTAGES = 2;      // tiles of keys and values in flight

// Shared memory: queries, CSTAGES x (keys, values), the keys' offsets.
template <int D, int MT, int KT>
struct ChunkSmem {
    static constexpr int TILE = KT * D * 2;
    static constexpr int KV = MT * D * 2;
    static constexpr int OFF = KV + CSTAGES * 2 * TILE;
    static constexpr int TOTAL = OFF + 2 * 2 * KT * 8 + 256;
};

// WM x WN warps over a tile of MT = 16 RM WM query rows and KT keys; each warp keeps its own running
// maximum, sum and output over its share of the keys.  Bound by the reads of keys and values.
template <typename T, int D, int MT, int WM, int WN, int RM, int KT>
__global__ void __launch_bounds__(32 * WM * WN) chunk_rows_kernel(const __grid_constant__ ChunkArgs a) {
    constexpr int NT = 32 * WM * WN;
    static_assert(MT == 16 * RM * WM && KT <= NT, "warp layout");
    using S = ChunkSmem<D, MT, KT>;
    constexpr int KW = KT / WN;       // keys per warp and tile
    constexpr int NF = KW / 8;        // score fragments
    constexpr int DC = D / 8;         // 16-byte chunks per row
    constexpr float UP = std::is_same<T, __half>::value ? 32768.f : 1.f;   // the weights' factor in the product
    static_assert(WN * MT * (D + 2) * 4 <= S::OFF, "the warps' parts fit where the tiles were");
    extern __shared__ __align__(128) unsigned char smem[];
    const uint32_t sbase = smem_u32(smem);
    int64_t* soff = reinterpret_cast<int64_t*>(smem + S::OFF);                       // [2][2][KT]
    int64_t* words = reinterpret_cast<int64_t*>(smem + S::OFF + 2 * 2 * KT * 8);     // scan, then the place found
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int wm = warp / WN, wn = warp % WN;
    const int cta = int(blockIdx.x);
    if (!few_starts(a)) return;

    // ---- this CTA's run of units
    const Run line = run_of<NT, MT, KT>(a, cta, words);
    const int64_t run = line.length, last = line.last;
    int64_t unit = line.first;
    Place pl = line.place;
    if (tid == 0) a.split[cta] = make_int4(0, 0, 0, 0);
    if (a.zero_rest) zero_rest<T, D>(a, cta, NT);

#pragma unroll 1
    while (unit < last) {
        // ---- the tile that the unit lies in
        Request x = request<false>(a, pl.r);
        while (unit >= pl.before + pl.units * a.Hkv) {
            pl.before += pl.units * a.Hkv;
            x = request<false>(a, ++pl.r);
            pl.units = units_of<MT, KT>(a, x);
        }
        const int head = int((unit - pl.before) / pl.units);
        const int M = x.rows(a);
        int64_t first = pl.before + head * pl.units;   // the tile's first unit
        int row0 = 0;
        KeyTiles<KT> kt(a, x.pos(a, 0), x.pos(a, min(MT, M) - 1));
        while (unit >= first + kt.n + FEW_START) {
            first += kt.n + FEW_START;
            row0 += MT;
            kt = KeyTiles<KT>(a, x.pos(a, row0), x.pos(a, min(row0 + MT, M) - 1));
        }
        // its key tiles in this run
        const int64_t after = first + kt.n + FEW_START;
        const int i0 = int(max(unit - first - FEW_START, int64_t(0))), i1 = max(int(min(after, last) - first) - FEW_START, i0);
        unit = min(after, last);
        if (i1 == i0) break;   // (a run that ends within a tile's FEW_START leaves all of it to the next)
        const bool whole = i0 == 0 && i1 == kt.n;
        const int p_lo = x.pos(a, row0), p_hi = x.pos(a, min(row0 + MT, M) - 1);
        const int* table = a.table + int64_t(pl.r) * a.width;
        const int tiles = i1 - i0;
        auto partial = [&](int k0) { return partial_keys(a, p_lo, p_hi, k0, KT); };

        __syncthreads();   // the tile before is done with shared memory
        for (int i = tid; i < MT * DC; i += NT) {
            const int r = i / DC, c = i % DC, row = row0 + r;
            const bool on = row < M;
            const int j = on ? row / a.gs : 0, h = head * a.gs + (on ? row % a.gs : 0);
            cp16(sbase + chunk_at<D>(r, c), static_cast<const T*>(a.q) + (x.q0 + j) * a.qs[0] + h * a.qs[1] + c * 8, on);
        }
        // ---- pipeline of key/value tiles.  A key's offsets are looked up one tile before its
        // loads are issued, by one thread per key.
        constexpr int64_t MISSING = NOWHERE + 1;   // of a page that does not exist
        auto look_up = [&](int tile, int64_t& ko, int64_t& vo) {
            ko = vo = NOWHERE;
            if (tid >= KT || tile >= tiles) return;
            const int key = kt.at(i0 + tile) + tid;
            if (kt.seen(key)) {
                const int pi = a.page_shift >= 0 ? key >> a.page_shift : key / a.page_size;
                const int page = get<false>(a, table + pi);
                if (page >= 0 && page < a.num_pages) {
                    const int s = key - pi * a.page_size;
                    ko = page * a.kc[0] + s * a.kc[1] + head * a.kc[2];
                    vo = page * a.vc[0] + s * a.vc[1] + head * a.vc[2];
                } else {
                    ko = MISSING;
                }
            }
        };
        auto put_offsets = [&](int tile, int64_t ko, int64_t vo) {
            if (tid < KT) {
                soff[(tile & 1) * 2 * KT + tid] = ko;
                soff[(tile & 1) * 2 * KT + KT + tid] = vo;
            }
        };
        auto issue = [&](int tile) {
            const int64_t* off = soff + (tile & 1) * 2 * KT;
            const uint32_t kd = sbase + S::KV + (tile % CSTAGES) * 2 * S::TILE;
#pragma unroll
            for (int i = 0; i < KT * DC / NT; ++i) {
                const int r = (tid + i * NT) / DC, c = (tid + i * NT) % DC;
                const int64_t ko = off[r], vo = off[KT + r];
                const bool on = vo != NOWHERE;
                if (ko == MISSING)   // its keys are NaN, and so is every query that sees it
                    *reinterpret_cast<uint4*>(smem + (kd - sbase) + chunk_at<D>(r, c)) =
                        make_uint4(0x7fff7fffu, 0x7fff7fffu, 0x7fff7fffu, 0x7fff7fffu);
                else
                    cp16(kd + chunk_at<D>(r, c), static_cast<const T*>(a.k) + (on ? ko + c * 8 : 0), on);
                cp16(kd + S::TILE + chunk_at<D>(r, c), static_cast<const T*>(a.v) + (on ? vo + c * 8 : 0), on);
            }
        };
        int64_t ko, vo;
#pragma unroll
        for (int t = 0; t < CSTAGES - 1; ++t) {
            look_up(t, ko, vo);
            put_offsets(t, ko, vo);
            __syncthreads();
            if (t < tiles) issue(t);
            cp_async_commit();
        }
        look_up(CSTAGES - 1, ko, vo);
        put_offsets(CSTAGES - 1, ko, vo);

        float o[RM][D / 8][4];
        float mrow[RM][2], lrow[RM][2];
        int pos[RM][2];
        bool odd_seen = false;
#pragma unroll
        for (int i = 0; i < RM; ++i) {
#pragma unroll
            for (int f = 0; f < D / 8; ++f)
#pragma unroll
                for (int e = 0; e < 4; ++e) o[i][f][e] = 0.f;
#pragma unroll
            for (int j = 0; j < 2; ++j) {
                mrow[i][j] = -INFINITY;
                lrow[i][j] = 0.f;
                pos[i][j] = x.pos(a, min(row0 + (wm * RM + i) * 16 + j * 8 + (lane >> 2), M - 1));
            }
        }
        const int qrow = (wm * RM) * 16 + (lane & 15), qch = lane >> 4;

#pragma unroll 1
        for (int t = 0; t < tiles; ++t) {
            cp_async_wait<CSTAGES - 2>();
            __syncthreads();  // tile t is there, tile t - 1 is done with, the next offsets are written
            if (t + CSTAGES - 1 < tiles) issue(t + CSTAGES - 1);
            cp_async_commit();
            look_up(t + CSTAGES, ko, vo);
            const uint32_t ks = sbase + S::KV + (t % CSTAGES) * 2 * S::TILE, vs = ks + S::TILE;
            const int k0 = kt.at(i0 + t);
            // A value that only some of the tokens see may be infinite or NaN, which a weight of
            // zero does not cancel: such values are taken out of the tile, and added at the end to the
            // outputs of the queries that see them.
            if (partial(k0)) {
                unsigned char* vb = smem + (vs - sbase);
                bool odd = false;
                for (int i = tid; i < KT * DC; i += NT) odd |= odd_words<T>(*reinterpret_cast<const uint4*>(vb + i * 16));
                if (__syncthreads_or(odd)) {
                    odd_seen = true;
                    for (int i = tid; i < KT * DC; i += NT) {
                        uint4* w = reinterpret_cast<uint4*>(vb + i * 16);
                        *w = even_words<T>(*w);
                    }
                    __syncthreads();
                }
            }

            // ---- scores of this warp's keys
            float s[RM][NF][4];
#pragma unroll
            for (int i = 0; i < RM; ++i)
#pragma unroll
                for (int f = 0; f < NF; ++f)
#pragma unroll
                    for (int e = 0; e < 4; ++e) s[i][f][e] = 0.f;
#pragma unroll
            for (int kk = 0; kk < D / 16; ++kk) {
                uint32_t af[RM][4];
#pragma unroll
                for (int i = 0; i < RM; ++i) ldsm4(af[i], sbase + chunk_at<D>(qrow + i * 16, kk * 2 + qch));
#pragma unroll
                for (int f = 0; f < NF; f += 2) {
                    uint32_t bf[4];
                    const int kr = wn * KW + f * 8 + ((lane >> 4) << 3) + (lane & 7);
                    ldsm4(bf, ks + chunk_at<D>(kr, kk * 2 + ((lane >> 3) & 1)));
#pragma unroll
                    for (int i = 0; i < RM; ++i) {
                        Mma<T>::run(s[i][f], af[i], bf[0], bf[1]);
                        Mma<T>::run(s[i][f + 1], af[i], bf[2], bf[3]);
                    }
                }
            }
            // ---- running maximum, weights and sum
            const int kbase = k0 + wn * KW + (lane & 3) * 2;
            const bool edge = p_hi - k0 >= a.window;   // (uniform) below some token's window
            uint32_t pf[RM][NF / 2][4];
#pragma unroll
            for (int i = 0; i < RM; ++i) {
#pragma unroll
                for (int j = 0; j < 2; ++j) {
                    const int lim = pos[i][j] + 1 - kbase;
                    float mx = -INFINITY;
#pragma unroll
                    for (int f = 0; f < NF; ++f)
#pragma unroll
                        for (int e = 0; e < 2; ++e) {
                            float& y = s[i][f][j * 2 + e];
                            y = f * 8 + e < lim ? y * a.scale : -INFINITY;
                        }
                    if (edge) {
                        const int low = pos[i][j] - a.window + 1 - kbase, few = a.sinks - kbase;
#pragma unroll
                        for (int f = 0; f < NF; ++f)
#pragma unroll
                            for (int e = 0; e < 2; ++e)
                                if (f * 8 + e < low && f * 8 + e >= few) s[i][f][j * 2 + e] = -INFINITY;
                    }
#pragma unroll
                    for (int f = 0; f < NF; ++f) mx = fmaxf(mx, fmaxf(s[i][f][j * 2], s[i][f][j * 2 + 1]));
                    mx = fmaxf(mx, __shfl_xor_sync(FULL, mx, 1));
                    mx = fmaxf(mx, __shfl_xor_sync(FULL, mx, 2));
                    const float mn = fmaxf(mrow[i][j], mx);
                    const float ms = mn == -INFINITY ? 0.f : mn;
                    const float alpha = exp2_fast(mrow[i][j] - ms);
                    mrow[i][j] = mn;
                    float sum = 0.f;
#pragma unroll
                    for (int f = 0; f < NF; ++f)
#pragma unroll
                        for (int e = 0; e < 2; ++e) {
                            float& y = s[i][f][j * 2 + e];
                            y = exp2_fast(y - ms);
                            sum += y;
                        }
                    lrow[i][j] = lrow[i][j] * alpha + sum;
                    if (__any_sync(FULL, alpha != 1.f)) {
#pragma unroll
                        for (int f = 0; f < D / 8; ++f) {
                            o[i][f][j * 2] *= alpha;
                            o[i][f][j * 2 + 1] *= alpha;
                        }
                    }
                }
                // The weights enter the product in 16 bits, as the matrix instruction takes them, each off by half a
                // step of the type; their sum stays in 32.  In f16 they are 2^15 larger: half a step down to 2^-29 of
                // the maximum, 2^-40 of it below.
                auto weights = [&](int f, int e) { return Mma<T>::pack(s[i][f][e] * UP, s[i][f][e + 1] * UP); };
#pragma unroll
                for (int f = 0; f < NF / 2; ++f) {
                    pf[i][f][0] = weights(2 * f, 0);
                    pf[i][f][1] = weights(2 * f, 2);
                    pf[i][f][2] = weights(2 * f + 1, 0);
                    pf[i][f][3] = weights(2 * f + 1, 2);
                }
            }
            // ---- values
#pragma unroll
            for (int f = 0; f < NF / 2; ++f) {
#pragma unroll
                for (int d = 0; d < D / 16; ++d) {
                    uint32_t bf[4];
                    const int kr = wn * KW + f * 16 + (((lane >> 3) & 1) << 3) + (lane & 7);
                    ldsm4_t(bf, vs + chunk_at<D>(kr, d * 2 + (lane >> 4)));
#pragma unroll
                    for (int i = 0; i < RM; ++i) {
                        Mma<T>::run(o[i][2 * d], pf[i][f], bf[0], bf[1]);
                        Mma<T>::run(o[i][2 * d + 1], pf[i][f], bf[2], bf[3]);
                    }
                }
            }
            put_offsets(t + CSTAGES, ko, vo);
        }

        // ---- the warps' parts joined through shared memory
        cp_async_wait<0>();
        __syncthreads();
        float* so = reinterpret_cast<float*>(smem);                  // [WN][MT][D]
        float* sm = so + WN * MT * D;                                // [WN][MT]
        float* sl = sm + WN * MT;                                    // [WN][MT]
#pragma unroll
        for (int i = 0; i < RM; ++i)
#pragma unroll
            for (int j = 0; j < 2; ++j) {
                const int r = (wm * RM + i) * 16 + j * 8 + (lane >> 2);
                float l = lrow[i][j];
                l += __shfl_xor_sync(FULL, l, 1);
                l += __shfl_xor_sync(FULL, l, 2);
                if ((lane & 3) == 0) {
                    sm[wn * MT + r] = mrow[i][j];
                    sl[wn * MT + r] = l;
                }
#pragma unroll
                for (int f = 0; f < D / 8; ++f)
                    *reinterpret_cast<float2*>(so + (wn * MT + r) * D + f * 8 + (lane & 3) * 2) =
                        make_float2(o[i][f][j * 2] * (1.f / UP), o[i][f][j * 2 + 1] * (1.f / UP));
            }
        __syncthreads();
        const int slot = 2 * cta + (i0 == 0);   // (a run has two parts at most, one of them from a tile's start)
        for (int i = tid; i < MT * (D / 4); i += NT) {
            const int r = i / (D / 4), c = i % (D / 4), row = row0 + r;
            if (row >= M) continue;
            float m = -INFINITY;
#pragma unroll
            for (int w = 0; w < WN; ++w) m = fmaxf(m, sm[w * MT + r]);
            const float ms = m == -INFINITY ? 0.f : m;
            float l = 0.f;
            float4 y = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
            for (int w = 0; w < WN; ++w) {
                const float f = exp2_fast(sm[w * MT + r] - ms);
                const float4 z = *reinterpret_cast<const float4*>(so + (w * MT + r) * D + c * 4);
                l += f * sl[w * MT + r];
                y.x += f * z.x, y.y += f * z.y, y.z += f * z.z, y.w += f * z.w;
            }
            const float inv = l == 0.f ? 0.f : 1.f / l;
            const float lse = l == 0.f ? -INFINITY : m + log2f(l);
            y = make_float4(y.x * inv, y.y * inv, y.z * inv, y.w * inv);
            if (odd_seen) {   // (their weights are positive: exp(s - m) > 0)
                const int p = x.pos(a, row);
                for (int t = 0; t < tiles; ++t) {
                    const int k0 = kt.at(i0 + t);
                    if (partial(k0)) add_odd<T, false>(a, table, p, k0, KT, head, c * 4, y);
                }
            }
            const int j = row / a.gs, h = head * a.gs + row % a.gs;
            if (whole) {
                T* out = static_cast<T*>(a.out) + (x.q0 + j) * a.os[0] + h * a.os[1] + c * 4;
                *reinterpret_cast<uint2*>(out) = make_uint2(Mma<T>::pack(y.x, y.y), Mma<T>::pack(y.z, y.w));
                if (c == 0 && a.lse) a.lse[int64_t(x.q0 + j) * a.Hq + h] = lse * 0.693147180559945309f;
            } else {
                const int64_t at = int64_t(slot) * MT + r;
                *reinterpret_cast<float4*>(a.part_o + at * D + c * 4) = y;
                if (c == 0) a.part_l[at] = make_float2(m, l);
            }
        }
        if (!whole && i0 == 0 && tid == 0)   // this CTA has the tile's first part and says how many CTAs have one
            a.split[cta] = make_int4(pl.r, head, row0, int((after - 1) / run) - cta + 1);
    }
}

// ------------------------------------------------------------------ parts joined

// A tile that was cut: its queries' first token, rows, head, first row, parts, and the CTA that has the first of them.
struct JoinTile {
    int q0, rows, head, row0, parts, cta;
};
constexpr int JOIN_CTAS = 2;    // on an SM

// Rows of the list's tiles: a lane has K times 4 elements of one, P parts' loads in flight at once.
template <typename T, int D, int K, int P>
__device__ __forceinline__ void join_rows(const ChunkArgs& a, const JoinTile* tiles, int few_tiles, int MT, int all) {
    constexpr int LANES = D / (4 * K), ROWS = 32 / LANES;   // of a row, of a warp
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, d = lane % LANES * 4, few_rows = few_tiles * MT;
#pragma unroll 1
    for (int at = (int(blockIdx.x) * 16 + warp) * ROWS; at < all; at += int(gridDim.x) * 16 * ROWS) {
        const bool few = at < few_rows;
        const int rows = few ? MT : MANY, n = few ? at : at - few_rows, r = n % rows + lane / LANES;
        const JoinTile& s = tiles[(few ? 0 : few_tiles) + n / rows];
        const int row = s.row0 + r, c = s.cta, parts = row < s.rows ? s.parts : 0;
        const float* part_o = few ? a.part_o : a.t_part_o;
        const float2* part_l = few ? a.part_l : a.t_part_l;
        // the first part is the one that starts its tile
        auto slot = [&](int i) { return (2 * (c + i) + (i == 0)) * rows + r; };
        float m = -INFINITY, l = 0.f;
        float4 y[K];
#pragma unroll
        for (int k = 0; k < K; ++k) y[k] = make_float4(0.f, 0.f, 0.f, 0.f);
        // P parts at a time: their joint maximum, then their sums.  (A NaN part makes the sum NaN through its own weight.)
        for (int p0 = 0; p0 < parts; p0 += P) {
            float2 w[P];
            float4 o[P][K];
#pragma unroll
            for (int j = 0; j < P; ++j) {
                w[j] = make_float2(-INFINITY, 0.f);
                if (p0 + j < parts) {
                    w[j] = part_l[slot(p0 + j)];
#pragma unroll
                    for (int k = 0; k < K; ++k)
                        o[j][k] = *reinterpret_cast<const float4*>(part_o + slot(p0 + j) * D + d + k * LANES * 4);
                }
            }
            float mn = m;
#pragma unroll
            for (int j = 0; j < P; ++j) mn = fmaxf(mn, w[j].x);
            const float ms = mn == -INFINITY ? 0.f : mn, f0 = exp2f(m - ms);
            m = mn;
            l *= f0;
#pragma unroll
            for (int k = 0; k < K; ++k) y[k] = make_float4(y[k].x * f0, y[k].y * f0, y[k].z * f0, y[k].w * f0);
#pragma unroll
            for (int j = 0; j < P; ++j)
                if (p0 + j < parts) {
                    const float f = exp2f(w[j].x - ms) * w[j].y;
                    l += f;
#pragma unroll
                    for (int k = 0; k < K; ++k)
                        y[k] = make_float4(y[k].x + f * o[j][k].x, y[k].y + f * o[j][k].y, y[k].z + f * o[j][k].z,
                                           y[k].w + f * o[j][k].w);
                }
        }
        if (row >= s.rows) continue;
        const float inv = l == 0.f ? 0.f : 1.f / l;
        const int j = row / a.gs, h = s.head * a.gs + row % a.gs;
        T* out = static_cast<T*>(a.out) + (s.q0 + j) * a.os[0] + h * a.os[1] + d;
#pragma unroll
        for (int k = 0; k < K; ++k)
            *reinterpret_cast<uint2*>(out + k * LANES * 4) =
                make_uint2(Mma<T>::pack(y[k].x * inv, y[k].y * inv), Mma<T>::pack(y[k].z * inv, y[k].w * inv));
        if (a.lse && d == 0) a.lse[int64_t(s.q0 + j) * a.Hq + h] = (l == 0.f ? -INFINITY : m + log2f(l)) * 0.693147180559945309f;
    }
}

// The CTAs, as many as are resident, list the tiles that were cut and share their rows: so that a warp has a row or two and many
// parts in flight where there are few rows, and else two parts of several rows.  (16 rows a CTA, 2736 CTAs that mostly found nothing to do:
// 12 to 18 us; four rows a warp, one part after the other, 21 us for the 148 rows and 9 parts of one short chunk.)
template <typename T, int D>
__global__ void __launch_bounds__(512, JOIN_CTAS) join_chunk_kernel(const __grid_constant__ ChunkArgs a, int MT) {
    extern __shared__ JoinTile tiles[];     // [grid] of the few rows' CTAs, [t_grid] of the tensor cores'
    __shared__ int count[2][16];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    grid_dependency_wait();
    allow_dependents();
    // The list, in the order of the CTAs, the same in all of this kernel's.
    int few_tiles = 0, n_tiles = 0;
    for (int i0 = 0; i0 < a.grid + a.t_grid; i0 += 512) {
        const int i = i0 + int(threadIdx.x), c = i < a.grid ? i : i - a.grid;
        const bool few = i < a.grid;
        int4 s = make_int4(0, 0, 0, 0);
        if (c < (few ? a.grid : a.t_grid)) s = (few ? a.split : a.t_split)[c];
        const unsigned cut = __ballot_sync(FULL, s.w > 0), cut_few = __ballot_sync(FULL, few && s.w > 0);
        __syncthreads();
        if (lane == 0) count[0][warp] = __popc(cut_few), count[1][warp] = __popc(cut);
        __syncthreads();
        int here = n_tiles + __popc(cut & ((1u << lane) - 1));
        for (int w = 0; w < 16; ++w) {
            if (w < warp) here += count[1][w];
            few_tiles += count[0][w], n_tiles += count[1][w];
        }
        if (s.w > 0) {
            const Request x = request<true>(a, s.x);
            tiles[here] = JoinTile{x.q0, x.rows(a), s.y, s.z, s.w, c};
        }
    }
    __syncthreads();
    const int all = few_tiles * MT + (n_tiles - few_tiles) * MANY;
    constexpr int K = D == 256 ? 2 : 1;
    if (all <= int(gridDim.x) * 16) join_rows<T, D, K, 4 / K>(a, tiles, few_tiles, MT, all);
    else join_rows<T, D, 2, 2>(a, tiles, few_tiles, MT, all);
}

// ------------------------------------------------------------------ host

template <typename... P, typename... A>
static fs_status launch_pdl(void (*kernel)(P...), dim3 grid, unsigned block, size_t smem, void* stream, const A&... args) {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = grid;
    cfg.blockDim = dim3(block, 1, 1);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = static_cast<cudaStream_t>(stream);
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    const cudaError_t e = cudaLaunchKernelEx(&cfg, kernel, args...);
    return e == cudaSuccess ? FS_OK : cuda_fail(e);
}

using Encode = CUresult (*)(CUtensorMap*, CUtensorMapDataType, cuuint32_t, void*, const cuuint64_t*, const cuuint64_t*,
                            const cuuint32_t*, const cuuint32_t*, CUtensorMapInterleave, CUtensorMapSwizzle,
                            CUtensorMapL2promotion, CUtensorMapFloatOOBfill);

static Encode encoder() {
    static const Encode fn = [] {
        void* p = nullptr;
        cudaDriverEntryPointQueryResult found;
        const cudaError_t e = cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &p, 12000, cudaEnableDefault, &found);
        if (e != cudaSuccess) cudaGetLastError();
        return e == cudaSuccess && found == cudaDriverEntryPointSuccess ? reinterpret_cast<Encode>(p) : nullptr;
    }();
    return fn;
}

static bool tensor_map(CUtensorMap* map, const void* base, int dtype, int rank, const cuuint64_t* dims, const cuuint64_t* pitch,
                       const cuuint32_t* box) {
    const cuuint32_t ones[4] = {1, 1, 1, 1};
    const Encode encode = encoder();
    return encode && encode(map, dtype == FS_BF16 ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16 : CU_TENSOR_MAP_DATA_TYPE_FLOAT16, rank,
                            const_cast<void*>(base), dims, pitch, box, ones, CU_TENSOR_MAP_INTERLEAVE_NONE,
                            CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                            CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// Rows of `dim` elements at offsets sum_i x_i strides[i], x_i < sizes[i], as the rows of one matrix: row number sum_i x_i
// steps[i].  False where the strides have no common divisor of a row's length or more.
static bool row_map(CUtensorMap* map, const void* base, int dtype, int dim, int n, const int64_t* strides, const int64_t* sizes,
                    int* steps) {
    int64_t g = 0;
    for (int i = 0; i < n; ++i) {
        if (sizes[i] < 2) continue;
        if (strides[i] < 0) return false;
        g = std::gcd(g, strides[i]);
    }
    if (g == 0) g = dim;
    if (g < dim || g >= int64_t(1) << 36) return false;
    int64_t last = 0;
    for (int i = 0; i < n; ++i) {
        const int64_t step = sizes[i] < 2 ? 0 : strides[i] / g;
        if (step > 0 && (sizes[i] - 1) > (int64_t(0x7ffffffe) - last) / step) return false;
        steps[i] = int(step);
        last += step * (std::max<int64_t>(sizes[i], 1) - 1);
    }
    const cuuint64_t dims[2] = {cuuint64_t(dim), cuuint64_t(last + 1)}, pitch[1] = {cuuint64_t(g) * 2};
    const cuuint32_t box[2] = {64, 1};
    return tensor_map(map, base, dtype, 2, dims, pitch, box);
}

// Boxes of `rows` slots of a page.
static bool box_map(CUtensorMap* map, const ChunkArgs& a, const void* base, int dtype, int dim, const int64_t* strides, int rows) {
    const int64_t sizes[3] = {a.page_size, a.Hkv, std::max(a.num_pages, 1)}, by[3] = {strides[1], strides[2], strides[0]};
    const cuuint64_t dims[4] = {cuuint64_t(dim), cuuint64_t(sizes[0]), cuuint64_t(sizes[1]), cuuint64_t(sizes[2])};
    cuuint64_t pitch[3];
    for (int i = 0; i < 3; ++i) {
        if (sizes[i] > 1 && (by[i] < dim || by[i] >= int64_t(1) << 38)) return false;
        pitch[i] = sizes[i] > 1 ? cuuint64_t(by[i]) * 2 : cuuint64_t(dim) * 2;
    }
    const cuuint32_t box[4] = {64, cuuint32_t(rows), 1, 1};
    return tensor_map(map, base, dtype, 4, dims, pitch, box);
}
bool chunk_maps(const ChunkArgs& a, int dtype, int head_dim, ChunkMaps& m) {
    const int64_t cache[3] = {a.num_pages, a.page_size, a.Hkv}, query[2] = {a.N, a.Hq};
    if (!row_map(&m.k.rows, a.k, dtype, head_dim, 3, a.kc, cache, m.k.step) ||
        !row_map(&m.v.rows, a.v, dtype, head_dim, 3, a.vc, cache, m.v.step) ||
        !row_map(&m.q.rows, a.q, dtype, head_dim, 2, a.qs, query, m.q.step))
        return false;
    if (a.page_shift >= 3) {
        m.k.box = m.v.box = std::min(a.page_size, 64);
        if (!box_map(&m.k.boxes, a, a.k, dtype, head_dim, a.kc, m.k.box)) m.k.box = 0;
        if (!box_map(&m.v.boxes, a, a.v, dtype, head_dim, a.vc, m.v.box)) m.v.box = 0;
    }
    constexpr int ROWS = MANY / 2;
    if (ROWS % a.gs == 0) {
        // (strides of dimensions of one element address nothing)
        const cuuint64_t dims[3] = {cuuint64_t(head_dim), cuuint64_t(a.Hq), cuuint64_t(a.N)};
        const int64_t by[2] = {a.Hq > 1 ? a.qs[1] : head_dim, a.N > 1 ? a.qs[0] : head_dim};
        const cuuint64_t pitch[2] = {cuuint64_t(by[0]) * 2, cuuint64_t(by[1]) * 2};
        const cuuint32_t box[3] = {64, cuuint32_t(a.gs), cuuint32_t(ROWS / a.gs)};
        m.qrows = by[0] >= head_dim && by[1] >= head_dim && tensor_map(&m.q.boxes, a.q, dtype, 3, dims, pitch, box);
    }
    return true;
}

// Tiles and CTAs of a call, and the bytes of its parts.
struct ChunkPlan {
    int MT, KT;         // chunk_rows_kernel's tile
    int grid, least;    // its CTAs; key tiles of a CTA at least
    size_t part_o, part_l, split, bytes;   // offsets
    int t_grid;                            // the tensor cores' CTAs (0: not launched)
    size_t t_part_o, t_part_l, t_split;
};

// A workspace lies at any multiple of 16 bytes; the tensor cores' parts are written 32 bytes a store.
constexpr size_t WS_ALIGN = 32;

static size_t add_bytes(size_t& at, size_t n) {
    const size_t here = at;
    at += (n + 255) & ~size_t(255);
    return here;
}

static ChunkPlan chunk_plan(const fs_paged_kv& c, int N, int R, int Hq, int width, int most, int sms) {
    ChunkPlan p = {};
    const int gs = Hq / c.num_heads, D = c.head_dim;
    // The most query rows that a request can have: all of them.
    const int64_t rows = int64_t(std::min(most, N)) * gs;
    const bool tensor = D <= 128 && rows > FEW;
    p.MT = rows <= FEW || tensor ? FEW : 64;
    p.KT = D == 256 && p.MT == 64 ? 32 : 64;
    // Two CTAs fit an SM (one with heads of 256); no more than there can be units.
    p.least = 2;
    const int64_t tiles = (int64_t(N) * gs + p.MT - 1) / p.MT + R;
    const int64_t units = tiles * c.num_heads * ((int64_t(width) * c.page_size + p.KT - 1) / p.KT + 2 + FEW_START);
    p.grid = int(std::max<int64_t>(1, std::min<int64_t>(int64_t(sms) * (D == 256 && p.MT == FEW ? 1 : 2), (units + p.least - 1) / p.least)));
    size_t at = 0;
    p.part_o = add_bytes(at, size_t(2) * p.grid * p.MT * D * 4);
    p.part_l = add_bytes(at, size_t(2) * p.grid * p.MT * 8);
    p.split = add_bytes(at, size_t(p.grid) * sizeof(int4));
    if (tensor) {
        // One CTA per SM.  A request of FEW rows or less has no tile there.
        const int64_t all = int64_t(N) * gs;
        const int64_t t_tiles = all / MANY + std::min<int64_t>(R, all / (FEW + 1) + 1);
        const int64_t t_units = t_tiles * c.num_heads * ((int64_t(width) * c.page_size + 127) / 128 + 4);
        p.t_grid = int(std::max<int64_t>(1, std::min<int64_t>(sms, t_units)));
        p.t_part_o = add_bytes(at, size_t(2) * p.t_grid * MANY * D * 4);
        p.t_part_l = add_bytes(at, size_t(2) * p.t_grid * MANY * 8);
        p.t_split = add_bytes(at, size_t(p.t_grid) * sizeof(int4));
    }
    p.bytes = at + WS_ALIGN - 16;    // (room to round a workspace's address up)
    return p;
}

template <typename T, int D, int MT, int WM, int WN, int RM, int KT>
static fs_status launch_rows(const ChunkArgs& a, void* stream) {
    const fs_status st = prepare_kernel(reinterpret_cast<const void*>(chunk_rows_kernel<T, D, MT, WM, WN, RM, KT>));
    if (st != FS_OK) return st;
    return launch_pdl(chunk_rows_kernel<T, D, MT, WM, WN, RM, KT>, dim3(unsigned(a.grid + (a.t_grid > 0))), 32 * WM * WN,
                      size_t(ChunkSmem<D, MT, KT>::TOTAL), stream, a);
}

template <typename T, int D>
static fs_status run_chunk(ChunkArgs& a, const ChunkPlan& p, int sms, int dtype, void* stream) {
    ChunkMaps maps = {};
    const bool mapped = chunk_maps(a, dtype, D, maps);
    fs_status st = FS_OK;
    if (a.t_grid > 0) st = launch_chunk_tensor(a, mapped ? &maps : nullptr, dtype, D, stream);
    if (st != FS_OK) return st;
    if (p.MT == FEW) st = mapped ? launch_chunk_few(a, maps, dtype, D, stream) : launch_rows<T, D, FEW, 1, 4, 1, 64>(a, stream);
    else if constexpr (D == 256) st = launch_rows<T, D, 64, 4, 1, 1, 32>(a, stream);
    else st = FS_ERR_INVALID_ARG;   // (heads of up to 128 go to the tensor cores)
    if (st != FS_OK) return st;
    const unsigned most = unsigned(a.grid * (p.MT / 16) + a.t_grid * (MANY / 16));
    return launch_pdl(join_chunk_kernel<T, D>, dim3(std::min(most, unsigned(JOIN_CTAS * sms))), 512,
                      size_t(a.grid + a.t_grid) * sizeof(JoinTile), stream, a, p.MT);
}

// The longest wait of the kernels for their own copies and products, in clock cycles.
static std::atomic<int64_t> wait_limit{PATIENCE};

static fs_status check_chunk(const fs_paged_kv* c, int N, int R, int Hq, int width, int most) {
    if (!c || N < 0 || R < 0 || Hq < 1 || width < 0 || most < 1) return FS_ERR_INVALID_ARG;
    if (c->num_pages < 0 || c->page_size < 1 || c->num_heads < 1 || c->head_dim < 1) return FS_ERR_INVALID_ARG;
    if (Hq % c->num_heads != 0) return FS_ERR_INVALID_ARG;
    if (c->dtype != FS_F32 && c->dtype != FS_BF16 && c->dtype != FS_F16) return FS_ERR_INVALID_ARG;
    if (c->dtype == FS_F32 || (c->head_dim != 64 && c->head_dim != 128 && c->head_dim != 256)) {
        set_last_error("chunk attention takes bf16 or f16 and heads of 64, 128 or 256");
        return FS_ERR_UNSUPPORTED;
    }
    const int64_t lim = 0x7fffffff - 4096;
    if (int64_t(N) * Hq > lim || int64_t(width) * c->page_size > lim) return FS_ERR_UNSUPPORTED;
    return FS_OK;
}

}  // namespace fsd

extern "C" {

fs_status fs_paged_chunk_attention_workspace_bytes(const fs_paged_kv* cache, int32_t tokens, int32_t requests,
                                                   int32_t q_heads, int32_t table_width, int32_t max_queries,
                                                   size_t* bytes) {
    using namespace fsd;
    if (!bytes) return FS_ERR_INVALID_ARG;
    fs_status st = check_chunk(cache, tokens, requests, q_heads, table_width, max_queries);
    if (st != FS_OK) return st;
    *bytes = 0;
    if (tokens == 0) return FS_OK;
    int sms = 0;
    size_t optin = 0;
    st = device_limits(sms, optin);
    if (st != FS_OK) return st;
    *bytes = chunk_plan(*cache, tokens, requests, q_heads, table_width, max_queries, sms).bytes;
    return FS_OK;
}

fs_status fs_paged_chunk_attention_wait_limit(int64_t cycles) {
    if (cycles < 0) return FS_ERR_INVALID_ARG;
    fsd::wait_limit.store(cycles, std::memory_order_relaxed);
    return FS_OK;
}

fs_status fs_paged_chunk_attention(const fs_paged_kv* cache, const void* query, const int64_t* query_strides,
                                   int32_t tokens, int32_t q_heads, const int32_t* page_table, int32_t requests,
                                   int32_t table_width, const int32_t* query_starts, const int32_t* lens,
                                   int32_t max_queries, int32_t window, int32_t sinks, float scale, int32_t zero_rest,
                                   void* out, const int64_t* out_strides, float* out_lse, void* workspace,
                                   size_t workspace_bytes, void* stream) {
    using namespace fsd;
    fs_status st = check_chunk(cache, tokens, requests, q_heads, table_width, max_queries);
    if (st != FS_OK) return st;
    if (window < 0 || sinks < 0 || (zero_rest != 0 && zero_rest != 1)) return FS_ERR_INVALID_ARG;
    if (tokens == 0) return FS_OK;
    if (!query || !query_strides || !out || !out_strides) return FS_ERR_INVALID_ARG;
    if (requests > 0 && (!query_starts || !lens || (table_width > 0 && !page_table))) return FS_ERR_INVALID_ARG;
    if (cache->num_pages > 0 && (!cache->k || !cache->v)) return FS_ERR_INVALID_ARG;
    ChunkArgs a = {};
    uintptr_t bits = reinterpret_cast<uintptr_t>(query) | reinterpret_cast<uintptr_t>(out) |
                     reinterpret_cast<uintptr_t>(cache->k) | reinterpret_cast<uintptr_t>(cache->v) |
                     reinterpret_cast<uintptr_t>(workspace);
    for (int i = 0; i < 3; ++i) {
        a.kc[i] = cache->k_strides[i];
        a.vc[i] = cache->v_strides[i];
        bits |= uintptr_t(a.kc[i] * 2) | uintptr_t(a.vc[i] * 2);
    }
    for (int i = 0; i < 2; ++i) {
        a.qs[i] = query_strides[i];
        a.os[i] = out_strides[i];
        bits |= uintptr_t(a.qs[i] * 2) | uintptr_t(a.os[i] * 2);
    }
    if (bits & 15) {
        set_last_error("chunk attention needs 16-byte aligned addresses and strides");
        return FS_ERR_INVALID_ARG;
    }
    int sms = 0;
    size_t optin = 0;
    st = device_limits(sms, optin);
    if (st != FS_OK) return st;
    const ChunkPlan p = chunk_plan(*cache, tokens, requests, q_heads, table_width, max_queries, sms);
    if (!workspace || workspace_bytes < p.bytes) {
        set_last_error("chunk attention: the workspace is too small");
        return FS_ERR_INVALID_ARG;
    }
    a.q = query;
    a.out = out;
    a.lse = out_lse;
    a.k = cache->num_pages > 0 ? cache->k : query;   // (without pages an address that nothing is read from)
    a.v = cache->num_pages > 0 ? cache->v : query;
    a.num_pages = cache->num_pages;
    a.page_size = cache->page_size;
    a.page_shift = -1;
    for (int s = 0; s < 31; ++s)
        if (cache->page_size == (1 << s)) a.page_shift = s;
    a.table = page_table;
    a.starts = query_starts;
    a.lens = lens;
    a.R = requests;
    a.width = table_width;
    a.N = tokens;
    a.Hq = q_heads;
    a.Hkv = cache->num_heads;
    a.gs = q_heads / cache->num_heads;
    a.window = window == 0 ? 0x7fffffff : window;
    a.sinks = window == 0 ? 0 : sinks;
    a.scale = scale * 1.44269504088896341f;
    a.zero_rest = zero_rest;
    a.patience = wait_limit.load(std::memory_order_relaxed);
    a.rows_upto = p.t_grid > 0 ? FEW : 0x7fffffff;
    a.grid = p.grid;
    a.least = p.least;
    unsigned char* ws = reinterpret_cast<unsigned char*>((reinterpret_cast<uintptr_t>(workspace) + WS_ALIGN - 1) & ~uintptr_t(WS_ALIGN - 1));
    a.part_o = reinterpret_cast<float*>(ws + p.part_o);
    a.part_l = reinterpret_cast<float2*>(ws + p.part_l);
    a.split = reinterpret_cast<int4*>(ws + p.split);
    a.t_grid = p.t_grid;
    a.t_start = cache->head_dim == 64 ? 2 : 3;   // (about 5000 and 8200 cycles, of 2150 and 2860 a unit)
    a.out_32 = (reinterpret_cast<uintptr_t>(out) % 32 == 0 && a.os[0] % 16 == 0 && a.os[1] % 16 == 0);
    if (p.t_grid > 0) {
        a.t_part_o = reinterpret_cast<float*>(ws + p.t_part_o);
        a.t_part_l = reinterpret_cast<float2*>(ws + p.t_part_l);
        a.t_split = reinterpret_cast<int4*>(ws + p.t_split);
    }
    const int D = cache->head_dim, dt = cache->dtype;
    if (dt == FS_BF16)
        return D == 64    ? run_chunk<__nv_bfloat16, 64>(a, p, sms, dt, stream)
               : D == 128 ? run_chunk<__nv_bfloat16, 128>(a, p, sms, dt, stream)
                          : run_chunk<__nv_bfloat16, 256>(a, p, sms, dt, stream);
    return D == 64    ? run_chunk<__half, 64>(a, p, sms, dt, stream)
           : D == 128 ? run_chunk<__half, 128>(a, p, sms, dt, stream)
                      : run_chunk<__half, 256>(a, p, sms, dt, stream);
}

}  // extern "C"
