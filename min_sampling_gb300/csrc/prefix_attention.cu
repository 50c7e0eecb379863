// Attention of a batch that shares a long prefix, over a paged key/value cache (sm_103a).
//
// For a query q of row b (head h, key/value head h / group size):
//   out = softmax(scale * q [Kp; Ks]^T) [Vp; Vs],
// Kp, Vp the prefix of b's group, Ks, Vs the row's own suffix.  The prefix's part is
// computed once for all queries of a group: its keys and values are read once per tile
// of queries instead of once per row.  The parts, over any split of the keys, are joined
// by their maxima and sums:
//   m = max_i m_i,  l = sum_i 2^(m_i - m) l_i,  out = sum_i 2^(m_i - m) l_i out_i / l.
//
// prefix_tensor.cu: the prefix's part where a group has many queries.
// attend_kernel: one CTA per (tile of queries, key/value head, range of keys), of the
// suffixes and of small groups' prefixes in one launch; scores, running maximum, sum and output stay
// in registers.  join_kernel: one CTA per query joins the parts in a fixed order (no
// atomics, the same result on every run).
#include "attention.cuh"

#include <type_traits>

namespace fsd {

constexpr int ASTAGES = 2;    // tiles of keys and values in flight

__device__ __forceinline__ void ldsm4(uint32_t (&r)[4], uint32_t addr) {
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0,%1,%2,%3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]) : "r"(addr));
}
__device__ __forceinline__ void ldsm4_t(uint32_t (&r)[4], uint32_t addr) {
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0,%1,%2,%3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]) : "r"(addr));
}
// Byte offset of 16-byte chunk c of row r in a tile of D 16-bit values a row: chunks are
// permuted within each row by its index, so that the eight rows of a matrix fragment fall
// into different banks.
template <int D>
__device__ __forceinline__ uint32_t chunk_at(int r, int c) { return uint32_t(r * (D * 2) + ((c ^ (r & 7)) << 4)); }

// ------------------------------------------------------------------ parts

// Shared memory: queries, then ASTAGES x (keys, values), then two slots of row offsets.
template <int D, int MT, int KT>
struct AttnSmem {
    static constexpr int Q = 0;
    static constexpr int TILE = KT * D * 2;
    static constexpr int KV = MT * D * 2;
    static constexpr int OFF = KV + ASTAGES * 2 * TILE;
    static constexpr int TOTAL = OFF + 2 * 2 * KT * 8 + 16;
    static constexpr int MERGE = 0;  // the warps' parts at the end, over everything before OFF
};

// WM x WN warps over a tile of MT = 16 RM WM queries and KT keys; each warp keeps its own
// running maximum, sum and output over its share of the keys.  Bound by the reads of keys and
// values; what it loses are the ends of its short ranges (look-ups, first tile, joining the
// warps): 256 rows of up to 512 keys, 8 heads of 128, 62 us, 4.3 TB/s; one row of 64000 keys 55 us, 4.8.
// Two warps and tiles of 32 keys, six CTAs on an SM instead of three, were slower (64 rows of
// 1000 keys 54.7 -> 64.7 us): a tile's chain of instructions, not its load, sets its time.
template <typename T, int D, int MT, int WM, int WN, int RM, int KT>
__global__ void __launch_bounds__(32 * WM * WN) attend_kernel(const AttnArgs a) {
    constexpr int ANT = 32 * WM * WN;
    static_assert(MT == 16 * RM * WM && KT <= ANT && RANGE % KT == 0, "warp layout");
    using S = AttnSmem<D, MT, KT>;
    constexpr int KW = KT / WN;       // keys per warp and tile
    constexpr int NF = KW / 8;        // score fragments
    constexpr int DC = D / 8;         // 16-byte chunks per row
    constexpr float UP = std::is_same<T, __half>::value ? 32768.f : 1.f;   // the weights' factor in the product
    static_assert(WN * MT * (D + 2) * 4 <= S::OFF, "the warps' parts fit where the tiles were");
    extern __shared__ __align__(128) unsigned char smem[];
    const uint32_t sbase = smem_u32(smem);
    int64_t* soff = reinterpret_cast<int64_t*>(smem + S::OFF);  // [2][2][KT]
    int* poison = reinterpret_cast<int*>(smem + S::OFF + 2 * 2 * KT * 8);  // a page that does not exist
    int* odd_seen = poison + 1;                                            // infinite or NaN values taken out
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int wm = warp / WN, wn = warp % WN;
    // When finishing, the launch before is the prefix's own: what that one waited for is there, and its
    // parts are waited for at the end, so that suffixes run where and as soon as it leaves room.
    if (!a.finish) grid_dependency_wait();
    allow_dependents();

    // ---- this CTA's queries and keys
    int item = blockIdx.x;
    const int np = a.ptiles * a.Hkv * a.SP;
    const bool pre = item < np;
    int head, split, b0, M, row0, len, begin, slot, page0 = -1;
    bool early = false;
    const int* table;
    if (pre) {
        const int tile = item % a.ptiles;
        item /= a.ptiles;
        head = item % a.Hkv;
        split = item / a.Hkv;
        const GroupTile gt = group_tile<MT>(a, tile, lane);
        if (gt.g < 0) return;
        b0 = gt.b0;
        M = (gt.b1 - b0) * a.Q * a.gs;
        row0 = gt.tile * MT;
        len = gt.len;
        const int step = range_len(len, a.SP);
        begin = split * step;
        if (begin >= len) return;
        len = min(len, begin + step);
        table = a.ptab + int64_t(gt.g) * a.pw;
        slot = split;
    } else {
        item -= np;
        head = item % a.Hkv;
        item /= a.Hkv;
        split = item % a.SS;
        item /= a.SS;
        const int tile = item % a.stiles;
        b0 = item / a.stiles;
        M = a.Q * a.gs;
        row0 = tile * MT;
        table = a.stab + int64_t(b0) * a.sw;
        // One range starts at the first key whatever the length: its first pages are read beside the length.
        early = a.SS == 1;
        if (early && tid < KT) {
            const int pi = a.page_shift >= 0 ? tid >> a.page_shift : tid / a.page_size;
            if (pi < a.sw) page0 = table[pi];
        }
        len = suffix_len(a, b0);
        const int step = range_len(len, a.SS);
        begin = split * step;
        if (begin >= len && !a.finish) return;
        slot = a.SP + split;
    }
    const int full = pre ? len : suffix_len(a, b0);          // the row's whole suffix
    const int end = pre ? len : min(len, begin + range_len(len, a.SS));
    const int tiles = (end - begin + KT - 1) / KT;   // 0: only when finishing

    // Query r of the tile: row b0 + r / (Q gs), query token, head; -1 past the last.
    auto query_at = [&](int r, int& b, int& qi, int& h) {
        const int per = a.Q * a.gs;
        b = b0 + r / per;
        const int rem = r % per;
        qi = rem / a.gs;
        h = head * a.gs + rem % a.gs;
    };
    if (tid == 0) *poison = 0, *odd_seen = 0;
    for (int i = tid; i < MT * DC; i += ANT) {
        const int r = i / DC, c = i % DC;
        int b = 0, qi = 0, h = 0;
        const bool on = row0 + r < M;
        if (on) query_at(row0 + r, b, qi, h);
        cp16(sbase + S::Q + chunk_at<D>(r, c),
             static_cast<const T*>(a.q) + b * a.qs[0] + qi * a.qs[1] + h * a.qs[2] + c * 8, on);
    }

    // ---- pipeline of key/value tiles.  A key's offsets are looked up one tile before its
    // loads are issued, by one thread per key.
    auto look_up = [&](int tile, int64_t& ko, int64_t& vo, bool& bad) {
        ko = vo = NOWHERE;
        bad = false;
        const int key = begin + tile * KT + tid;
        if (tid < KT && key < end) {
            const int pi = a.page_shift >= 0 ? key >> a.page_shift : key / a.page_size;
            const int page = tile == 0 && early ? page0 : table[pi];
            if (page >= 0 && page < a.num_pages) {
                const int s = key - pi * a.page_size;
                ko = page * a.kc[0] + s * a.kc[1] + head * a.kc[2];
                vo = page * a.vc[0] + s * a.vc[1] + head * a.vc[2];
            } else {
                bad = true;
            }
        }
    };
    auto put_offsets = [&](int tile, int64_t ko, int64_t vo, bool bad) {
        if (tid < KT) {
            soff[(tile & 1) * 2 * KT + tid] = ko;
            soff[(tile & 1) * 2 * KT + KT + tid] = vo;
        }
        if (bad) *poison = 1;
    };
    auto issue = [&](int tile) {
        const int64_t* off = soff + (tile & 1) * 2 * KT;
        const uint32_t kd = sbase + S::KV + (tile % ASTAGES) * 2 * S::TILE;
#pragma unroll
        for (int i = 0; i < KT * DC / ANT; ++i) {
            const int r = (tid + i * ANT) / DC, c = (tid + i * ANT) % DC;
            const int64_t ko = off[r], vo = off[KT + r];
            const bool on = ko != NOWHERE;
            cp16(kd + chunk_at<D>(r, c), static_cast<const T*>(a.k) + (on ? ko + c * 8 : 0), on);
            cp16(kd + S::TILE + chunk_at<D>(r, c), static_cast<const T*>(a.v) + (on ? vo + c * 8 : 0), on);
        }
    };
    int64_t ko, vo;
    bool bad;
    __syncthreads();  // poison is clear
#pragma unroll
    for (int t = 0; t < ASTAGES - 1; ++t) {
        look_up(t, ko, vo, bad);
        put_offsets(t, ko, vo, bad);
        __syncthreads();
        if (t < tiles) issue(t);
        cp_async_commit();
    }
    look_up(ASTAGES - 1, ko, vo, bad);
    put_offsets(ASTAGES - 1, ko, vo, bad);
    int parts = 0;      // of the prefix, to be joined here
    if (a.finish) {
        const int g = group_of(a, b0, lane);
        if (g >= 0) {
            const int plen = prefix_len(a, g);
            if (plen > 0) { const int pstep = range_len(plen, a.SP); parts = (plen + pstep - 1) / pstep; }
        }
    }

    float o[RM][D / 8][4];
    float mrow[RM][2], lrow[RM][2];
    int limit[RM][2];
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
            // keys this query sees: all of the prefix; of the suffix, up to its own position
            const int r = row0 + (wm * RM + i) * 16 + j * 8 + (lane >> 2);
            int b, qi, h;
            query_at(r, b, qi, h);
            limit[i][j] = pre ? end : min(end, full - (a.Q - 1 - qi));
        }
    }
    const int qrow = (wm * RM) * 16 + (lane & 15), qch = lane >> 4;

#pragma unroll 1
    for (int t = 0; t < tiles; ++t) {
        cp_async_wait<ASTAGES - 2>();
        __syncthreads();  // tile t is there, tile t - 1 is done with, the next offsets are written
        if (t + ASTAGES - 1 < tiles) issue(t + ASTAGES - 1);
        cp_async_commit();
        look_up(t + ASTAGES, ko, vo, bad);
        const uint32_t ks = sbase + S::KV + (t % ASTAGES) * 2 * S::TILE, vs = ks + S::TILE;
        // A value that only some of the queries see may be infinite or NaN, which a weight of
        // zero does not cancel: such values are taken out of the tile, and added at the end to the
        // outputs of the queries that see them.
        const int k0 = begin + t * KT;
        if (!pre && a.Q > 1 && k0 + KT > full - (a.Q - 1)) {
            const int lo = max(0, full - (a.Q - 1) - k0), hi = min(KT, end - k0);
            unsigned char* vb = smem + S::KV + (t % ASTAGES) * 2 * S::TILE + S::TILE;
            bool odd = false;
            for (int i = tid; i < (hi - lo) * D; i += ANT) {
                const int r = lo + i / D, d = i % D;
                const float x = Mma<T>::get(*reinterpret_cast<const T*>(vb + chunk_at<D>(r, d >> 3) + (d & 7) * 2));
                odd |= !(fabsf(x) <= 3.402823466e38f);
            }
            if (__syncthreads_or(odd)) {
                if (tid == 0) *odd_seen = 1;
                for (int i = tid; i < (hi - lo) * D; i += ANT) {
                    const int r = lo + i / D, d = i % D;
                    T* p = reinterpret_cast<T*>(vb + chunk_at<D>(r, d >> 3) + (d & 7) * 2);
                    if (!(fabsf(Mma<T>::get(*p)) <= 3.402823466e38f)) *p = Mma<T>::put(0.f);
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
            for (int i = 0; i < RM; ++i) ldsm4(af[i], sbase + S::Q + chunk_at<D>(qrow + i * 16, kk * 2 + qch));
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
        uint32_t pf[RM][NF / 2][4];
#pragma unroll
        for (int i = 0; i < RM; ++i) {
#pragma unroll
            for (int j = 0; j < 2; ++j) {
                const int lim = limit[i][j] - kbase;
                float mx = -INFINITY;
#pragma unroll
                for (int f = 0; f < NF; ++f)
#pragma unroll
                    for (int e = 0; e < 2; ++e) {
                        float& x = s[i][f][j * 2 + e];
                        x = f * 8 + e < lim ? x * a.scale : -INFINITY;
                        mx = fmaxf(mx, x);
                    }
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
                        float& x = s[i][f][j * 2 + e];
                        x = exp2_fast(x - ms);
                        sum += x;
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
            // step of the type; their sum stays in 32.  In f16 they are 2^15 larger: half a step down to 2^-29 of the
            // maximum, 2^-40 of it below.
            auto weights = [&](int f, int e) {
                return Mma<T>::pack(s[i][f][e] * UP, s[i][f][e + 1] * UP);
            };
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
        put_offsets(t + ASTAGES, ko, vo, bad);
    }

    // ---- the warps' parts joined through shared memory, written as this CTA's part
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
    const float nan = *poison ? __int_as_float(0x7fffffff) : 0.f;
    const bool add_odd = a.Q > 1 && *odd_seen;
    const int64_t rows = int64_t(a.B) * a.Q * a.Hq;
    if (a.finish) grid_dependency_wait();
    for (int i = tid; i < MT * (D / 4); i += ANT) {
        const int r = i / (D / 4), c = i % (D / 4);
        if (row0 + r >= M) continue;
        int b, qi, h;
        query_at(row0 + r, b, qi, h);
        const int64_t row = (int64_t(b) * a.Q + qi) * a.Hq + h;
        float m = -INFINITY;
#pragma unroll
        for (int w = 0; w < WN; ++w) m = fmaxf(m, sm[w * MT + r]);
#pragma unroll 8
        for (int s = 0; s < parts; ++s) m = fmaxf(m, a.part_l[s * rows + row]);
        const float ms = m == -INFINITY ? 0.f : m;
        float l = 0.f;
        float4 x = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
        for (int w = 0; w < WN; ++w) {
            const float f = exp2_fast(sm[w * MT + r] - ms);
            const float4 y = *reinterpret_cast<const float4*>(so + (w * MT + r) * D + c * 4);
            l += f * sl[w * MT + r];
            x.x += f * y.x, x.y += f * y.y, x.z += f * y.z, x.w += f * y.w;
        }
#pragma unroll 4
        for (int s = 0; s < parts; ++s) {
            const float f = exp2f(a.part_l[s * rows + row] - ms);
            const float4 y = *reinterpret_cast<const float4*>(a.part_o + (s * rows + row) * D + c * 4);
            l += f;
            x.x += f * y.x, x.y += f * y.y, x.z += f * y.z, x.w += f * y.w;
        }
        const float inv = (l == 0.f ? 0.f : 1.f / l) + nan;
        const float lse = (l == 0.f ? -INFINITY : m + log2f(l)) + nan;
        x = make_float4(x.x * inv, x.y * inv, x.z * inv, x.w * inv);
        if (add_odd) {   // (their weights are positive: exp(s - m) > 0)
            const int last = min(end, full - (a.Q - 1 - qi));
            for (int key = max(begin, full - (a.Q - 1)); key < last; ++key) {
                const int pi = key / a.page_size, page = table[pi];
                if (page < 0 || page >= a.num_pages) continue;
                const T* v = static_cast<const T*>(a.v) + page * a.vc[0] + (key - pi * a.page_size) * a.vc[1] + head * a.vc[2] + c * 4;
                auto odd = [&](int e) {
                    const float y = Mma<T>::get(v[e]);
                    return fabsf(y) <= 3.402823466e38f ? 0.f : y;
                };
                x = make_float4(x.x + odd(0), x.y + odd(1), x.z + odd(2), x.w + odd(3));
            }
        }
        if (a.finish) {
            T* out = static_cast<T*>(a.out) + b * a.os[0] + qi * a.os[1] + h * a.os[2] + c * 4;
            *reinterpret_cast<uint2*>(out) = make_uint2(Mma<T>::pack(x.x, x.y), Mma<T>::pack(x.z, x.w));
            if (c == 0 && a.lse) a.lse[row] = lse * 0.693147180559945309f;
        } else {
            const int64_t at = slot * rows + row;
            *reinterpret_cast<float4*>(a.part_o + at * D + c * 4) = x;
            if (c == 0) a.part_l[at] = lse;
        }
    }
}

// ------------------------------------------------------------------ the parts joined

template <int E>
struct alignas(E >= 4 ? 16 : E * 4) Run {
    float v[E];
};

// One CTA of four warps per query: the warps take the parts in turn, each lane E neighbouring
// elements; the warps' sums are added in order.
template <typename T, int D>
__global__ void __launch_bounds__(128) join_kernel(const AttnArgs a) {
    constexpr int E = D / 32, W = 4;
    __shared__ float so[W][D], sl[W];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    grid_dependency_wait();
    allow_dependents();
    const int64_t rows = int64_t(a.B) * a.Q * a.Hq;
    const int row = blockIdx.x;
    const int h = row % a.Hq, qi = row / a.Hq % a.Q, b = row / a.Hq / a.Q;
    const int g = group_of(a, b, lane);
    int n0 = 0, n1 = 0;  // parts of the prefix, of the suffix
    if (g >= 0) {
        const int len = prefix_len(a, g);
        if (len > 0) { const int step = range_len(len, a.SP); n0 = (len + step - 1) / step; }
    }
    {
        const int len = suffix_len(a, b);
        if (len > 0) { const int step = range_len(len, a.SS); n1 = (len + step - 1) / step; }
    }
    const int n = n0 + n1;
    auto slot = [&](int i) { return int64_t(i < n0 ? i : a.SP + i - n0) * rows + row; };
    // (a NaN part makes the maximum's users NaN through its own weight)
    float m = -INFINITY;
    for (int i = lane; i < n; i += 32) m = fmaxf(m, a.part_l[slot(i)]);
#pragma unroll
    for (int s = 16; s > 0; s >>= 1) m = fmaxf(m, __shfl_xor_sync(FULL, m, s));
    const float ms = m == -INFINITY ? 0.f : m;
    float l = 0.f, x[E];
#pragma unroll
    for (int e = 0; e < E; ++e) x[e] = 0.f;
#pragma unroll 4
    for (int i = warp; i < n; i += W) {
        const int64_t at = slot(i);
        const float f = exp2f(a.part_l[at] - ms);
        Run<E> y = *reinterpret_cast<const Run<E>*>(a.part_o + at * D + lane * E);
        l += f;
#pragma unroll
        for (int e = 0; e < E; ++e) x[e] += f * y.v[e];
    }
#pragma unroll
    for (int e = 0; e < E; ++e) so[warp][lane * E + e] = x[e];
    if (lane == 0) sl[warp] = l;
    __syncthreads();
    l = 0.f;
#pragma unroll
    for (int w = 0; w < W; ++w) l += sl[w];
    const float inv = l == 0.f ? 0.f : 1.f / l;
    T* out = static_cast<T*>(a.out) + b * a.os[0] + qi * a.os[1] + h * a.os[2];
    for (int i = threadIdx.x * 2; i < D; i += 256) {
        float y0 = 0.f, y1 = 0.f;
#pragma unroll
        for (int w = 0; w < W; ++w) y0 += so[w][i], y1 += so[w][i + 1];
        *reinterpret_cast<uint32_t*>(out + i) = Mma<T>::pack(y0 * inv, y1 * inv);
    }
    if (a.lse && threadIdx.x == 0) a.lse[row] = (l == 0.f ? -INFINITY : m + log2f(l)) * 0.693147180559945309f;
}

// ------------------------------------------------------------------ host

template <typename K>
static fs_status launch_pdl(K kernel, unsigned grid, unsigned block, size_t smem, void* stream, const AttnArgs& a) {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(grid, 1, 1);
    cfg.blockDim = dim3(block, 1, 1);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = static_cast<cudaStream_t>(stream);
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    const cudaError_t e = cudaLaunchKernelEx(&cfg, kernel, a);
    return e == cudaSuccess ? FS_OK : cuda_fail(e);
}

// Queries per tile of attend_kernel: the smallest tile that holds `per` queries, so that keys are read once.
static int tile_rows(int64_t per) { return per <= 16 ? 16 : (per <= 32 ? 32 : 64); }

struct AttnPlan {
    int MT, SP, SS, ptiles, stiles;
    int tensor;     // queries per tile on the tensor cores, 0: the prefix runs in attend_kernel
    size_t bytes;
};

// The lengths are on the device, so the plan goes by the most that the tables can name.
static AttnPlan attn_plan(int B, int Q, int Hq, int Hkv, int D, int G, int64_t max_prefix, int64_t max_suffix, int sms) {
    AttnPlan p;
    const int gs = Hq / Hkv;
    const int64_t all = int64_t(B) * Q * gs, per = G > 0 ? all / G : 0;
    const bool prefix = G > 0 && max_prefix > 0;
    // From 33 queries on: 36 over 512 / 2048 / 32768 keys take 15.5 / 18.6 / 71.5 us in attend_kernel and
    // 11.6 / 13.0 / 37.8 there (8 heads of 128); 32 still fit one tile of attend_kernel, 12.7 / 15.0 / 43.7.
    p.tensor = prefix && D <= 128 && per > 32 && max_prefix >= 512 ? (per > 128 ? 256 : 128) : 0;
    p.MT = tile_rows(prefix && !p.tensor ? per : int64_t(Q) * gs);
    const int rows = p.tensor ? p.tensor : p.MT;
    // the most tiles that `all` queries in G groups can take
    p.ptiles = prefix ? int(std::min<int64_t>(all, (all + int64_t(G) * (rows - 1)) / rows)) : 0;
    p.stiles = max_suffix > 0 ? int((int64_t(Q) * gs + p.MT - 1) / p.MT) : 0;
    // Key ranges in attend_kernel: about three CTAs for every SM, no range shorter than 128 keys (of 64,
    // 128 and 256, 128 was the fastest for one to eight rows over 256 to 64000 keys).
    auto splits = [&](int64_t items, int64_t len) {
        if (items == 0 || len <= 0) return int64_t(0);
        const int64_t by_len = (len + 2 * RANGE - 1) / (2 * RANGE);
        return std::max<int64_t>(1, std::min<int64_t>({(int64_t(sms) * 3 + items - 1) / items, by_len, 256}));
    };
    p.SP = int(splits(int64_t(p.ptiles) * Hkv, max_prefix));
    if (p.tensor) {
        // One CTA per SM: the number of ranges that takes the least time in whole waves, a
        // range's start and end counted as four tiles.
        const int64_t items = int64_t(p.ptiles) * Hkv, n = (max_prefix + 127) / 128;
        int64_t best = INT64_MAX;
        for (int64_t s = 1; s <= std::min<int64_t>(n, 64); ++s) {
            const int64_t cost = (items * s + sms - 1) / sms * ((n + s - 1) / s + 4);
            if (cost < best) best = cost, p.SP = int(s);
        }
    }
    p.SS = int(splits(int64_t(B) * p.stiles * Hkv, max_suffix));
    // Behind the prefix's own launch a suffix of one range is joined where it is computed, which
    // saves a launch: 48 rows of up to 700 keys 53.7 -> 43.9 us, 16 of 300 66.3 -> 62.5; but 16 of
    // 1000 28.2 -> 34.5, so not where the ranges shorten it by more than that.
    if (p.tensor && (max_suffix <= 5 * RANGE || (p.SS <= 2 && max_suffix <= 16 * RANGE))) p.SS = std::min(p.SS, 1);
    p.bytes = size_t(p.SP + p.SS) * size_t(B) * Q * Hq * (size_t(D) + 1) * 4;
    return p;
}

template <typename T, int D, int MT, int WM, int WN, int RM, int KT>
static fs_status launch_attend(const AttnArgs& a, unsigned grid, void* stream) {
    const void* fn = reinterpret_cast<const void*>(attend_kernel<T, D, MT, WM, WN, RM, KT>);
    const fs_status st = prepare_kernel(fn);
    if (st != FS_OK) return st;
    return launch_pdl(attend_kernel<T, D, MT, WM, WN, RM, KT>, grid, 32 * WM * WN, size_t(AttnSmem<D, MT, KT>::TOTAL), stream, a);
}

template <typename T, int D>
static fs_status run_attention(AttnArgs& a, const AttnPlan& p, int dtype, int sms, void* stream) {
    const int64_t pre = int64_t(p.ptiles) * a.Hkv * p.SP;
    const int64_t items = (p.tensor ? 0 : pre) + int64_t(a.B) * p.stiles * a.Hkv * p.SS;
    if (items > 0x7fffffffLL || pre > 0x7fffffffLL) return FS_ERR_UNSUPPORTED;
    fs_status st = FS_OK;
    if (p.tensor) {
        st = launch_prefix_tensor(a, dtype, D, p.tensor, stream);
        if (st != FS_OK) return st;
        a.ptiles = 0;
        a.finish = p.SS == 1;
    }
    if (items > 0) {
        if constexpr (D <= 128) {
            if (p.MT == 16) st = launch_attend<T, D, 16, 1, 4, 1, 64>(a, unsigned(items), stream);
            else if (p.MT == 32) st = launch_attend<T, D, 32, 2, 2, 1, 64>(a, unsigned(items), stream);
            else st = launch_attend<T, D, 64, 2, 2, 2, 64>(a, unsigned(items), stream);
        } else {
            // Tiles of 64 keys of 256 leave room for one CTA on an SM, of 32 keys for two or three: 64 rows
            // with 700 keys of their own behind 4096 166.8 -> 131.5 us, one row of 32768 keys 78.3 -> 56.6.
            // While every CTA has an SM to itself the longer tiles are ahead (one row of 512 keys 11.4, 14.0
            // with tiles of 32); with 64 queries a tile the two were even there.
            const bool alone = items <= sms;
            if (p.MT == 16 && alone) st = launch_attend<T, D, 16, 1, 4, 1, 64>(a, unsigned(items), stream);
            else if (p.MT == 16) st = launch_attend<T, D, 16, 1, 2, 1, 32>(a, unsigned(items), stream);
            else if (p.MT == 32 && alone) st = launch_attend<T, D, 32, 2, 2, 1, 64>(a, unsigned(items), stream);
            else if (p.MT == 32) st = launch_attend<T, D, 32, 2, 2, 1, 32>(a, unsigned(items), stream);
            else st = launch_attend<T, D, 64, 4, 1, 1, 32>(a, unsigned(items), stream);
        }
        if (st != FS_OK || a.finish) return st;
    }
    const int64_t rows = int64_t(a.B) * a.Q * a.Hq;
    return launch_pdl(join_kernel<T, D>, unsigned(rows), 128, 0, stream, a);
}

static fs_status check_shape(const fs_paged_kv* c, int B, int Q, int Hq, int G, int pw, int sw) {
    if (!c || B < 0 || Q < 1 || Hq < 1 || G < 0 || pw < 0 || sw < 0) return FS_ERR_INVALID_ARG;
    if (c->num_pages < 0 || c->page_size < 1 || c->num_heads < 1 || c->head_dim < 1) return FS_ERR_INVALID_ARG;
    if (Hq % c->num_heads != 0) return FS_ERR_INVALID_ARG;
    if (c->dtype != FS_F32 && c->dtype != FS_BF16 && c->dtype != FS_F16) return FS_ERR_INVALID_ARG;
    if (c->dtype == FS_F32 || (c->head_dim != 64 && c->head_dim != 128 && c->head_dim != 256)) {
        set_last_error("shared-prefix attention takes bf16 or f16 and heads of 64, 128 or 256");
        return FS_ERR_UNSUPPORTED;
    }
    const int64_t lim = 0x7fffffff - 4096;
    if (int64_t(B) * Q * Hq > lim || int64_t(pw) * c->page_size > lim || int64_t(sw) * c->page_size > lim)
        return FS_ERR_UNSUPPORTED;
    return FS_OK;
}

}  // namespace fsd

extern "C" {

fs_status fs_shared_prefix_attention_workspace_bytes(const fs_paged_kv* cache, int32_t batch, int32_t queries,
                                                     int32_t q_heads, int32_t groups, int32_t prefix_width,
                                                     int32_t suffix_width, size_t* bytes) {
    using namespace fsd;
    if (!bytes) return FS_ERR_INVALID_ARG;
    fs_status st = check_shape(cache, batch, queries, q_heads, groups, prefix_width, suffix_width);
    if (st != FS_OK) return st;
    *bytes = 0;
    if (batch == 0) return FS_OK;
    int sms = 0;
    size_t optin = 0;
    st = device_limits(sms, optin);
    if (st != FS_OK) return st;
    *bytes = attn_plan(batch, queries, q_heads, cache->num_heads, cache->head_dim, groups,
                       int64_t(prefix_width) * cache->page_size, int64_t(suffix_width) * cache->page_size, sms).bytes;
    return FS_OK;
}

fs_status fs_shared_prefix_attention(const fs_paged_kv* cache, const void* query, const int64_t* query_strides,
                                     int32_t batch, int32_t queries, int32_t q_heads, const int32_t* group_starts,
                                     int32_t groups, const int32_t* prefix_table, int32_t prefix_width,
                                     const int32_t* prefix_lens, const int32_t* suffix_table, int32_t suffix_width,
                                     const int32_t* suffix_lens, float scale, void* out, const int64_t* out_strides,
                                     float* out_lse, void* workspace, size_t workspace_bytes, void* stream) {
    using namespace fsd;
    fs_status st = check_shape(cache, batch, queries, q_heads, groups, prefix_width, suffix_width);
    if (st != FS_OK) return st;
    if (!group_starts && groups > 1) return FS_ERR_INVALID_ARG;
    if (batch == 0) return FS_OK;
    if (!query || !query_strides || !out || !out_strides) return FS_ERR_INVALID_ARG;
    if (groups > 0 && (!prefix_lens || (prefix_width > 0 && !prefix_table))) return FS_ERR_INVALID_ARG;
    if (!suffix_lens || (suffix_width > 0 && !suffix_table)) return FS_ERR_INVALID_ARG;
    if (cache->num_pages > 0 && (!cache->k || !cache->v)) return FS_ERR_INVALID_ARG;
    AttnArgs a = {};
    uintptr_t bits = reinterpret_cast<uintptr_t>(query) | reinterpret_cast<uintptr_t>(out) |
                     reinterpret_cast<uintptr_t>(cache->k) | reinterpret_cast<uintptr_t>(cache->v) |
                     reinterpret_cast<uintptr_t>(workspace);
    for (int i = 0; i < 3; ++i) {
        a.qs[i] = query_strides[i];
        a.os[i] = out_strides[i];
        a.kc[i] = cache->k_strides[i];
        a.vc[i] = cache->v_strides[i];
        bits |= uintptr_t(a.qs[i] * 2) | uintptr_t(a.os[i] * 2) | uintptr_t(a.kc[i] * 2) | uintptr_t(a.vc[i] * 2);
    }
    if (bits & 15) {
        set_last_error("shared-prefix attention needs 16-byte aligned addresses and strides");
        return FS_ERR_INVALID_ARG;
    }
    int sms = 0;
    size_t optin = 0;
    st = device_limits(sms, optin);
    if (st != FS_OK) return st;
    const int64_t maxp = int64_t(prefix_width) * cache->page_size, maxs = int64_t(suffix_width) * cache->page_size;
    const AttnPlan p = attn_plan(batch, queries, q_heads, cache->num_heads, cache->head_dim, groups, maxp, maxs, sms);
    if (p.bytes > 0 && (!workspace || workspace_bytes < p.bytes)) {
        set_last_error("shared-prefix attention: the workspace is too small");
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
    a.ptab = prefix_table;
    a.plens = prefix_lens;
    a.starts = group_starts;
    a.G = groups;
    a.pw = prefix_width;
    a.stab = suffix_table;
    a.slens = suffix_lens;
    a.sw = suffix_width;
    a.B = batch;
    a.Q = queries;
    a.Hq = q_heads;
    a.Hkv = cache->num_heads;
    a.gs = q_heads / cache->num_heads;
    a.scale = scale * 1.44269504088896341f;
    a.SP = p.SP;
    a.SS = p.SS;
    a.ptiles = p.ptiles;
    a.stiles = p.stiles;
    a.part_o = static_cast<float*>(workspace);
    a.part_l = a.part_o + size_t(p.SP + p.SS) * batch * queries * q_heads * cache->head_dim;
    const int D = cache->head_dim;
    if (cache->dtype == FS_BF16)
        return D == 64    ? run_attention<__nv_bfloat16, 64>(a, p, FS_BF16, sms, stream)
               : D == 128 ? run_attention<__nv_bfloat16, 128>(a, p, FS_BF16, sms, stream)
                          : run_attention<__nv_bfloat16, 256>(a, p, FS_BF16, sms, stream);
    return D == 64    ? run_attention<__half, 64>(a, p, FS_F16, sms, stream)
           : D == 128 ? run_attention<__half, 128>(a, p, FS_F16, sms, stream)
                      : run_attention<__half, 256>(a, p, FS_F16, sms, stream);
}

}  // extern "C"
