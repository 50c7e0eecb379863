// What the kernels of chunk attention have in common: arguments, the requests' query tiles and
// the keys that a tile sees.
#pragma once

#include <type_traits>

#include "attention.cuh"

namespace fsd {

constexpr int FEW = 16;         // query rows that a tile of chunk_few_kernel holds beside the tensor cores' tiles
constexpr int MANY = 256;       // query rows of a tensor-core tile
constexpr int FEW_START = 2;    // key tiles of 64 that start and end of such a tile take as long as

struct ChunkArgs {
    const void* q;
    void* out;
    float* lse;                 // [N][Hq], nullable
    int64_t qs[2], os[2];       // strides: token, head
    const void* k;
    const void* v;
    int64_t kc[3], vc[3];       // strides: page, slot, head
    int num_pages, page_size, page_shift;  // page_shift: log2(page_size), -1 when it is no power of two
    const int* table;           // [R][width]
    const int* starts;          // [R + 1]
    const int* lens;            // [R]
    int R, width, N, Hq, Hkv, gs;   // gs = Hq / Hkv
    int window, sinks;          // window: INT_MAX without one
    float scale;                // the score's scale times log2(e)
    int zero_rest;              // rows of no request get zeros (and lse -infinity)
    long long patience;         // clock cycles before a wait gives up
    int rows_upto;              // chunk_rows_kernel takes requests of up to this many query rows a key/value head
    // chunk_rows_kernel: CTAs, their parts, what the parts belong to
    int grid, least;            // least: units (key tiles) of a CTA at least
    float* part_o;              // [2 grid][MT][D]
    float2* part_l;             // [2 grid][MT], each part's maximum m and sum of 2^(score - m): apart, for m that swallow the sum's
                                // logarithm
    int4* split;                // [grid]: request, head, row0, parts; parts 0: none
    // chunk_tensor_kernel's
    int t_grid;                 // 0: not launched
    int t_start;                // units that start and end of a tile take as long as
    int out_32;                 // the output's rows are aligned to 32 bytes
    float* t_part_o;            // [2 t_grid][MANY][D]
    float2* t_part_l;
    int4* t_split;
};

// A request: its queries [q0, q0 + nq), query rows per key/value head (a row is a token's query head: token
// j's heads follow one another), tokens.
struct Request {
    int q0, nq, len;
    __device__ __forceinline__ int rows(const ChunkArgs& a) const { return nq * a.gs; }
    // Position of the token of a query row; below 0 it sees nothing.
    __device__ __forceinline__ int pos(const ChunkArgs& a, int row) const { return len - nq + row / a.gs; }
};
// Lengths and tables, by a kernel that has waited for what comes before it or not (few rows behind the tensor cores): then from
// L2, since an SM's L1 may hold what was there before.  (For all from L2, the window case took 113 us instead of 106.)
template <bool WAITED>
__device__ __forceinline__ int get(const ChunkArgs& a, const int* p) { return WAITED || a.t_grid == 0 ? *p : __ldcg(p); }
template <bool WAITED>
__device__ __forceinline__ Request request(const ChunkArgs& a, int r) {
    Request x;
    x.q0 = min(max(get<WAITED>(a, a.starts + r), 0), a.N);
    x.nq = max(min(max(get<WAITED>(a, a.starts + r + 1), 0), a.N) - x.q0, 0);
    x.len = int(min(int64_t(max(get<WAITED>(a, a.lens + r), 0)), int64_t(a.width) * a.page_size));
    return x;
}

// The keys that the tokens at positions p_lo .. p_hi see between them, [lo, hi) and [0, sink), in tiles of KT keys:
// tile i holds the keys from at(i) on.
template <int KT>
struct KeyTiles {
    int lo, hi, sink;
    int few, skip, n;           // tiles before the gap, first tile behind it, tiles (at least 1)
    KeyTiles() = default;
    __device__ __forceinline__ KeyTiles(const ChunkArgs& a, int p_lo, int p_hi) {
        hi = max(p_hi + 1, 0);
        lo = max(0, max(p_lo, 0) - a.window + 1);
        sink = min(a.sinks, hi);
        skip = lo / KT;
        few = min((sink + KT - 1) / KT, skip);
        n = max(few + (hi + KT - 1) / KT - skip, 1);
    }
    __device__ __forceinline__ int at(int i) const { return (i < few ? i : i - few + skip) * KT; }
    // Whether some token sees key k.
    __device__ __forceinline__ bool seen(int k) const { return k < hi && (k >= lo || k < sink); }
};
// Whether the token at position p sees key k.
__device__ __forceinline__ bool sees(const ChunkArgs& a, int p, int k) {
    return k <= p && (p - k < a.window || k < a.sinks);
}

// A key tile of KT keys from k0 on of which some token at p_lo .. p_hi does not see all the keys that are loaded.
__device__ __forceinline__ bool partial_keys(const ChunkArgs& a, int p_lo, int p_hi, int k0, int KT) {
    return p_lo != p_hi && (k0 + KT > p_lo + 1 || (p_hi - k0 >= a.window && k0 + KT > a.sinks));
}

// ------------------------------------------------------------------ the line of work

// A CTA's place in the line of units.
struct Place {
    int r;              // request
    int64_t before;     // the units before the request's
    int64_t units;      // the request's units of one key/value head
};

// Units of one key/value head of a request that is not the tensor cores': key tiles, and FEW_START for each query tile.
template <int MT, int KT>
__device__ __forceinline__ int64_t units_of(const ChunkArgs& a, const Request& x) {
    const int M = x.rows(a);
    if (M == 0 || M > a.rows_upto) return 0;
    int64_t n = 0;
    for (int row = 0; row < M; row += MT) n += KeyTiles<KT>(a, x.pos(a, row), x.pos(a, min(row + MT, M) - 1)).n + FEW_START;
    return n;
}

// Exclusive sum over a block of NT threads, and the total.
template <int NT>
__device__ __forceinline__ int64_t block_sum_before(int64_t mine, int64_t* words, int64_t& total) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    int64_t x = mine;
#pragma unroll
    for (int s = 1; s < 32; s <<= 1) {
        const int64_t y = __shfl_up_sync(FULL, x, s);
        if (lane >= s) x += y;
    }
    if (lane == 31) words[warp] = x;
    __syncthreads();
    int64_t before = 0;
    total = 0;
#pragma unroll
    for (int w = 0; w < NT / 32; ++w) {
        if (w == warp) before = total;
        total += words[w];
    }
    __syncthreads();
    return before + x - mine;
}

// A tensor-core tile of MANY query rows: a unit for every key tile, and t_start more.  (Of 128 rows or less it takes as long: it is
// the chain of products and weights of a tile that is waited for, not their rate.)
struct ManyTile {
    int p_lo, p_hi;             // positions of its first and last token
    KeyTiles<128> kt;
    int units;
    ManyTile() = default;
    __device__ __forceinline__ ManyTile(const ChunkArgs& a, const Request& x, int row0) {
        const int M = x.rows(a);
        p_lo = x.pos(a, row0), p_hi = x.pos(a, min(row0 + MANY, M) - 1);
        kt = KeyTiles<128>(a, p_lo, p_hi);
        units = a.t_start + kt.n;
    }
    // Key tiles within the first n units.
    __device__ __forceinline__ int tiles(int64_t n) const { return int(max(n - (units - kt.n), int64_t(0))); }
};

// A CTA's run of the tensor cores' units, of the tiles' for every key/value head.  It begins in the tile of rows row0 on of
// request r, whose units (of all heads) have `before` units before them.
struct ManyRun {
    int64_t first, last, total, before;
    int r, row0, ctas;
    // The CTA of unit u.
    __device__ __forceinline__ int owner(int64_t u) const { return int(((u + 1) * ctas - 1) / total); }
};
// Every CTA looks all requests over: threads share the requests to count their tiles, then the tiles to count their units.
// words: 32 and NT more.  The run is in shared memory behind the next barrier; whether there is one.
template <int NT>
__device__ __forceinline__ bool many_run(const ChunkArgs& a, int cta, int64_t* words, ManyRun& run) {
    const int tid = threadIdx.x, per = (a.R + NT - 1) / NT, r0 = min(tid * per, a.R), r1 = min(r0 + per, a.R);
    int64_t* tiles_before = words + 32;     // [NT]: the tiles of the threads before
    auto tiles_of = [&](const Request& x) {
        const int M = x.rows(a);
        return M > a.rows_upto ? (M + MANY - 1) / MANY : 0;
    };
    auto units = [&](const Request& x, int row0) { return ManyTile(a, x, row0).units; };
    if (tid == 0) run.r = run.row0 = 0, run.before = 0;    // (a request that there is, whatever the lengths)
    int64_t tiles, total, mine = 0;
    for (int r = r0; r < r1; ++r) mine += tiles_of(request<true>(a, r));
    tiles_before[tid] = block_sum_before<NT>(mine, words, tiles);
    __syncthreads();
    // tiles [i0, i1) are this thread's; the first is one of the last thread's that has no more than i0 before it
    const int64_t each = (tiles + NT - 1) / NT, i0 = min(tid * each, tiles), i1 = min(i0 + each, tiles);
    int lo = 0;
    for (int hi = NT; i0 < i1 && hi - lo > 1;) {
        const int mid = (lo + hi) / 2;
        if (tiles_before[mid] <= i0) lo = mid;
        else hi = mid;
    }
    int64_t at = tiles_before[lo];
    int r = lo * per;
    Request x = {};
    for (; i0 < i1 && r < a.R; at += tiles_of(x), ++r) {
        x = request<true>(a, r);
        if (at + tiles_of(x) > i0) break;
    }
    // f(request, its number, first row) for each of them
    auto walk = [&](auto f) {
        Request y = x;
        int k = r, row0 = int(i0 - at) * MANY;
        for (int64_t i = i0; i < i1; ++i) {
            while ((row0 >= y.rows(a) || y.rows(a) <= a.rows_upto) && k + 1 < a.R) y = request<true>(a, ++k), row0 = 0;
            if (!f(y, k, row0)) return;
            row0 += MANY;
        }
    };
    mine = 0;
    walk([&](const Request& y, int, int row0) { return mine += units(y, row0), true; });
    int64_t before = block_sum_before<NT>(mine, words, total) * a.Hkv;
    total *= a.Hkv;
    const int ctas = int(max(min(int64_t(a.t_grid), total), int64_t(1)));
    const int64_t first = cta < ctas ? total * cta / ctas : total, last = cta < ctas ? total * (cta + 1) / ctas : total;
    if (tid == 0) run.first = first, run.last = last, run.total = total, run.ctas = ctas;
    if (first < last && before <= first && first < before + mine * a.Hkv)
        walk([&](const Request& y, int k, int row0) {
            const int64_t n = int64_t(units(y, row0)) * a.Hkv;
            if (first >= before + n) return before += n, true;
            run.r = k, run.row0 = row0, run.before = before;
            return false;
        });
    return first < last;
}

// A CTA's run of units, cut from all of the launch's in equal lengths.
struct Run {
    int64_t first, last, length;
    Place place;
};
template <int NT, int MT, int KT>
__device__ __forceinline__ Run run_of(const ChunkArgs& a, int cta, int64_t* words) {
    const int tid = threadIdx.x, per = (a.R + NT - 1) / NT, r0 = min(tid * per, a.R), r1 = min(r0 + per, a.R);
    int64_t mine = 0;
    for (int r = r0; r < r1; ++r) mine += units_of<MT, KT>(a, request<false>(a, r));
    int64_t total, before = block_sum_before<NT>(mine, words, total);
    total *= a.Hkv;
    Run run;
    run.length = max(int64_t(a.least), (total + a.grid - 1) / a.grid);
    run.first = min(cta * run.length, total);
    run.last = min(run.first + run.length, total);
    if (run.first < run.last && before * a.Hkv <= run.first && run.first < (before + mine) * a.Hkv) {
        for (int r = r0; r < r1; ++r) {
            const int64_t n = units_of<MT, KT>(a, request<false>(a, r));
            if (run.first < (before + n) * a.Hkv) {
                words[16] = r, words[17] = before * a.Hkv, words[18] = n;
                break;
            }
            before += n;
        }
    }
    __syncthreads();
    run.place = Place{run.first < run.last ? int(words[16]) : 0, words[17], words[18]};
    __syncthreads();
    return run;
}

// The start of the kernel of few rows; whether a CTA has a run.  Behind the tensor cores' kernel it does not wait for that one, which
// has waited for what comes before both of them; one CTA more waits for it in the end, so that what comes behind has both.
__device__ __forceinline__ bool few_starts(const ChunkArgs& a) {
    if (a.t_grid == 0) grid_dependency_wait();
    allow_dependents();
    if (int(blockIdx.x) < a.grid) return true;
    grid_dependency_wait();
    return false;
}

// Rows of no request become zeros.
template <typename T, int D>
__device__ __forceinline__ void zero_rest(const ChunkArgs& a, int cta, int threads) {
    constexpr int DC = D / 8;
    const int lo = a.R > 0 ? min(max(__ldcg(a.starts), 0), a.N) : a.N,
              hi = a.R > 0 ? max(min(max(__ldcg(a.starts + a.R), 0), a.N), lo) : a.N;
    const int rest = lo + a.N - hi;
    for (int64_t i = int64_t(cta) * threads + threadIdx.x; i < int64_t(rest) * a.Hq * DC; i += int64_t(a.grid) * threads) {
        const int c = int(i % DC), h = int(i / DC % a.Hq), j = int(i / DC / a.Hq), t = j < lo ? j : hi + j - lo;
        *reinterpret_cast<uint4*>(static_cast<T*>(a.out) + t * a.os[0] + h * a.os[1] + c * 8) = make_uint4(0, 0, 0, 0);
        if (c == 0 && a.lse) a.lse[int64_t(t) * a.Hq + h] = -INFINITY;
    }
}

// A tile of a CTA that gave up, sg its part: NaN for its rows (of a cut tile, for the sums that they are joined by).  By one warp.
template <typename T, int D, int ROWS, typename Seg>
__device__ __forceinline__ void lost_tile(const ChunkArgs& a, const Seg& sg, float2* part_l, int4* split, int cta, int lane) {
    const float nan = __int_as_float(0x7fffffff);
#pragma unroll 1
    for (int r = 0; r < min(ROWS, sg.M - sg.row0); ++r) {
        const int row = sg.row0 + r, j = row / a.gs, h = sg.head * a.gs + row - j * a.gs;
        if (sg.whole) {
            T* out = static_cast<T*>(a.out) + (sg.x.q0 + j) * a.os[0] + h * a.os[1];
            if (lane < D / 8) *reinterpret_cast<uint4*>(out + lane * 8) = make_uint4(0x7fff7fffu, 0x7fff7fffu, 0x7fff7fffu, 0x7fff7fffu);
            if (lane == 0 && a.lse) a.lse[int64_t(sg.x.q0 + j) * a.Hq + h] = nan;
        } else if (lane == 0) {
            part_l[int64_t(2 * cta + (sg.i0 == 0)) * ROWS + r] = make_float2(-INFINITY, nan);
        }
    }
    if (sg.parts > 0 && lane == 0) split[cta] = make_int4(sg.r, sg.head, sg.row0, sg.parts);
}

// ------------------------------------------------------------------ infinite and NaN values

// Whether an element of a 16-byte word is infinite or NaN, and the word with zeros in their place.
template <typename T>
constexpr uint32_t exponent_bits() { return std::is_same<T, __half>::value ? 0x7c00u : 0x7f80u; }
template <typename T>
__device__ __forceinline__ bool odd_half(uint32_t x) { return (x & exponent_bits<T>()) == exponent_bits<T>(); }
template <typename T>
__device__ __forceinline__ bool odd_words(uint4 w) {
    // (an exponent of ones, and no other, carries into the bit above when its lowest bit is added)
    constexpr uint32_t E = exponent_bits<T>(), M = E | E << 16, ONE = (E & (~E + 1)) | (E & (~E + 1)) << 16;
    return ((((w.x & M) + ONE) | ((w.y & M) + ONE) | ((w.z & M) + ONE) | ((w.w & M) + ONE)) & 0x80008000u) != 0;
}
template <typename T>
__device__ __forceinline__ uint32_t even_word(uint32_t x) {
    return (odd_half<T>(x) ? 0u : x & 0xffffu) | (odd_half<T>(x >> 16) ? 0u : x & 0xffff0000u);
}
template <typename T>
__device__ __forceinline__ uint4 even_words(uint4 w) {
    return make_uint4(even_word<T>(w.x), even_word<T>(w.y), even_word<T>(w.z), even_word<T>(w.w));
}
// The infinite and NaN values, elements d .. d + 3 of a head, of the keys k0 .. k0 + n - 1 that the
// token at position p sees, added to y.
template <typename T, bool WAITED>
__device__ __noinline__ void add_odd(const ChunkArgs& a, const int* table, int p, int k0, int n, int head, int d, float4& y) {
    for (int k = k0; k < k0 + n && k <= p; ++k) {
        if (!sees(a, p, k)) continue;
        const int pi = k / a.page_size, page = get<WAITED>(a, table + pi);
        if (page < 0 || page >= a.num_pages) continue;
        const T* v = static_cast<const T*>(a.v) + page * a.vc[0] + (k - pi * a.page_size) * a.vc[1] + head * a.vc[2] + d;
        auto odd = [&](int e) {
            const float z = Mma<T>::get(WAITED ? v[e] : __ldcg(v + e));
            return fabsf(z) <= 3.402823466e38f ? 0.f : z;
        };
        y = make_float4(y.x + odd(0), y.y + odd(1), y.z + odd(2), y.w + odd(3));
    }
}

// Which of the keys k0 .. k0 + 31 of request r have no page (within what its table can name).
template <bool WAITED>
__device__ __noinline__ unsigned missing_pages(const ChunkArgs& a, int r, int k0) {
    unsigned bits = 0;
    for (int e = 0; e < 32; ++e) {
        const int pi = (k0 + e) / a.page_size;
        if (pi >= a.width) break;
        const int page = get<WAITED>(a, a.table + int64_t(r) * a.width + pi);
        if (page < 0 || page >= a.num_pages) bits |= 1u << e;
    }
    return bits;
}

// Requests of up to FEW query rows (chunk_few.cu); of more, for heads of 64 or 128, on the tensor cores (chunk_tensor.cu; without
// maps: nullptr).
struct ChunkMaps;
fs_status launch_chunk_few(const ChunkArgs& a, const ChunkMaps& maps, int dtype, int head_dim, void* stream);
fs_status launch_chunk_tensor(const ChunkArgs& a, const ChunkMaps* maps, int dtype, int head_dim, void* stream);

}  // namespace fsd
