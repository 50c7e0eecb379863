// Page tables and token places of one serving step, from the requests' lengths (sm_103a).
//
// Request r holds lens[r] tokens and gets new_lens[r] more.  With p the page size its new pages are
//   need[r] = ceil((lens[r] + new_lens[r]) / p) - ceil(lens[r] / p),
// taken from the top of a stack of free pages, and its tokens lie one behind the other in the step's
// batch.  Which requests are granted follows from two running sums over what was asked for (pages up
// to r <= free pages, tokens up to r <= budget), where the granted ones lie from two more over what was granted.
//
// A few kilobytes: bound by latency, so one launch.  Every CTA makes the sums over all requests itself
// (8 bytes a request, from L2) and then fills its own window of token places or of new pages:
// each granted request marks its first place in the window, and a running maximum over the
// window tells every place whose it is, whatever the mix of one-token and long requests.
// (64 requests 5.4 us a pass, most of it the call; 1512 requests and 16384 places 6.8 us.)
#include <algorithm>

#include "fs_device.cuh"
#include "fs_host.h"

namespace fsd {

constexpr int TNTH = 512;              // threads
constexpr int TPER = 4;                // places per thread
constexpr int TWIN = TNTH * TPER;      // places of a CTA

struct TablesArgs {
    const int* lens;
    const int* new_lens;
    int* table;                  // [R][width]
    const int* free_pages;       // [free_size], a stack
    const int* free_count;
    int R, width, free_size, page_size, budget;
    int* starts;                 // [R + 1]
    int* rows;                   // [budget]
    int* positions;              // [budget]
    int* totals;                 // [R]
    int* free_left;
    int token_ctas;              // windows of token places; the other CTAs have windows of pages
};

// Exclusive sums of two 64-bit values over the block's threads; the totals in *at and *bt.  `red`: 2 x 32 values.
__device__ __forceinline__ void block_scan2(long long& a, long long& b, long long* at, long long* bt, long long* red) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    long long x = a, y = b;
#pragma unroll
    for (int s = 1; s < 32; s <<= 1) {
        const long long u = __shfl_up_sync(FULL, x, s), v = __shfl_up_sync(FULL, y, s);
        if (lane >= s) x += u, y += v;
    }
    if (lane == 31) red[warp] = x, red[32 + warp] = y;
    __syncthreads();
    long long pa = 0, pb = 0, ta = 0, tb = 0;
#pragma unroll
    for (int w = 0; w < TNTH / 32; ++w) {
        if (w == warp) pa = ta, pb = tb;
        ta += red[w], tb += red[32 + w];
    }
    __syncthreads();
    a = pa + x - a, b = pb + y - b;
    *at = ta, *bt = tb;
}

__global__ void __launch_bounds__(TNTH) tables_kernel(const TablesArgs a) {
    __shared__ long long red[64];
    __shared__ int mark[TWIN];       // the request that starts at a place of the window, -1: none
    __shared__ int base[TWIN];       // its position (token) or table index (page) at the window's start
    __shared__ int top[TNTH / 32];
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    grid_dependency_wait();
    allow_dependents();
    const int per = (a.R + TNTH - 1) / TNTH, r0 = min(tid * per, a.R), r1 = min(r0 + per, a.R);
    const int free = min(max(*a.free_count, 0), a.free_size);
    const long long room = (long long)(a.width) * a.page_size;
#pragma unroll
    for (int i = 0; i < TPER; ++i) mark[tid + i * TNTH] = -1;

    // what request r asks for: nothing when its lengths are out of range
    auto ask = [&](int r, int& len, int& need, int& tok) {
        const int n = a.new_lens[r];
        len = a.lens[r];
        need = tok = 0;
        if (n > 0 && len >= 0 && (long long)(len) + n <= room) {
            const int have = int((unsigned(len) + unsigned(a.page_size) - 1) / unsigned(a.page_size));
            need = int((unsigned(len) + unsigned(n) + unsigned(a.page_size) - 1) / unsigned(a.page_size)) - have;
            tok = n;
        }
    };
    long long pages = 0, toks = 0, tp, tt;
    for (int r = r0; r < r1; ++r) {
        int len, need, tok;
        ask(r, len, need, tok);
        pages += need, toks += tok;
    }
    block_scan2(pages, toks, &tp, &tt, red);
    // granted: by the sums over everything asked for so far
    auto granted = [&](int need, int tok, long long p, long long t) {
        return tok > 0 && (need == 0 || p + need <= free) && t + tok <= a.budget;
    };
    long long gp = 0, gt = 0, p = pages, t = toks;
    for (int r = r0; r < r1; ++r) {
        int len, need, tok;
        ask(r, len, need, tok);
        if (granted(need, tok, p, t)) gp += need, gt += tok;
        p += need, t += tok;
    }
    block_scan2(gp, gt, &tp, &tt, red);   // (tp, tt: all granted)

    const bool tokens = int(blockIdx.x) < a.token_ctas;
    const int w0 = (tokens ? blockIdx.x : blockIdx.x - a.token_ctas) * TWIN;   // (fits: the host checks it)
    // this CTA's share of the per-request outputs
    const long long share = (a.R + (long long)(gridDim.x) - 1) / gridDim.x;
    const long long out0 = blockIdx.x * share, out1 = out0 + share;
    p = pages, t = toks;
    for (int r = r0; r < r1; ++r) {
        int len, need, tok;
        ask(r, len, need, tok);
        const bool ok = granted(need, tok, p, t);
        p += need, t += tok;
        if (r >= out0 && r < out1) {
            a.starts[r] = int(gt);
            a.totals[r] = ok ? len + tok : max(len, 0);
        }
        if (!ok) continue;
        const int first = int(tokens ? gt : gp), n = tokens ? tok : need;
        const int at = max(first - w0, 0);
        if (n > 0 && first + n > w0 && first - w0 < TWIN) {
            mark[at] = r;
            const int begin = tokens ? len : int((unsigned(len) + unsigned(a.page_size) - 1) / unsigned(a.page_size));
            base[at] = begin + w0 - first;
        }
        gp += need, gt += tok;
    }
    if (blockIdx.x == 0 && tid == 0) {
        a.starts[a.R] = int(tt);
        *a.free_left = free - int(tp);
    }
    __syncthreads();
    // Whose is each place: the running maximum of the marks' places (marks ascend with the requests).
    int who[TPER];
    int last = -1;
#pragma unroll
    for (int i = 0; i < TPER; ++i) {
        const int j = tid * TPER + i;
        if (mark[j] >= 0) last = j;
        who[i] = last;
    }
    int run = last;
#pragma unroll
    for (int s = 1; s < 32; s <<= 1) {
        const int u = __shfl_up_sync(FULL, run, s);
        if (lane >= s) run = max(run, u);
    }
    if (lane == 31) top[warp] = run;
    int before = __shfl_up_sync(FULL, run, 1);
    if (lane == 0) before = -1;
    __syncthreads();
    for (int w = 0; w < warp; ++w) before = max(before, top[w]);
    const int all = int(tokens ? tt : tp);
#pragma unroll
    for (int i = 0; i < TPER; ++i) {
        const int j = tid * TPER + i, at = who[i] >= 0 ? who[i] : before;
        const bool real = w0 + j < all && at >= 0;
        if (tokens) {
            if (w0 + j < a.budget) {
                a.rows[w0 + j] = real ? mark[at] : -1;
                a.positions[w0 + j] = real ? base[at] + j : -1;
            }
        } else if (real) {
            a.table[int64_t(mark[at]) * a.width + base[at] + j] = a.free_pages[free - 1 - (w0 + j)];
        }
    }
}

}  // namespace fsd

extern "C" {

fs_status fs_paged_step_tables(const int32_t* lens, const int32_t* new_lens, int32_t requests, int32_t* page_table,
                               int32_t table_width, const int32_t* free_pages, int32_t free_size,
                               const int32_t* free_count, int32_t page_size, int32_t budget, int32_t* query_starts,
                               int32_t* rows, int32_t* positions, int32_t* totals, int32_t* free_left, void* stream) {
    using namespace fsd;
    if (requests < 0 || table_width < 0 || free_size < 0 || page_size < 1 || budget < 0) return FS_ERR_INVALID_ARG;
    if (!query_starts || !free_left || !free_count || (budget > 0 && (!rows || !positions))) return FS_ERR_INVALID_ARG;
    if (requests > 0 && (!lens || !new_lens || !totals)) return FS_ERR_INVALID_ARG;
    if ((int64_t(requests) * table_width > 0 && !page_table) || (free_size > 0 && !free_pages)) return FS_ERR_INVALID_ARG;
    const int64_t lim = 0x7fffffff - 2 * TWIN;
    if (int64_t(table_width) * page_size > lim || int64_t(budget) + requests > lim) return FS_ERR_UNSUPPORTED;
    TablesArgs a = {};
    a.lens = lens;
    a.new_lens = new_lens;
    a.table = page_table;
    a.free_pages = free_pages;
    a.free_count = free_count;
    a.R = requests;
    a.width = table_width;
    a.free_size = free_size;
    a.page_size = page_size;
    a.budget = budget;
    a.starts = query_starts;
    a.rows = rows;
    a.positions = positions;
    a.totals = totals;
    a.free_left = free_left;
    // The most pages that `budget` tokens of the requests can start, and the most there are.
    const int64_t pages = std::min<int64_t>({int64_t(budget) / page_size + requests, budget, free_size});
    a.token_ctas = std::max(1, (budget + TWIN - 1) / TWIN);
    const int64_t grid = a.token_ctas + (pages + TWIN - 1) / TWIN;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(unsigned(grid), 1, 1);
    cfg.blockDim = dim3(TNTH, 1, 1);
    cfg.stream = static_cast<cudaStream_t>(stream);
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    const cudaError_t e = cudaLaunchKernelEx(&cfg, tables_kernel, a);
    return e == cudaSuccess ? FS_OK : cuda_fail(e);
}

}  // extern "C"
