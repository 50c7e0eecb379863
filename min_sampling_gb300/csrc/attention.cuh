// What the kernels of shared-prefix attention have in common: arguments, groups and key
// ranges, 16-bit types.
#pragma once

#include <algorithm>
#include <cstdint>

#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include "fs_device.cuh"
#include "fs_host.h"

namespace fsd {

constexpr int RANGE = 64;     // unit of key ranges: whole tiles of every kernel
constexpr int64_t NOWHERE = INT64_MIN;  // the offset of what is not there (strides, and so offsets, may be negative)

struct AttnArgs {
    const void* q;
    void* out;
    float* lse;                 // [B][Q][Hq], nullable
    int64_t qs[3], os[3];       // strides: row, query, head
    const void* k;
    const void* v;
    int64_t kc[3], vc[3];       // strides: page, slot, head
    int num_pages, page_size, page_shift;  // page_shift: log2(page_size), -1 when it is no power of two
    const int* ptab;            // [G][pw]
    const int* plens;           // [G]
    const int* starts;          // [G + 1], nullable (one group of every row)
    int G, pw;
    const int* stab;            // [B][sw]
    const int* slens;           // [B]
    int sw;
    int B, Q, Hq, Hkv, gs;      // gs = Hq / Hkv
    float scale;                // the score's scale times log2(e)
    float* part_o;              // [SP + SS][B * Q * Hq][D], each part's own softmax output
    float* part_l;              // [SP + SS][B * Q * Hq], log2 of each part's sum of 2^score
    int SP, SS;                 // key ranges: prefix, suffix
    int finish;                 // attend_kernel joins its suffix part with the prefix's parts (of an earlier launch) itself
    int ptiles, stiles;         // query tiles: of all groups together (at most), of one row
};

// ------------------------------------------------------------------ groups and ranges

__device__ __forceinline__ int clamp_row(int x, int B) { return min(max(x, 0), B); }
__device__ __forceinline__ int group_begin(const AttnArgs& a, int g) { return a.starts ? clamp_row(a.starts[g], a.B) : 0; }
__device__ __forceinline__ int group_end(const AttnArgs& a, int g) {
    return a.starts ? max(group_begin(a, g), clamp_row(a.starts[g + 1], a.B)) : a.B;
}
__device__ __forceinline__ int prefix_len(const AttnArgs& a, int g) {
    return int(min(int64_t(max(a.plens[g], 0)), int64_t(a.pw) * a.page_size));
}
__device__ __forceinline__ int suffix_len(const AttnArgs& a, int b) {
    return int(min(int64_t(max(a.slens[b], 0)), int64_t(a.sw) * a.page_size));
}
// Keys per range when `len` keys are cut into at most `splits` ranges.
__device__ __forceinline__ int range_len(int len, int splits) {
    return ((len + splits - 1) / splits + RANGE - 1) / RANGE * RANGE;
}

// The group that row b belongs to, -1 for none: the last one that starts at or before b.
// Warp-collective.
__device__ __forceinline__ int group_of(const AttnArgs& a, int b, int lane) {
    if (!a.starts) return a.G > 0 ? 0 : -1;
    int n = 0;
    for (int g0 = 0; g0 < a.G; g0 += 32) {
        const bool le = g0 + lane < a.G && a.starts[g0 + lane] <= b;
        n += __popc(__ballot_sync(FULL, le));
    }
    return n > 0 && b < group_end(a, n - 1) ? n - 1 : -1;
}

// A group's query tile: its rows [b0, b1), prefix length, and the tile's number inside it.
struct GroupTile {
    int g, tile, b0, b1, len;
};

// The `tile`-th query tile of all groups (tiles of MT queries per key/value head); g = -1
// past the last.  Each lane reads one group, all its words in one round trip.  Warp-collective.
template <int MT>
__device__ __forceinline__ GroupTile group_tile(const AttnArgs& a, int tile, int lane) {
    int before = 0;
    for (int g0 = 0; g0 < a.G; g0 += 32) {
        const int g = g0 + lane;
        int lo = 0, hi = 0, len = 0;
        if (g < a.G) {
            if (a.starts) {
                lo = clamp_row(a.starts[g], a.B);
                hi = max(lo, clamp_row(a.starts[g + 1], a.B));
            } else {
                hi = a.B;
            }
            len = prefix_len(a, g);
        }
        const int n = int((int64_t(hi - lo) * a.Q * a.gs + MT - 1) / MT);
        const int incl = warp_incl_scan_i(n, lane);
        const unsigned hit = __ballot_sync(FULL, before + incl > tile);
        if (hit) {
            const int l = __ffs(hit) - 1;
            return GroupTile{g0 + l, tile - before - __shfl_sync(FULL, incl - n, l), __shfl_sync(FULL, lo, l),
                             __shfl_sync(FULL, hi, l), __shfl_sync(FULL, len, l)};
        }
        before += __shfl_sync(FULL, incl, 31);
    }
    return GroupTile{-1, 0, 0, 0, 0};
}

// ------------------------------------------------------------------ matrix fragments

template <typename T> struct Mma;
template <> struct Mma<__nv_bfloat16> {
    static __device__ __forceinline__ void run(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
        asm volatile(
            "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
            : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
            : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
    }
    static __device__ __forceinline__ uint32_t pack(float x, float y) {
        const __nv_bfloat162 h = __floats2bfloat162_rn(x, y);
        return *reinterpret_cast<const uint32_t*>(&h);
    }
    static __device__ __forceinline__ float get(__nv_bfloat16 x) { return __bfloat162float(x); }
    static __device__ __forceinline__ __nv_bfloat16 put(float x) { return __float2bfloat16_rn(x); }
};
template <> struct Mma<__half> {
    static __device__ __forceinline__ void run(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
        asm volatile(
            "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
            : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
            : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
    }
    static __device__ __forceinline__ uint32_t pack(float x, float y) {
        const __half2 h = __floats2half2_rn(x, y);
        return *reinterpret_cast<const uint32_t*>(&h);
    }
    static __device__ __forceinline__ float get(__half x) { return __half2float(x); }
    static __device__ __forceinline__ __half put(float x) { return __float2half_rn(x); }
};

// 2^x to 2^-22, and the 16-byte asynchronous copy (nothing read and zeros written when off).
__device__ __forceinline__ float exp2_fast(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}
__device__ __forceinline__ void cp16(uint32_t dst, const void* src, bool on) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(on ? 16 : 0) : "memory");
}

// The prefix's part on the tensor cores (prefix_tensor.cu): tiles of 128 or 256 queries, for heads of 64 or 128.
fs_status launch_prefix_tensor(const AttnArgs& a, int dtype, int head_dim, int tile, void* stream);

}  // namespace fsd
