// Copies of keys, values and queries into swizzled tiles in shared memory.
//
// By TMA.  Rows of which every key is there are boxes of up to 64 slots of a page, for pages of 8, 16, 32 ... slots.
// The others, and all of other page sizes, are gathers of four rows: caches and queries are matrices whose rows
// lie a common divisor of their strides apart, so any page size and order of slots and heads is a list of row
// numbers, and a key that no query sees is a row outside, which reads as zeros.  (A gather of 512 bytes takes the
// copy engine about 33 cycles, 4250 for 128 keys and values of 128.)
#pragma once

#include <cuda.h>

#include "chunk.cuh"
#include "tensor_core.cuh"

namespace fsd {

// A tensor as the rows of one matrix: row numbers of its dimensions' steps (a page, a slot, a head; a token, a head), and as
// boxes (not always).
struct RowMap {
    CUtensorMap rows, boxes;    // boxes: [pages][heads][slots][dim]; [tokens][heads][dim]
    int step[3];
    int box;                    // rows of a box, 0: none
};
struct ChunkMaps {
    RowMap k, v, q;
    int qrows;                  // a tensor-core tile's queries are one box
};

// Maps for a call's tensors, false where the strides have no common divisor of a row's length or more.
bool chunk_maps(const ChunkArgs& a, int dtype, int head_dim, ChunkMaps& maps);

// Four rows of 64 elements from element x of each on, into 512 bytes of a swizzled tile.
__device__ __forceinline__ void gather4(uint32_t dst, const CUtensorMap* map, int x, const int (&row)[4], uint32_t bar) {
    asm volatile("cp.async.bulk.tensor.2d.shared::cluster.global.tile::gather4.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3, %4, %5, %6}], [%7];"
                 ::"r"(dst), "l"(map), "r"(x), "r"(row[0]), "r"(row[1]), "r"(row[2]), "r"(row[3]), "r"(bar) : "memory");
}
// A box of a page's slots, 64 elements of each.
__device__ __forceinline__ void copy_box(uint32_t dst, const CUtensorMap* map, int x, int slot, int head, int page, uint32_t bar) {
    asm volatile("cp.async.bulk.tensor.4d.shared::cluster.global.tile.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3, %4, %5}], [%6];"
                 ::"r"(dst), "l"(map), "r"(x), "r"(slot), "r"(head), "r"(page), "r"(bar) : "memory");
}
__device__ __forceinline__ void copy_box(uint32_t dst, const CUtensorMap* map, int x, int head, int token, uint32_t bar) {
    asm volatile("cp.async.bulk.tensor.3d.shared::cluster.global.tile.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3, %4}], [%5];"
                 ::"r"(dst), "l"(map), "r"(x), "r"(head), "r"(token), "r"(bar) : "memory");
}
__device__ __forceinline__ void bar_expect(uint32_t bar, uint32_t bytes) {
    asm volatile("{ .reg .b64 t; mbarrier.arrive.expect_tx.shared::cta.b64 t, [%0], %1; }" ::"r"(bar), "r"(bytes) : "memory");
}

// The pages of a lane's four keys of 64: lane l has keys 4 (l % 16) .. + 3 (both halves of a warp the same).
struct Pages {
    int at[4];
    // As the table has them; the loads are not waited for here.
    template <bool WAITED>
    __device__ __forceinline__ void look_up(const ChunkArgs& a, const int* table, int key) {
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            if (j > 0 && a.page_shift >= 2) break;   // four keys of one page
            const int pi = a.page_shift >= 0 ? (key + j) >> a.page_shift : (key + j) / a.page_size;
            at[j] = pi < a.width ? get<WAITED>(a, table + pi) : -1;
        }
    }
    // -1 for a key that no query of the tile sees, and for one whose page does not exist.  Whether there is one of the latter:
    // its score is NaN for every query that sees it.
    template <int KT>
    __device__ __forceinline__ bool resolve(const ChunkArgs& a, const KeyTiles<KT>& kt, int key) {
        bool gone = false;
        if (a.page_shift >= 2) at[1] = at[2] = at[3] = at[0];
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const bool there = at[j] >= 0 && at[j] < a.num_pages, seen = kt.seen(key + j);
            gone |= seen && !there;
            if (!seen || !there) at[j] = -1;
        }
        return gone;
    }
};

// 64 rows of a head from key k0 (a multiple of 64) on, by one warp; blocks of 64 elements `block` bytes apart.
template <int D>
__device__ __forceinline__ void copy_rows(const ChunkArgs& a, const RowMap& m, const Pages& p, int k0, int head, uint32_t dst,
                                          uint32_t block, uint32_t bar, int lane) {
    constexpr int B = D / 64;
    if (m.box > 0 && __all_sync(FULL, (p.at[0] | p.at[1] | p.at[2] | p.at[3]) >= 0)) {
        const int per = 64 / m.box * B;      // boxes, 32 at a time
        for (int i = 0; i < per; i += 32) {
            const int at = (i + lane) / B * m.box, x = (i + lane) % B, page = __shfl_sync(FULL, p.at[0], (at >> 2) & 15);
            if (at < 64) copy_box(dst + x * block + at * 128, &m.boxes, x * 64, (k0 + at) & (a.page_size - 1), head, page, bar);
        }
    } else {
        const int row = (lane & 15) * 4;
        int rows[4];
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const int key = k0 + row + j, slot = a.page_shift >= 0 ? key & (a.page_size - 1) : key % a.page_size;
            rows[j] = p.at[j] >= 0 ? p.at[j] * m.step[0] + slot * m.step[1] + head * m.step[2] : -1;
        }
#pragma unroll
        for (int x = lane >> 4; x < B; x += 2) gather4(dst + x * block + row * 128, &m.rows, x * 64, rows, bar);
    }
}

}  // namespace fsd
