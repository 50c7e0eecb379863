// Matrix fragments in shared memory for mma.sync, 16-bit types.
#pragma once

#include "attention.cuh"

namespace fsd {

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

}  // namespace fsd
