// Barriers in shared memory, tensor memory and the 5th-generation tensor cores' instructions, as the
// attention kernels use them.
#pragma once

#include <type_traits>

#include "attention.cuh"

namespace fsd {

constexpr long long PATIENCE = 4000000000ll;  // clock cycles, two seconds or more, before a wait gives up

// ------------------------------------------------------------------ barriers

__device__ __forceinline__ void bar_init(uint32_t bar, uint32_t count) {
    asm volatile("mbarrier.init.shared::cta.b64 [%0], %1;" ::"r"(bar), "r"(count) : "memory");
}
__device__ __forceinline__ void bar_arrive(uint32_t bar) {
    asm volatile("{ .reg .b64 t; mbarrier.arrive.shared::cta.b64 t, [%0]; }" ::"r"(bar) : "memory");
}
__device__ __forceinline__ bool bar_try(uint32_t bar, uint32_t parity) {
    uint32_t ok;
    asm volatile(
        "{ .reg .pred p; mbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2; selp.u32 %0, 1, 0, p; }"
        : "=r"(ok) : "r"(bar), "r"(parity) : "memory");
    return ok != 0;
}
// Without a try's suspension, which is longer than the longest wait that there is while all goes well.
__device__ __forceinline__ bool bar_test(uint32_t bar, uint32_t parity) {
    uint32_t ok;
    asm volatile(
        "{ .reg .pred p; mbarrier.test_wait.parity.shared::cta.b64 p, [%1], %2; selp.u32 %0, 1, 0, p; }"
        : "=r"(ok) : "r"(bar), "r"(parity) : "memory");
    return ok != 0;
}
// False when the wait ran out here or in another role of the CTA.  (A try suspends the thread for some time by itself; with
// a time of 2 us asked for, a warp woke up later: chunks of 1021 tokens behind 16384 431 us, 412 without.)
__device__ __forceinline__ bool bar_wait(uint32_t bar, uint32_t parity, volatile int* dead, long long patience = PATIENCE) {
    if (bar_try(bar, parity)) return true;
    const long long start = clock64();
    for (uint32_t i = 1;; ++i) {
        if (bar_try(bar, parity)) return true;
        if ((i & 7) == 0) {
            if (*dead) return false;
            if (clock64() - start > patience) break;
        }
    }
    *dead = 1;
    return false;
}
// The same, but a limit shorter than the default is kept to the cycle.  For a role that nothing is waiting for: with the choice in
// every wait a prompt of 8190 tokens took 433 us instead of 420.
__device__ __forceinline__ bool bar_wait_exactly(uint32_t bar, uint32_t parity, volatile int* dead, long long patience) {
    if (patience >= PATIENCE) return bar_wait(bar, parity, dead, patience);
    const long long start = clock64();
    do {
        if (bar_test(bar, parity)) return true;
    } while (clock64() - start < patience && !*dead);
    *dead = 1;
    return false;
}
// What has been issued on its way to a barrier, waited for by a role that gives up.
__device__ __forceinline__ void bar_drain(uint32_t bar) {
    const long long start = clock64();
    while (!bar_try(bar, 0) && clock64() - start < PATIENCE) {}
}

// ------------------------------------------------------------------ tensor memory and matrix instructions

__device__ __forceinline__ void tmem_fence_before() { asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory"); }
__device__ __forceinline__ void tmem_fence_after() { asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory"); }
__device__ __forceinline__ void tmem_wait_ld() { asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory"); }
__device__ __forceinline__ void tmem_wait_st() { asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory"); }
__device__ __forceinline__ void proxy_fence() { asm volatile("fence.proxy.async.shared::cta;" ::: "memory"); }

#define R8(x, i) "=r"(x[i]), "=r"(x[i + 1]), "=r"(x[i + 2]), "=r"(x[i + 3]), "=r"(x[i + 4]), "=r"(x[i + 5]), "=r"(x[i + 6]), "=r"(x[i + 7])
#define W8(x, i) "r"(x[i]), "r"(x[i + 1]), "r"(x[i + 2]), "r"(x[i + 3]), "r"(x[i + 4]), "r"(x[i + 5]), "r"(x[i + 6]), "r"(x[i + 7])
// 32 columns of this thread's lane.
__device__ __forceinline__ void tmem_ld32(uint32_t (&x)[32], uint32_t addr) {
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x32.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16,%17,%18,%19,"
        "%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31}, [%32];"
        : R8(x, 0), R8(x, 8), R8(x, 16), R8(x, 24) : "r"(addr));
}
__device__ __forceinline__ void tmem_ld16(uint32_t (&x)[16], uint32_t addr) {
    asm volatile("tcgen05.ld.sync.aligned.32x32b.x16.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15}, [%16];"
                 : R8(x, 0), R8(x, 8) : "r"(addr));
}
__device__ __forceinline__ void tmem_st32(uint32_t addr, const uint32_t (&x)[32]) {
    asm volatile(
        "tcgen05.st.sync.aligned.32x32b.x32.b32 [%32], {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16,%17,%18,"
        "%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31};"
        ::W8(x, 0), W8(x, 8), W8(x, 16), W8(x, 24), "r"(addr) : "memory");
}
__device__ __forceinline__ void tmem_st16(uint32_t addr, const uint32_t (&x)[16]) {
    asm volatile(
        "tcgen05.st.sync.aligned.32x32b.x16.b32 [%16], {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15};"
        ::W8(x, 0), W8(x, 8), "r"(addr) : "memory");
}
// What is read from these registers is read behind this point (and so behind a wait before it).
__device__ __forceinline__ void keep32(uint32_t (&x)[32]) {
#define K8(x, i) "+r"(x[i]), "+r"(x[i + 1]), "+r"(x[i + 2]), "+r"(x[i + 3]), "+r"(x[i + 4]), "+r"(x[i + 5]), "+r"(x[i + 6]), "+r"(x[i + 7])
    asm volatile("" : K8(x, 0), K8(x, 8));
    asm volatile("" : K8(x, 16), K8(x, 24));
#undef K8
}
#undef R8
#undef W8

// The weights of the second product are 16 bits, as its matrix instruction takes them: each is off by half a step of the
// type, and their sum is not.  bf16 has float32's exponents; f16 ends at 2^-14 (in steps of 2^-24) and 65504, so its weights
// are 2^SHIFT larger: rounded by half a step down to 2^-(14 + SHIFT) of the maximum, by 2^-(25 + SHIFT) below.  (Unshifted,
// 65536 keys 17 nats below one were off by 1.5 % together.)  With a maximum that may lag by GROWTH they stay
// below 2^15.
template <typename T> struct Weights { static constexpr float GROWTH = 8.f, SHIFT = 0.f; };
template <> struct Weights<__half> { static constexpr float GROWTH = 4.f, SHIFT = 11.f; };

// The i-th run of N registers of an array.
template <int N, int K>
__device__ __forceinline__ uint32_t (&part(uint32_t (&x)[K], int i))[N] { return reinterpret_cast<uint32_t (&)[N]>(x[i * N]); }

// Shared-memory operand with 128-byte swizzle: low word, the address / 16 and, above it, the byte
// stride / 16 between blocks of 64 elements along the rows' contiguous direction (operands
// whose rows run along M or N only); high word, groups of eight 128-byte rows 1024 bytes apart, the
// format's version, the swizzle.
__device__ __forceinline__ uint32_t operand_high() { return (1024u >> 4) | 1u << 14 | 2u << 29; }
// Float32 accumulator, 128 rows, n columns; b_rows: B's rows run along N.
template <typename T>
constexpr uint32_t product(int n, bool b_rows) {
    const uint32_t f = sizeof(T) == 2 && std::is_same<T, __nv_bfloat16>::value ? 1u : 0u;
    return 1u << 4 | f << 7 | f << 10 | (b_rows ? 1u << 16 : 0u) | uint32_t(n / 8) << 17 | (128u / 16) << 24;
}
// Issued where `lead` holds, by one lane of a warp whose operands are uniform.
__device__ __forceinline__ bool elect() {
    uint32_t p;
    asm volatile("{ .reg .pred p; elect.sync _|p, 0xffffffff; selp.u32 %0, 1, 0, p; }" : "=r"(p));
    return p != 0;
}
__device__ __forceinline__ void mma_smem(bool lead, uint32_t d, uint32_t a, int a_lead, uint32_t b, int b_lead, uint32_t hi,
                                         uint32_t desc, bool add) {
    if (lead)
        asm volatile("{ .reg .pred p; .reg .b64 x, y; mov.b64 x, {%1, %3}; mov.b64 y, {%2, %3}; setp.ne.u32 p, %5, 0;"
                     " tcgen05.mma.cta_group::1.kind::f16 [%0], x, y, %4, p; }"
                     ::"r"(d), "r"(a | uint32_t(a_lead >> 4) << 16), "r"(b | uint32_t(b_lead >> 4) << 16), "r"(hi), "r"(desc),
                     "r"(uint32_t(add)) : "memory");
}
__device__ __forceinline__ void mma_tmem(bool lead, uint32_t d, uint32_t a, uint32_t b, int b_lead, uint32_t hi, uint32_t desc,
                                         bool add) {
    if (lead)
        asm volatile("{ .reg .pred p; .reg .b64 y; mov.b64 y, {%2, %3}; setp.ne.u32 p, %5, 0;"
                     " tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], y, %4, p; }"
                     ::"r"(d), "r"(a), "r"(b | uint32_t(b_lead >> 4) << 16), "r"(hi), "r"(desc), "r"(uint32_t(add)) : "memory");
}
// The barrier completes once every matrix instruction issued so far by this thread has.
__device__ __forceinline__ void mma_commit(bool lead, uint32_t bar) {
    if (lead)
        asm volatile("tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];" ::"r"(bar) : "memory");
}

// Byte offset of 16-byte chunk c of row r in a tile of ROWS rows: blocks of 64 elements (128 bytes a
// row), chunks permuted by the row's index within eight.
template <int ROWS>
__device__ __forceinline__ uint32_t tile_at(int r, int c) {
    return uint32_t((c >> 3) * (ROWS * 128) + r * 128 + (((c & 7) ^ (r & 7)) << 4));
}

}  // namespace fsd
