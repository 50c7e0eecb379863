// Penalties for repeated tokens, biases and grammar masks on logits (sm_103a).
//
// Row b with logits z, its history's tokens, a list of biases and a bit mask:
//   z > 0 ? z / repetition : z * repetition     where the token is in the history,
//   - frequency * count - presence * (count > 0)   count: how often it is behind the prompt,
//   + bias,   -infinity where the mask has no bit;
// in float32, rounded once.  Bound by memory: every logit is read once and written once.  A CTA owns a
// segment of a row (16 KB): its logits are in flight while it goes through the row's history and
// counts in shared memory the tokens that fall into the segment, with a bit for each logit that is touched, so that
// the others look nothing up.  No scratch memory, no order that matters: counts are integers, and of
// several biases of one token the last one counts.  In place only what changes is read and written.
#include <algorithm>

#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include "fs_device.cuh"
#include "fs_host.h"

namespace fsd {

constexpr int ADJ_NT = 256;      // threads
// Logits of a CTA: 16 KB, so that five CTAs on an SM are at different points of the way from the first load to the last store.
// (32 KB, two CTAs of 512 threads: 256 rows of 151665 71 us.)
template <typename T> constexpr int ADJ_SEG = 16384 / int(sizeof(T));

struct AdjustArgs {
    const void* x;
    void* out;
    int64_t xs, os;              // row strides (elements)
    int B, V, segs;
    const int* tokens;           // [B][history], rows `ts` apart; nullable
    int64_t ts;
    int history;
    const int* lens;             // nullable: history
    const int* prompt_lens;      // nullable: 0
    const float* repetition;     // nullable
    const float* presence;
    const float* frequency;
    const int* bias_starts;      // [B + 1], nullable
    const int* bias_tokens;
    const float* bias_values;
    int biases;
    const uint32_t* allowed;     // [masks][words], nullable
    const int* allowed_rows;     // nullable: row b
    int masks, words;
    int tokens4;                 // histories can be read four tokens at a time
};

template <typename T> struct Num;
template <> struct Num<float> {
    static __device__ __forceinline__ float get(float x) { return x; }
    static __device__ __forceinline__ float put(float x) { return x; }
};
template <> struct Num<__nv_bfloat16> {
    static __device__ __forceinline__ float get(__nv_bfloat16 x) { return __bfloat162float(x); }
    static __device__ __forceinline__ __nv_bfloat16 put(float x) { return __float2bfloat16_rn(x); }
};
template <> struct Num<__half> {
    static __device__ __forceinline__ float get(__half x) { return __half2float(x); }
    static __device__ __forceinline__ __half put(float x) { return __float2half_rn(x); }
};

template <typename T>
union Words {
    uint4 w;
    T e[16 / sizeof(T)];
};

// The 16 bytes from `p` on, any address that is a multiple of the element's size, of a row [begin, end): lanes ask for
// neighbouring 16 bytes, and each takes what it lacks of its aligned word from the next.  Warp-collective.
__device__ __forceinline__ uint4 load_words(uintptr_t p, uintptr_t begin, uintptr_t end) {
    const uint32_t off = p & 15;
    const uintptr_t q = p - off;
    uint4 a = make_uint4(0, 0, 0, 0);
    // (an aligned word that holds a byte of the row is in the same 16 bytes as memory of the row's)
    if (q < end && q + 16 > begin) a = __ldcs(reinterpret_cast<const uint4*>(q));
    if (off == 0) return a;     // (the same in every lane)
    uint4 b;
    b.x = __shfl_down_sync(FULL, a.x, 1);
    b.y = __shfl_down_sync(FULL, a.y, 1);
    b.z = __shfl_down_sync(FULL, a.z, 1);
    b.w = __shfl_down_sync(FULL, a.w, 1);
    if ((threadIdx.x & 31) == 31 && q + 16 < end && q + 32 > begin) b = __ldcs(reinterpret_cast<const uint4*>(q + 16));
    const uint32_t sh = (off & 3) * 8;
    uint32_t x0, x1, x2, x3, x4;
    switch (off >> 2) {
        case 0: x0 = a.x, x1 = a.y, x2 = a.z, x3 = a.w, x4 = b.x; break;
        case 1: x0 = a.y, x1 = a.z, x2 = a.w, x3 = b.x, x4 = b.y; break;
        case 2: x0 = a.z, x1 = a.w, x2 = b.x, x3 = b.y, x4 = b.z; break;
        default: x0 = a.w, x1 = b.x, x2 = b.y, x3 = b.z, x4 = b.w; break;
    }
    return make_uint4(__funnelshift_r(x0, x1, sh), __funnelshift_r(x1, x2, sh), __funnelshift_r(x2, x3, sh),
                      __funnelshift_r(x3, x4, sh));
}

// Shared memory: a bit per touched logit, a bit per biased one, then a word per logit: its count and, in the upper half, the
// number of its last bias plus one; where either may pass 16 bits (WIDE), a word each.
template <typename T, bool IN_PLACE, bool WIDE>
__global__ void __launch_bounds__(ADJ_NT, WIDE ? 2 : 5) adjust_kernel(const AdjustArgs a) {
    constexpr int SEG = ADJ_SEG<T>, VW = 16 / sizeof(T), PER = SEG / VW / ADJ_NT;
    extern __shared__ __align__(16) uint32_t smem[];
    uint32_t* touched = smem;                   // [SEG / 32]
    uint32_t* biased = smem + SEG / 32;         // [SEG / 32]
    uint32_t* count = smem + SEG / 16;          // [SEG]
    uint32_t* which = WIDE ? count + SEG : count;
    const int tid = threadIdx.x;
    grid_dependency_wait();
    allow_dependents();
    const int row = blockIdx.x / a.segs, seg = blockIdx.x - row * a.segs;
    const T* x = static_cast<const T*>(a.x) + row * a.xs;
    T* out = static_cast<T*>(a.out) + row * a.os;
    // The output's 16-byte words: word j of the segment holds logits e0 + j VW on.
    const int mis = int((reinterpret_cast<uintptr_t>(out) & 15) / sizeof(T));
    const int e0 = seg * SEG - mis;
    auto whole = [&](int j) { return e0 + j * VW >= 0 && e0 + (j + 1) * VW <= a.V; };
    constexpr uint32_t ALL = (1u << VW) - 1;
    Words<T> w[PER];
    if (!IN_PLACE) {
        const uintptr_t begin = reinterpret_cast<uintptr_t>(x), end = reinterpret_cast<uintptr_t>(x + a.V);
#pragma unroll
        for (int i = 0; i < PER; ++i)
            w[i].w = load_words(begin + (e0 + (tid + i * ADJ_NT) * VW) * int64_t(sizeof(T)), begin, end);
    }
    const bool hist = a.tokens != nullptr, bias = a.bias_starts != nullptr;
    // The history's first tokens are on their way before its length is known.
    const int* tok = a.tokens + row * a.ts;
    int4 ahead = make_int4(-1, -1, -1, -1);
    if (hist && a.tokens4 && tid * 4 < a.history) ahead = *reinterpret_cast<const int4*>(tok + tid * 4);
    // The row's mask: mrow -1 none; one that does not exist allows nothing.  Bits of the VW logits from e on.
    int mrow = -1;
    if (a.allowed) mrow = a.allowed_rows ? a.allowed_rows[row] : row;
    const bool none = a.allowed && mrow >= a.masks;
    auto mask = [&](int e) {
        if (none) return 0u;
        if (mrow < 0 || e < 0 || e >= a.V) return ALL;
        const uint32_t* m = a.allowed + int64_t(mrow) * a.words;
        const int k = e >> 5;
        const uint32_t m0 = m[k], m1 = (e & 31) > 32 - VW && k + 1 < a.words ? m[k + 1] : 0u;
        return __funnelshift_r(m0, m1, e & 31) & ALL;
    };
    uint32_t allow[PER];
#pragma unroll
    for (int i = 0; i < PER; ++i) allow[i] = mask(e0 + (tid + i * ADJ_NT) * VW);
    const int len = !hist ? 0 : a.lens ? min(max(a.lens[row], 0), a.history) : a.history;
    const int prompt = a.prompt_lens ? a.prompt_lens[row] : 0;
    float rep = 1.f, pres = 0.f, freq = 0.f;
    int b0 = 0, b1 = 0;
    if (hist) {
        if (a.repetition) rep = a.repetition[row];
        if (a.presence) pres = a.presence[row];
        if (a.frequency) freq = a.frequency[row];
    }
    if (bias) b0 = min(max(a.bias_starts[row], 0), a.biases), b1 = min(a.bias_starts[row + 1], a.biases);
    if (hist || bias) {
        constexpr int N = SEG / 16 + (WIDE ? 2 : 1) * SEG;
        for (int i = tid; i < N / 4; i += ADJ_NT) reinterpret_cast<uint4*>(smem)[i] = make_uint4(0, 0, 0, 0);
        const int lo = max(e0, 0), hi = min(e0 + SEG, a.V);
        __syncthreads();
        for (int i = b0 + tid; i < b1; i += ADJ_NT) {
            const int t = a.bias_tokens[i];
            if (t >= lo && t < hi) {
                atomicOr(&biased[(t - e0) >> 5], 1u << ((t - e0) & 31));
                atomicMax(&which[t - e0], WIDE ? uint32_t(i - b0) + 1 : (uint32_t(i - b0) + 1) << 16);
            }
        }
        if (!WIDE && bias) __syncthreads();     // (counts go into the same words)
        auto add = [&](int t, int i) {
            if (t >= lo && t < hi) {
                atomicOr(&touched[(t - e0) >> 5], 1u << ((t - e0) & 31));
                if (i >= prompt) atomicAdd(&count[t - e0], 1u);
            }
        };
        if (a.tokens4) {
#pragma unroll 2
            for (int i = tid * 4; i < len; i += ADJ_NT * 4) {
                const int4 t = i == tid * 4 ? ahead : *reinterpret_cast<const int4*>(tok + i);
                add(t.x, i);
                if (i + 1 < len) add(t.y, i + 1);
                if (i + 2 < len) add(t.z, i + 2);
                if (i + 3 < len) add(t.w, i + 3);
            }
        } else {
#pragma unroll 4
            for (int i = tid; i < len; i += ADJ_NT) add(tok[i], i);
        }
        __syncthreads();
    }
    // Logit at place i of the segment.
    auto value = [&](float z, int i, bool t, bool b, bool ok) {
        const uint32_t n = t || b ? count[i] : 0u, c = WIDE ? n : n & 0xffffu;
        if (t) {
            z = z > 0.f ? z / rep : z * rep;
            if (c) z = fmaf(-freq, float(c), z) - pres;
        }
        if (b) z += a.bias_values[b0 + int(WIDE ? which[i] : n >> 16) - 1];
        return ok ? z : __int_as_float(0xff800000);
    };
    // Bits of the VW logits from place i (a multiple of VW) on.
    auto bits = [&](const uint32_t* map, int i) { return (map[i >> 5] >> (i & 31)) & ALL; };
#pragma unroll
    for (int i = 0; i < PER; ++i) {
        const int j = tid + i * ADJ_NT, p = j * VW, e = e0 + p;
        if (whole(j)) {
            const uint32_t tb = hist ? bits(touched, p) : 0, bb = bias ? bits(biased, p) : 0, ok = allow[i];
            if (IN_PLACE) {
                if (!(tb | bb) && ok == ALL) continue;
                w[i].w = *reinterpret_cast<const uint4*>(x + e);
            }
            if (tb | bb) {
#pragma unroll
                for (int k = 0; k < VW; ++k)
                    if ((tb | bb) >> k & 1) w[i].e[k] = Num<T>::put(value(Num<T>::get(w[i].e[k]), p + k, tb >> k & 1, bb >> k & 1, true));
            }
            if (ok != ALL) {
#pragma unroll
                for (int k = 0; k < VW; ++k)
                    if (!(ok >> k & 1)) w[i].e[k] = Num<T>::put(__int_as_float(0xff800000));
            }
            __stcs(reinterpret_cast<uint4*>(out + e), w[i].w);
        } else {
            for (int k = 0; k < VW; ++k) {
                if (e + k < 0 || e + k >= a.V) continue;
                const bool t = hist && (touched[(p + k) >> 5] >> ((p + k) & 31) & 1), b = bias && (biased[(p + k) >> 5] >> ((p + k) & 31) & 1);
                const bool ok = mask(e + k) & 1;
                if (t || b || !ok) out[e + k] = Num<T>::put(value(Num<T>::get(x[e + k]), p + k, t, b, ok));
                else if (!IN_PLACE) out[e + k] = x[e + k];
            }
        }
    }
}

template <typename T, bool IN_PLACE, bool WIDE>
static fs_status launch_adjust(const AdjustArgs& a, void* stream) {
    const void* fn = reinterpret_cast<const void*>(adjust_kernel<T, IN_PLACE, WIDE>);
    constexpr int SEG = ADJ_SEG<T>;
    const size_t smem = a.tokens || a.bias_starts ? (SEG / 16 + (WIDE ? 2 : 1) * SEG) * 4 : 0;
    const fs_status st = prepare_kernel(fn);
    if (st != FS_OK) return st;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(unsigned(int64_t(a.B) * a.segs), 1, 1);
    cfg.blockDim = dim3(ADJ_NT, 1, 1);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = static_cast<cudaStream_t>(stream);
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    const cudaError_t e = cudaLaunchKernelEx(&cfg, adjust_kernel<T, IN_PLACE, WIDE>, a);
    return e == cudaSuccess ? FS_OK : cuda_fail(e);
}

template <typename T>
static fs_status adjust_type(AdjustArgs& a, void* stream) {
    // (a row's first word may start up to 15 bytes before it)
    a.segs = int((a.V + 16 / int(sizeof(T)) - 1 + ADJ_SEG<T> - 1) / ADJ_SEG<T>);
    if (int64_t(a.B) * a.segs > 0x7fffffffLL) return FS_ERR_UNSUPPORTED;
    const bool wide = a.history > 65535 || a.biases > 65534, in_place = a.x == a.out && (a.xs == a.os || a.B == 1);
    if (in_place) return wide ? launch_adjust<T, true, true>(a, stream) : launch_adjust<T, true, false>(a, stream);
    return wide ? launch_adjust<T, false, true>(a, stream) : launch_adjust<T, false, false>(a, stream);
}

}  // namespace fsd

extern "C" {

fs_status fs_adjust_logits(const void* logits, int32_t dtype, int64_t row_stride, int32_t batch, int32_t vocab,
                           const int32_t* tokens, int64_t token_stride, int32_t history, const int32_t* lens,
                           const int32_t* prompt_lens, const float* repetition, const float* presence,
                           const float* frequency, const int32_t* bias_starts, const int32_t* bias_tokens,
                           const float* bias_values, int32_t biases, const uint32_t* allowed, int32_t masks,
                           const int32_t* allowed_rows, void* out, int64_t out_stride, void* stream) {
    using namespace fsd;
    if (batch < 0 || vocab < 1 || history < 0 || biases < 0 || masks < 0) return FS_ERR_INVALID_ARG;
    if (dtype != FS_F32 && dtype != FS_BF16 && dtype != FS_F16) return FS_ERR_INVALID_ARG;
    if (vocab > FS_MAX_VOCAB) return FS_ERR_UNSUPPORTED;
    if (batch > 1 && (row_stride < vocab || out_stride < vocab || (tokens && token_stride < history))) return FS_ERR_INVALID_ARG;
    if (!tokens && (lens || prompt_lens || repetition || presence || frequency)) return FS_ERR_INVALID_ARG;
    if (bias_starts ? biases > 0 && (!bias_tokens || !bias_values) : bias_tokens || bias_values || biases) return FS_ERR_INVALID_ARG;
    if (!allowed && (allowed_rows || masks)) return FS_ERR_INVALID_ARG;
    if (allowed && !allowed_rows && masks < batch) return FS_ERR_INVALID_ARG;
    if (batch == 0) return FS_OK;
    if (!logits || !out) return FS_ERR_INVALID_ARG;
    const uintptr_t es = dtype == FS_F32 ? 4 : 2;
    if (reinterpret_cast<uintptr_t>(logits) % es || reinterpret_cast<uintptr_t>(out) % es) return FS_ERR_INVALID_ARG;
    AdjustArgs a = {};
    a.x = logits;
    a.out = out;
    a.xs = row_stride;
    a.os = out_stride;
    a.B = batch;
    a.V = vocab;
    a.tokens = tokens;
    a.ts = token_stride;
    a.history = history;
    a.tokens4 = (reinterpret_cast<uintptr_t>(tokens) % 16 == 0 && (token_stride % 4 == 0 || batch == 1) && history % 4 == 0);
    a.lens = lens;
    a.prompt_lens = prompt_lens;
    a.repetition = repetition;
    a.presence = presence;
    a.frequency = frequency;
    a.bias_starts = bias_starts;
    a.bias_tokens = bias_tokens;
    a.bias_values = bias_values;
    a.biases = biases;
    a.allowed = allowed;
    a.allowed_rows = allowed_rows;
    a.masks = masks;
    a.words = (vocab + 31) / 32;
    if (dtype == FS_F32) return adjust_type<float>(a, stream);
    return dtype == FS_BF16 ? adjust_type<__nv_bfloat16>(a, stream) : adjust_type<__half>(a, stream);
}

}  // extern "C"
