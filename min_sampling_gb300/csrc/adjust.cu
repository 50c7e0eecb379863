// Penalties for repeated tokens, biases and grammar masks on logits (sm_103a).
//
// Row b with logits z, its history's tokens, a list of biases and a bit mask:
//   z > 0 ? z / repetition : z * repetition     where the token is in the history,
//   - frequency * count - presence * (count > 0)   count: how often it is behind the prompt,
//   + bias,   -infinity where the mask has no bit;
// in float32, rounded once.  Bound by memory: every logit is read once and written once.  A CTA owns a
// segment of a row: its first logits are in flight while it goes through the row's history and
// counts in shared memory the tokens that fall into the segment (a bit for each logit that is touched, so that
// the others look nothing up).  No scratch memory, no order that matters: counts are integers, and of
// several biases of one token the last one counts.  In place only what changes is read and
// written.
#include <algorithm>

#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include "fs_device.cuh"
#include "fs_host.h"

namespace fsd {

constexpr int ADJ_NT = 512;      // threads
constexpr int ADJ_SEG = 8192;    // logits of a CTA

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

// 16 bytes from any address that is a multiple of the element's size.
template <typename T>
__device__ __forceinline__ uint4 load_words(const T* p) {
    const uintptr_t at = reinterpret_cast<uintptr_t>(p);
    const uint32_t off = at & 15;
    const uint4* q = reinterpret_cast<const uint4*>(at - off);
    const uint4 a = __ldcs(q);
    if (off == 0) return a;
    const uint4 b = __ldcs(q + 1);   // (holds the last bytes asked for)
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

// Shared memory: a bit per touched logit, a bit per biased one, counts, then (with biases) the
// number of each logit's last bias, plus one.
template <typename T, bool IN_PLACE>
__global__ void __launch_bounds__(ADJ_NT) adjust_kernel(const AdjustArgs a) {
    constexpr int VW = 16 / sizeof(T), PER = ADJ_SEG / VW / ADJ_NT;
    extern __shared__ __align__(16) uint32_t smem[];
    uint32_t* touched = smem;                       // [ADJ_SEG / 32]
    uint32_t* biased = smem + ADJ_SEG / 32;         // [ADJ_SEG / 32]
    uint32_t* count = smem + ADJ_SEG / 16;          // [ADJ_SEG]
    uint32_t* which = count + ADJ_SEG;              // [ADJ_SEG]
    const int tid = threadIdx.x;
    grid_dependency_wait();
    allow_dependents();
    const int row = blockIdx.x / a.segs, seg = blockIdx.x - row * a.segs;
    const T* x = static_cast<const T*>(a.x) + row * a.xs;
    T* out = static_cast<T*>(a.out) + row * a.os;
    // The output's 16-byte words: word j of the segment holds logits e0 + j VW on.
    const int mis = int((reinterpret_cast<uintptr_t>(out) & 15) / sizeof(T));
    const int e0 = seg * ADJ_SEG - mis;
    auto whole = [&](int j) { return e0 + j * VW >= 0 && e0 + (j + 1) * VW <= a.V; };
    Words<T> w[PER];
    if (!IN_PLACE) {
#pragma unroll
        for (int i = 0; i < PER; ++i) {
            const int j = tid + i * ADJ_NT;
            if (whole(j)) w[i].w = load_words(x + e0 + j * VW);
        }
    }
    const bool hist = a.tokens != nullptr, bias = a.bias_starts != nullptr;
    const int len = !hist ? 0 : a.lens ? min(max(a.lens[row], 0), a.history) : a.history;
    const int prompt = a.prompt_lens ? a.prompt_lens[row] : 0;
    float rep = 1.f, pres = 0.f, freq = 0.f;
    if (hist) {
        if (a.repetition) rep = a.repetition[row];
        if (a.presence) pres = a.presence[row];
        if (a.frequency) freq = a.frequency[row];
    }
    int mrow = -1;      // the row's mask, -1: none
    bool none = false;  // a mask that does not exist: nothing is allowed
    if (a.allowed) {
        mrow = a.allowed_rows ? a.allowed_rows[row] : row;
        none = mrow >= a.masks;
    }
    if (hist || bias) {
        for (int i = tid; i < ADJ_SEG / 16; i += ADJ_NT) smem[i] = 0;
        const int n = (ADJ_SEG * (bias ? 2 : 1)) / 4;
        for (int i = tid; i < n; i += ADJ_NT) reinterpret_cast<uint4*>(count)[i] = make_uint4(0, 0, 0, 0);
        __syncthreads();
        const int* tok = a.tokens + row * a.ts;
        const int lo = max(e0, 0), hi = min(e0 + ADJ_SEG, a.V);
#pragma unroll 4
        for (int i = tid; i < len; i += ADJ_NT) {
            const int t = tok[i];
            if (t >= lo && t < hi) {
                atomicOr(&touched[(t - e0) >> 5], 1u << ((t - e0) & 31));
                if (i >= prompt) atomicAdd(&count[t - e0], 1u);
            }
        }
        if (bias) {
            const int b0 = min(max(a.bias_starts[row], 0), a.biases), b1 = min(a.bias_starts[row + 1], a.biases);
            for (int i = b0 + tid; i < b1; i += ADJ_NT) {
                const int t = a.bias_tokens[i];
                if (t >= lo && t < hi) {
                    atomicOr(&biased[(t - e0) >> 5], 1u << ((t - e0) & 31));
                    atomicMax(&which[t - e0], uint32_t(i) + 1);
                }
            }
        }
        __syncthreads();
    }
    // Logit at place i of the segment.
    auto value = [&](float z, int i, bool t, bool b, bool ok) {
        if (t) {
            z = z > 0.f ? z / rep : z * rep;
            const uint32_t c = count[i];
            if (c) z = fmaf(-freq, float(c), z) - pres;
        }
        if (b) z += a.bias_values[which[i] - 1];
        return ok ? z : __int_as_float(0xff800000);
    };
    constexpr uint32_t ALL = (1u << VW) - 1;
    // Bits of the VW logits from place i (a multiple of VW) on.
    auto bits = [&](const uint32_t* map, int i) { return (map[i >> 5] >> (i & 31)) & ALL; };
    auto mask = [&](int e) {   // from logit e >= 0 on; bits past the row's end are undefined
        if (none) return 0u;
        if (mrow < 0) return ALL;
        const uint32_t* m = a.allowed + int64_t(mrow) * a.words;
        const int k = e >> 5;
        const uint32_t m0 = m[k], m1 = (e & 31) > 32 - VW && k + 1 < a.words ? m[k + 1] : 0u;
        return __funnelshift_r(m0, m1, e & 31) & ALL;
    };
#pragma unroll
    for (int i = 0; i < PER; ++i) {
        const int j = tid + i * ADJ_NT, p = j * VW, e = e0 + p;
        if (whole(j)) {
            const uint32_t tb = hist ? bits(touched, p) : 0, bb = bias ? bits(biased, p) : 0, ok = mask(e);
            if (IN_PLACE) {
                if (!(tb | bb) && ok == ALL) continue;
                w[i].w = *reinterpret_cast<const uint4*>(x + e);
            }
            if ((tb | bb) || ok != ALL) {
#pragma unroll
                for (int k = 0; k < VW; ++k)
                    w[i].e[k] = (tb | bb) >> k & 1 || !(ok >> k & 1)
                                    ? Num<T>::put(value(Num<T>::get(w[i].e[k]), p + k, tb >> k & 1, bb >> k & 1, ok >> k & 1))
                                    : w[i].e[k];
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

template <typename T, bool IN_PLACE>
static fs_status launch_adjust(const AdjustArgs& a, void* stream) {
    const void* fn = reinterpret_cast<const void*>(adjust_kernel<T, IN_PLACE>);
    const size_t smem = a.bias_starts ? (ADJ_SEG / 16 + 2 * ADJ_SEG) * 4 : a.tokens ? (ADJ_SEG / 16 + ADJ_SEG) * 4 : 0;
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
    const cudaError_t e = cudaLaunchKernelEx(&cfg, adjust_kernel<T, IN_PLACE>, a);
    return e == cudaSuccess ? FS_OK : cuda_fail(e);
}

template <typename T>
static fs_status adjust_type(const AdjustArgs& a, void* stream) {
    return a.x == a.out && (a.xs == a.os || a.B == 1) ? launch_adjust<T, true>(a, stream) : launch_adjust<T, false>(a, stream);
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
    // (a row's first word may start up to 15 bytes before it)
    a.segs = int((vocab + 16 / int(es) - 1 + ADJ_SEG - 1) / ADJ_SEG);
    if (int64_t(batch) * a.segs > 0x7fffffffLL) return FS_ERR_UNSUPPORTED;
    a.tokens = tokens;
    a.ts = token_stride;
    a.history = history;
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
