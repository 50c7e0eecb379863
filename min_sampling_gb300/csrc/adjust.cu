// Penalties for repeated tokens, biases and grammar masks on logits (sm_103a).
//
// Row b with logits z, its history's tokens, a list of biases and a bit mask:
//   z > 0 ? z / repetition : z * repetition     where the token is in the history,
//   - frequency * count - presence * (count > 0)   count: how often it is behind the prompt,
//   + bias,   -infinity where the mask has no bit;
// in float32, rounded once.  Bound by memory: every logit is read once and written once.  Two launches:
//   copy_kernel    streams the matrix with the masks applied, 16 KB a CTA
//   change_kernel  the logits of the history's and the biases' tokens.  Each of a row's CTAs takes the tokens whose hash
//                  names it, counts them in a table in shared memory and computes
//                  their logits, while the copy ends; then it writes them.  Where a table overflows, or there would be too many, the
//                  tokens are counted by ranges, a word each.
// 64 rows of 151936 logits in float32 with histories of 4096: 23 us, 3.5 TB/s (copied alone 10 us); 256 of 151665 in bf16
// with masks and histories of 700: 41 us, 3.8 TB/s (copied alone 30 us): what is left is change_kernel's way through a history, of which
// only the copy's last wave is beside it.
// In place, and where there is nothing to mask or to change, one of them is left out. (In one launch, each CTA counting
// for its own 8192 logits: 64 rows of 151936 28 us, 256 of 151665 with masks 64 us; a CTA's way through the history
// is longer than that through its logits.)  No scratch memory, no order that matters: counts are integers, and of
// several biases of one token the last one counts.
#include <algorithm>

#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include "fs_device.cuh"
#include "fs_host.h"

namespace fsd {

constexpr int COPY_NT = 256;                                          // threads of copy_kernel
template <typename T> constexpr int COPY_SEG = 16384 / int(sizeof(T));   // logits of its CTA
constexpr int CHANGE_NT = 512;                                        // threads of change_kernel
constexpr int SLOTS = 4096;                                           // of its table, at most; tokens of a range
constexpr int STAGED = 4096;                                          // tokens of the history in shared memory at a time

struct AdjustArgs {
    const void* x;
    void* out;
    int64_t xs, os;              // row strides (elements)
    int B, V, segs, split;       // split: log2 of change_kernel's CTAs for a row
    int copied;                  // behind copy_kernel
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

// A row's mask: bits of the logits from e on (those past the row's end are undefined).
struct Mask {
    const uint32_t* words;      // nullptr: none
    bool nothing;               // a mask that does not exist allows nothing
    int n;
    __device__ __forceinline__ Mask(const AdjustArgs& a, int row) : words(nullptr), nothing(false), n(a.words) {
        if (!a.allowed) return;
        const int m = a.allowed_rows ? __ldcg(a.allowed_rows + row) : row;
        nothing = m >= a.masks;
        if (m >= 0 && !nothing) words = a.allowed + int64_t(m) * a.words;
    }
    template <int N, bool L2 = false>
    __device__ __forceinline__ uint32_t bits(int e) const {
        constexpr uint32_t ALL = (1u << N) - 1;
        if (!words) return nothing ? 0u : ALL;
        const int k = e >> 5;
        const uint32_t w = L2 ? __ldcg(words + k) : words[k];
        return __funnelshift_r(w, (e & 31) > 32 - N && k + 1 < n ? words[k + 1] : 0u, e & 31) & ALL;
    }
};

template <typename T, bool IN_PLACE>
__global__ void __launch_bounds__(COPY_NT) copy_kernel(const AdjustArgs a) {
    constexpr int SEG = COPY_SEG<T>, VW = 16 / sizeof(T), PER = SEG / VW / COPY_NT;
    constexpr uint32_t ALL = (1u << VW) - 1;
    const int tid = threadIdx.x;
    grid_dependency_wait();
    allow_dependents();
    const int row = blockIdx.x / a.segs, seg = blockIdx.x - row * a.segs;
    const T* x = static_cast<const T*>(a.x) + row * a.xs;
    T* out = static_cast<T*>(a.out) + row * a.os;
    // The output's 16-byte words: word j of the segment holds logits e0 + j VW on.
    const int mis = int((reinterpret_cast<uintptr_t>(out) & 15) / sizeof(T));
    const int e0 = seg * SEG - mis;
    auto whole = [&](int e) { return e >= 0 && e + VW <= a.V; };
    Words<T> w[PER];
    if (!IN_PLACE) {
        const uintptr_t begin = reinterpret_cast<uintptr_t>(x), end = reinterpret_cast<uintptr_t>(x + a.V);
#pragma unroll
        for (int i = 0; i < PER; ++i)
            w[i].w = load_words(begin + (e0 + (tid + i * COPY_NT) * VW) * int64_t(sizeof(T)), begin, end);
    }
    const Mask mask(a, row);
    uint32_t allow[PER];
#pragma unroll
    for (int i = 0; i < PER; ++i) {
        const int e = e0 + (tid + i * COPY_NT) * VW;
        allow[i] = whole(e) ? mask.bits<VW>(e) : ALL;
    }
    const T banned = Num<T>::put(__int_as_float(0xff800000));
#pragma unroll
    for (int i = 0; i < PER; ++i) {
        const int e = e0 + (tid + i * COPY_NT) * VW;
        if (whole(e)) {
            if (IN_PLACE) {
                if (allow[i] == ALL) continue;
                w[i].w = *reinterpret_cast<const uint4*>(x + e);
            }
            if (allow[i] != ALL) {
#pragma unroll
                for (int k = 0; k < VW; ++k)
                    if (!(allow[i] >> k & 1)) w[i].e[k] = banned;
            }
            *reinterpret_cast<uint4*>(out + e) = w[i].w;
        } else {
            for (int k = max(-e, 0); k < VW && e + k < a.V; ++k) {
                if (!mask.bits<1>(e + k)) out[e + k] = banned;
                else if (!IN_PLACE) out[e + k] = x[e + k];
            }
        }
    }
}

// Per token: its count, with bit 31 when it is in the history, and the number of its last bias plus one.
template <typename T>
__global__ void __launch_bounds__(CHANGE_NT, 2) change_kernel(const AdjustArgs a) {
    constexpr uint32_t SEEN = 0x80000000u, EMPTY = 0xffffffffu;
    extern __shared__ __align__(16) uint32_t smem[];
    const int tid = threadIdx.x;
    // (Behind copy_kernel, what that one waited for is there: in L2, from which all is read; an SM's L1 may hold what was there before.)
    if (!a.copied) grid_dependency_wait();
    allow_dependents();
    const int row = blockIdx.x >> a.split, part = blockIdx.x & ((1 << a.split) - 1);
    const T* x = static_cast<const T*>(a.x) + row * a.xs;
    T* out = static_cast<T*>(a.out) + row * a.os;
    const bool hist = a.tokens != nullptr;
    // The history, STAGED tokens at a time; the first are on their way before its length is known.
    const int* tok = a.tokens + row * a.ts;
    int* staged = reinterpret_cast<int*>(smem + 3 * SLOTS + 4);
    auto stage = [&](int first, int last) {
        if (a.tokens4) {
            for (int i = first + tid * 4; i < min(first + STAGED, last); i += CHANGE_NT * 4)    // (rows end behind whole words)
                cp_async16(reinterpret_cast<float*>(staged + i - first), reinterpret_cast<const float*>(tok + i), 16);
        } else {
            for (int i = first + tid; i < min(first + STAGED, last); i += CHANGE_NT) staged[i - first] = __ldcg(tok + i);
        }
        cp_async_commit();
    };
    if (hist) stage(0, a.history);
    const int len = !hist ? 0 : a.lens ? min(max(__ldcg(a.lens + row), 0), a.history) : a.history;
    const int prompt = a.prompt_lens ? __ldcg(a.prompt_lens + row) : 0;
    int b0 = 0, b1 = 0;
    if (a.bias_starts)
        b0 = min(max(__ldcg(a.bias_starts + row), 0), a.biases), b1 = max(min(__ldcg(a.bias_starts + row + 1), a.biases), b0);
    const Mask mask(a, row);
    float rep = 1.f, pres = 0.f, freq = 0.f;
    if (a.repetition) rep = __ldcg(a.repetition + row);
    if (a.presence) pres = __ldcg(a.presence + row);
    if (a.frequency) freq = __ldcg(a.frequency + row);
    // f(token, number in the history) for every token; the first STAGED are in shared memory.
    auto history = [&](bool again, auto f) {
        for (int first = 0; first < len; first += STAGED) {
            if (first > 0 || (again && len > STAGED)) {
                __syncthreads();
                stage(first, len);
            }
            cp_async_wait<0>();
            __syncthreads();
#pragma unroll 1
            for (int i = first + tid; i < min(first + STAGED, len); i += CHANGE_NT) f(staged[i - first], i);
        }
    };
    // A logit z, changed: `n` is its token's count and SEEN.
    auto value = [&](float z, uint32_t n, bool biased, float bias) {
        if (n) {
            z = z > 0.f ? z / rep : z * rep;
            if (n & ~SEEN) z = fmaf(-freq, float(n & ~SEEN), z) - pres;
        }
        return biased ? z + bias : z;
    };
    // Twice as many slots as this CTA's tokens are likely to be.
    const int all = len + b1 - b0, likely = (all >> a.split) + 32;
    volatile uint32_t& full = smem[3 * SLOTS];
    if (tid == 0) full = 0;
    if (all > 0 && 2 * likely <= SLOTS) {
        int bits = 6;
        while ((1 << bits) < 2 * likely) ++bits;
        uint32_t *key = smem, *word = key + (1 << bits), *which = word + (1 << bits);
        for (int i = tid; i < 1 << bits; i += CHANGE_NT) key[i] = EMPTY, word[i] = which[i] = 0;
        __syncthreads();
        // f(slot, number) where the token is this CTA's
        auto find = [&](int t, int i, auto f) {
            const uint32_t g = uint32_t(t) * 2654435769u;
            if (uint32_t(t) >= uint32_t(a.V) || (a.split > 0 && int(g >> (32 - a.split)) != part)) return;
            uint32_t at = g << a.split >> (32 - bits);
            for (int n = 0; n < 1 << bits; ++n) {
                const uint32_t k = atomicCAS(&key[at], EMPTY, uint32_t(t));
                if (k == EMPTY || k == uint32_t(t)) {
                    f(at, i);
                    return;
                }
                at = (at + 1) & ((1u << bits) - 1);
            }
            full = 1;
        };
        history(false, [&](int t, int i) {
            find(t, i, [&](uint32_t at, int i) {
                if (i >= prompt) atomicAdd(&word[at], 1u);
                else atomicOr(&word[at], SEEN);
            });
        });
        for (int i = b0 + tid; i < b1; i += CHANGE_NT)
            find(__ldcg(a.bias_tokens + i), i, [&](uint32_t at, int i) { atomicMax(&which[at], uint32_t(i - b0 + 1)); });
        __syncthreads();
        if (!full) {
            // Each slot's logit is computed, and once the copy is done written, by one thread; the loads of all of a thread's
            // slots are in flight together.
            constexpr int PER = SLOTS / CHANGE_NT;
            uint32_t t[PER], biased = 0;
            float z[PER], add[PER];
#pragma unroll
            for (int j = 0; j < PER; ++j) {
                const int i = tid + j * CHANGE_NT;
                t[j] = i < 1 << bits ? key[i] : EMPTY;
            }
#pragma unroll
            for (int j = 0; j < PER; ++j)
                if (t[j] != EMPTY) z[j] = Num<T>::get(__ldcg(x + t[j]));
#pragma unroll
            for (int j = 0; j < PER; ++j) {
                if (t[j] == EMPTY) continue;
                const uint32_t b = which[tid + j * CHANGE_NT];
                if (b) biased |= 1u << j, add[j] = __ldcg(a.bias_values + b0 + int(b) - 1);
            }
#pragma unroll
            for (int j = 0; j < PER; ++j) {
                if (t[j] == EMPTY) continue;
                if (mask.bits<1, true>(int(t[j]))) z[j] = value(z[j], word[tid + j * CHANGE_NT], biased >> j & 1, add[j]);
                else t[j] = EMPTY;      // (the copy's -infinity stays)
            }
            if (a.copied) grid_dependency_wait();
#pragma unroll
            for (int j = 0; j < PER; ++j)
                if (t[j] != EMPTY) out[t[j]] = Num<T>::put(z[j]);
            return;
        }
    }
    __syncthreads();
    if (a.copied) grid_dependency_wait();
    cp_async_wait<0>();
    if (all == 0) return;
    // By ranges.  (A CTA whose table was full takes its own tokens in all of them; else the row's CTAs share the ranges.)
    const bool own = full;
    uint32_t *word = smem, *which = smem + SLOTS;
    auto mine = [&](int t) { return !own || a.split == 0 || int(uint32_t(t) * 2654435769u >> (32 - a.split)) == part; };
    const int64_t step = int64_t(SLOTS) << (own ? 0 : a.split);
    for (int64_t lo = own ? 0 : part * SLOTS; lo < a.V; lo += step) {
        const int first = int(lo), n = min(SLOTS, a.V - first);
        __syncthreads();
        for (int i = tid; i < 2 * SLOTS; i += CHANGE_NT) smem[i] = 0;
        __syncthreads();
        for (int i = b0 + tid; i < b1; i += CHANGE_NT) {
            const int t = a.bias_tokens[i];
            if (t >= first && t - first < n && mine(t)) atomicMax(&which[t - first], uint32_t(i - b0 + 1));
        }
        history(true, [&](int t, int i) {
            if (t >= first && t - first < n && mine(t)) {
                if (i >= prompt) atomicAdd(&word[t - first], 1u);
                else atomicOr(&word[t - first], SEEN);
            }
        });
        __syncthreads();
        for (int i = tid; i < n; i += CHANGE_NT) {
            const uint32_t c = word[i], b = which[i];
            if ((c | b) && mask.bits<1>(first + i))
                out[first + i] = Num<T>::put(value(Num<T>::get(x[first + i]), c, b != 0, b ? a.bias_values[b0 + int(b) - 1] : 0.f));
        }
    }
}

template <typename K>
static fs_status launch_adjust(K kernel, unsigned grid, unsigned block, size_t smem, const AdjustArgs& a, void* stream) {
    const fs_status st = prepare_kernel(reinterpret_cast<const void*>(kernel));
    if (st != FS_OK) return st;
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

template <typename T>
static fs_status adjust_type(AdjustArgs& a, void* stream) {
    int sms = 0;
    size_t optin = 0;
    fs_status st = device_limits(sms, optin);
    if (st != FS_OK) return st;
    // (a row's first word may start up to 15 bytes before it)
    a.segs = int((a.V + 16 / int(sizeof(T)) - 1 + COPY_SEG<T> - 1) / COPY_SEG<T>);
    const bool in_place = a.x == a.out && (a.xs == a.os || a.B == 1), change = a.tokens || a.bias_starts;
    // A row's CTAs: one for about 512 tokens of the history while all of them fit the GPU at once (two on an SM), and more
    // than that only where the table would be too small.  (64 rows of 151936 and histories of 4096: 256 CTAs 28.7 us, 512 32.8, with
    // the caches flushed.)
    a.split = 0;
    while (a.split < 6 && (512 << a.split) < a.history &&
           ((int64_t(a.B) << (a.split + 1)) <= 2 * sms || 2 * ((a.history >> a.split) + 64) > SLOTS))
        ++a.split;
    if (int64_t(a.B) * std::max(a.segs, 1 << a.split) > 0x7fffffffLL) return FS_ERR_UNSUPPORTED;
    const auto changes = [&](auto kernel) { return launch_adjust(kernel, unsigned(a.B << a.split), CHANGE_NT, (3 * SLOTS + 4 + STAGED) * 4, a, stream); };
    a.copied = !in_place || a.allowed;
    if (a.copied) {
        st = in_place ? launch_adjust(copy_kernel<T, true>, unsigned(a.B * a.segs), COPY_NT, 0, a, stream)
                      : launch_adjust(copy_kernel<T, false>, unsigned(a.B * a.segs), COPY_NT, 0, a, stream);
        if (st != FS_OK) return st;
    }
    return change ? changes(change_kernel<T>) : FS_OK;
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
    if (vocab > FS_MAX_VOCAB || history >= 1 << 30) return FS_ERR_UNSUPPORTED;
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
