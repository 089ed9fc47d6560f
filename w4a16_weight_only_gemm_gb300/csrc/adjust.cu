// adjust.cu -- penalties, biases and masks on logits before a token is sampled.
//
// With c the times a token was generated, and r, f, p the row's repetition,
// frequency and presence penalties:
//   y = x, or where the prompt or the generation has the token x / r (x > 0), x r (else)
//   y = y - f c - p [c > 0] + bias,   -infinity where the mask's bit is 0.
//
// A copy of the logits, bound by HBM, but for the few tokens that a row has
// said.  Those a block finds without a table in memory: it takes a slice of one
// row's vocabulary, holds a word of counts for each token of it in shared
// memory, and reads the whole history, which the row's other blocks find in L2
// (8191 tokens are 32 KB, as many bytes as 16384 logits of 16 bits).  Counts are
// integers, so the order of the atomics changes nothing.  A piece of 16 bytes
// without a token that was said moves as it is, one that the mask has none of
// is not read, and in place only what changes is touched.
#include <cuda_bf16.h>

#include <algorithm>
#include <mutex>

#include "common.cuh"
#include "kernels.h"

namespace w4a16 {
namespace {

constexpr int kThreads = 512;
constexpr int kMostSlice = 16384;
constexpr int kMostBiases = W4A16_MAX_BIASES;
constexpr int kBiasesEach = (kMostBiases + kThreads - 1) / kThreads;
constexpr uint32_t kPrompt = 1u << 31;  // of a token's word; the rest counts its generation

struct AdjustArgs {
    w4a16_adjust_tensors t;
    w4a16_adjust_shape s;
    int slice, slices;
    bool in_place;
};

__device__ __forceinline__ float to_float(__half v) { return __half2float(v); }
__device__ __forceinline__ float to_float(__nv_bfloat16 v) { return __bfloat162float(v); }
__device__ __forceinline__ float to_float(float v) { return v; }
template <typename T>
__device__ __forceinline__ T from_float(float v) {
    return (T)v;
}

struct Penalties {
    float repetition, presence, frequency;

    __device__ __forceinline__ float apply(float x, uint32_t word) const {
        if (word) x = x > 0.f ? x / repetition : x * repetition;
        const uint32_t count = word & ~kPrompt;
        if (count) x = x - frequency * (float)count - presence;
        return x;
    }
};

template <typename T, int V>
struct alignas(sizeof(T) * V) Piece {
    T x[V];
};

// Whether the row's mask allows token j (all of them without a mask).
__device__ __forceinline__ bool allowed(const uint32_t* mask, int64_t j) {
    return !mask || (mask[j >> 5] >> (j & 31) & 1);
}

// V: logits of a piece, 16 bytes where the rows of logits and out lie alike to that boundary, else 1.
template <typename T, int V>
__global__ void __launch_bounds__(kThreads) adjust_kernel(AdjustArgs a) {
    extern __shared__ __align__(16) uint32_t words[];  // of the slice's tokens
    __shared__ int32_t bias_ids[kMostBiases];
    const int64_t row = blockIdx.x / a.slices;
    const int64_t vocabulary = a.s.vocabulary;
    grid_dependency_wait();
    grid_launch_dependents();
    const T* x = static_cast<const T*>(a.t.logits) + row * a.s.logits_stride;
    T* out = static_cast<T*>(a.t.out) + row * a.s.out_stride;
    const uint32_t* mask = a.t.mask ? a.t.mask + row * a.s.mask_stride : nullptr;
    // The slice begins where a piece does: `shift` values before the row's first one are passed over.
    const int shift = (int)(reinterpret_cast<uintptr_t>(x) / sizeof(T) % V);
    const int64_t begin = (int64_t)(blockIdx.x % a.slices) * a.slice - shift;
    const int64_t from = max(begin, (int64_t)0), to = min(begin + a.slice, vocabulary);
    if (from >= to) return;
    for (int i = threadIdx.x * 4; i < a.slice; i += kThreads * 4)
        *reinterpret_cast<uint4*>(words + i) = make_uint4(0, 0, 0, 0);
    const Penalties p = {a.t.repetition ? a.t.repetition[row] : (float)a.s.repetition,
                         a.t.presence ? a.t.presence[row] : (float)a.s.presence,
                         a.t.frequency ? a.t.frequency[row] : (float)a.s.frequency};
    const int biases = a.t.bias_ids ? (int)a.s.biases : 0;
    for (int i = threadIdx.x; i < biases; i += kThreads)
        bias_ids[i] = a.t.bias_ids[row * a.s.bias_stride + i];
    __syncthreads();
    if (a.t.tokens) {
        const int64_t length = a.t.lengths ? min(max((int64_t)a.t.lengths[row], (int64_t)0), a.s.width)
                                           : a.s.width;
        const int64_t prompt = a.t.prompts ? a.t.prompts[row] : 0;
        const auto note = [&](int64_t i, int64_t token) {
            if (token < from || token >= to) return;
            uint32_t* w = words + (token - begin);
            if (i < prompt)
                atomicOr(w, kPrompt);
            else
                atomicAdd(w, 1u);
        };
        if (a.s.wide) {
            const int64_t* tokens = static_cast<const int64_t*>(a.t.tokens) + row * a.s.token_stride;
#pragma unroll 4
            for (int64_t i = threadIdx.x; i < length; i += kThreads) note(i, tokens[i]);
        } else {
            const int32_t* tokens = static_cast<const int32_t*>(a.t.tokens) + row * a.s.token_stride;
#pragma unroll 4
            for (int64_t i = threadIdx.x; i < length; i += kThreads) note(i, tokens[i]);
        }
    }
    __syncthreads();
    // Biased tokens: what they become is computed before the pass (in place it writes over their
    // logits) and written after it.  A token listed twice is its first listing's, with the biases
    // added in the order of the list.
    float biased[kBiasesEach];
    int mine = 0;
#pragma unroll
    for (int k = 0; k < kBiasesEach; ++k) {
        const int i = threadIdx.x + k * kThreads;
        const int64_t id = i < biases ? bias_ids[i] : -1;
        if (id < from || id >= to || !allowed(mask, id)) continue;
        const float* value = a.t.biases + row * a.s.bias_stride;
        float y = p.apply(to_float(x[id]), words[id - begin]) + value[i];
        bool earlier = false;
        for (int j = 0; j < biases; ++j)
            if (bias_ids[j] == id && j != i) {
                earlier = earlier || j < i;
                y += value[j];
            }
        if (!earlier) mine |= 1 << k;
        biased[k] = y;
    }
    if (biases) __syncthreads();
    const T masked = from_float<T>(-INFINITY);
    for (int i = threadIdx.x * V; i < a.slice; i += kThreads * V) {
        const int64_t j = begin + i;
        if (j + V <= 0 || j >= vocabulary) continue;
        const bool whole = j >= 0 && j + V <= vocabulary;
        uint32_t w[V], any = 0;
#pragma unroll
        for (int k = 0; k < V; ++k) any |= w[k] = words[i + k];
        if (whole) {
            uint32_t bits = ~0u;
            if (mask) {
                // the V bits from token j on, which may lie in two words
                bits = mask[j >> 5];
                const int64_t last = j + V - 1;
                bits = __funnelshift_r(bits, (last >> 5) > (j >> 5) ? mask[last >> 5] : 0, j & 31);
            }
            bits &= (1u << V) - 1;
            const bool full = bits == (1u << V) - 1;
            if (a.in_place && full && !any) continue;
            Piece<T, V> v;
            if (bits) v = *reinterpret_cast<const Piece<T, V>*>(x + j);
            if (any) {
#pragma unroll
                for (int k = 0; k < V; ++k)
                    if (w[k]) v.x[k] = from_float<T>(p.apply(to_float(v.x[k]), w[k]));
            }
            if (!full) {
#pragma unroll
                for (int k = 0; k < V; ++k)
                    if (!(bits >> k & 1)) v.x[k] = masked;
            }
            *reinterpret_cast<Piece<T, V>*>(out + j) = v;
        } else {
#pragma unroll
            for (int k = 0; k < V; ++k) {
                if (j + k < 0 || j + k >= vocabulary) continue;
                const bool in = allowed(mask, j + k);
                if (a.in_place && in && !w[k]) continue;
                T y = x[j + k];
                if (w[k]) y = from_float<T>(p.apply(to_float(y), w[k]));
                out[j + k] = in ? y : masked;
            }
        }
    }
    if (!biases) return;
    __syncthreads();
#pragma unroll
    for (int k = 0; k < kBiasesEach; ++k)
        if (mine >> k & 1) out[bias_ids[threadIdx.x + k * kThreads]] = from_float<T>(biased[k]);
}

template <typename T, int V>
cudaError_t launch(AdjustArgs a, cudaStream_t stream, const DeviceCtx& ctx) {
    static std::once_flag once[64];
    static cudaError_t set[64];
    int device = 0;
    cudaError_t e = cudaGetDevice(&device);
    if (e != cudaSuccess) return e;
    std::call_once(once[device], [&]() {
        set[device] = cudaFuncSetAttribute(adjust_kernel<T, V>,
                                           cudaFuncAttributeMaxDynamicSharedMemorySize, 4 * kMostSlice);
    });
    if (set[device] != cudaSuccess) return set[device];
    // a slice of 16384 tokens, less where that leaves fewer than four blocks an SM
    const int64_t padded = a.s.vocabulary + V - 1;  // a row may begin inside a piece
    int64_t slice = std::min<int64_t>(kMostSlice, padded * a.s.rows / (4 * ctx.num_sms));
    slice = std::max<int64_t>(1024, slice / 1024 * 1024);
    a.slice = (int)slice;
    a.slices = (int)((padded + slice - 1) / slice);
    if (a.s.rows * a.slices >= (int64_t)1 << 31) return cudaErrorInvalidValue;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)(a.s.rows * a.slices));
    cfg.blockDim = dim3(kThreads);
    cfg.dynamicSmemBytes = 4 * slice;
    cfg.stream = stream;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, adjust_kernel<T, V>, a);
}

template <typename T>
cudaError_t launch(const AdjustArgs& a, cudaStream_t stream, const DeviceCtx& ctx) {
    constexpr int V = 16 / sizeof(T);
    // 16-byte pieces where every row of logits and of out begins as far past a 16-byte boundary
    const auto from = reinterpret_cast<uintptr_t>(a.t.logits), to = reinterpret_cast<uintptr_t>(a.t.out);
    const int64_t apart = (a.s.logits_stride - a.s.out_stride) * (int64_t)sizeof(T);
    if ((from - to) % 16 == 0 && (a.s.rows == 1 || apart % 16 == 0))
        return launch<T, V>(a, stream, ctx);
    return launch<T, 1>(a, stream, ctx);
}

}  // namespace

cudaError_t launch_adjust_logits(const w4a16_adjust_tensors& tensors,
                                 const w4a16_adjust_shape& shape, cudaStream_t stream,
                                 const DeviceCtx& ctx) {
    AdjustArgs a;
    a.t = tensors;
    a.s = shape;
    a.in_place = tensors.logits == tensors.out;
    if (shape.rows == 1) a.s.logits_stride = a.s.out_stride = 0;
    if (shape.type == W4A16_BF16) return launch<__nv_bfloat16>(a, stream, ctx);
    return shape.type == W4A16_F16 ? launch<__half>(a, stream, ctx) : launch<float>(a, stream, ctx);
}

}  // namespace w4a16
