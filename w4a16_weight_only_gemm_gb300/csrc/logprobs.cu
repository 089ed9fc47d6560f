// logprobs.cu -- the scores of given tokens under rows of logits: log
// probability, entropy and the likeliest alternatives.
#include <cuda_bf16.h>

#include "common.cuh"
#include "kernels.h"

namespace w4a16 {
namespace {

constexpr int kScoreThreads = 512;
constexpr int kScoreWarps = kScoreThreads / 32;

__device__ __forceinline__ float to_float(__half v) { return __half2float(v); }
__device__ __forceinline__ float to_float(__nv_bfloat16 v) { return __bfloat162float(v); }
__device__ __forceinline__ float to_float(float v) { return v; }

struct ScoreArgs {
    const void *logits, *tokens;
    float *logprob, *entropy, *top_logprobs;
    int32_t* top_ids;
    int64_t rows, vocabulary, row_stride;
    int wide, top;
};

// Whole numbers in the order of the values, NaN above all, -0 equal to 0, and
// of equal values the lower index above the higher.
__device__ __forceinline__ uint64_t rank_of(float x, int index) {
    int bits = __float_as_int(x + 0.f);
    if (x != x) bits = 0x7FFFFFFF;
    const uint32_t ordered = (uint32_t)(bits ^ ((bits >> 31) & 0x7FFFFFFF)) ^ 0x80000000u;
    return ((uint64_t)ordered << 32) | (uint32_t)~index;
}

__device__ uint64_t block_max(uint64_t v, uint64_t* shared) {
#pragma unroll
    for (int d = 16; d > 0; d /= 2) v = max(v, __shfl_xor_sync(~0u, v, d));
    if (threadIdx.x % 32 == 0) shared[threadIdx.x / 32] = v;
    __syncthreads();
    v = shared[threadIdx.x % kScoreWarps];
#pragma unroll
    for (int d = 16; d > 0; d /= 2) v = max(v, __shfl_xor_sync(~0u, v, d));
    __syncthreads();
    return v;
}

__device__ float block_sum(float v, float* shared) {
#pragma unroll
    for (int d = 16; d > 0; d /= 2) v += __shfl_xor_sync(~0u, v, d);
    if (threadIdx.x % 32 == 0) shared[threadIdx.x / 32] = v;
    __syncthreads();
    v = 0.f;
    for (int i = 0; i < kScoreWarps; ++i) v += shared[i];
    __syncthreads();
    return v;
}

// One block a row: the maximum, the two sums under it, then one sweep for each alternative.
template <typename T>
__global__ void __launch_bounds__(kScoreThreads) score_kernel(ScoreArgs a) {
    __shared__ uint64_t shared_rank[kScoreWarps];
    __shared__ float shared_sum[kScoreWarps];
    const int64_t row = blockIdx.x;
    const T* x = static_cast<const T*>(a.logits) + row * a.row_stride;
    const int n = (int)a.vocabulary;
    uint64_t best = 0;
    for (int i = threadIdx.x; i < n; i += kScoreThreads) best = max(best, rank_of(to_float(x[i]), i));
    best = block_max(best, shared_rank);
    const float m = to_float(x[(int)~(uint32_t)best]);
    const bool nothing = m == -INFINITY;
    float s = 0.f, t = 0.f;
    for (int i = threadIdx.x; i < n && !nothing; i += kScoreThreads) {
        const float d = to_float(x[i]) - m, e = expf(d);
        s += e;
        t += e > 0.f ? e * d : (e == 0.f ? 0.f : e);
    }
    s = block_sum(s, shared_sum);
    t = block_sum(t, shared_sum);
    const float ln = logf(s);
    if (threadIdx.x == 0) {
        const int64_t token = a.wide ? static_cast<const int64_t*>(a.tokens)[row]
                                     : static_cast<const int32_t*>(a.tokens)[row];
        const bool inside = token >= 0 && token < n;
        a.logprob[row] = !inside ? NAN : nothing ? -INFINITY : to_float(x[token]) - m - ln;
        a.entropy[row] = nothing ? 0.f : ln - t / s;
    }
    for (int k = 0; k < a.top; ++k) {
        if (threadIdx.x == 0) {
            const int id = (int)~(uint32_t)best;
            a.top_ids[row * a.top + k] = id;
            a.top_logprobs[row * a.top + k] = nothing ? -INFINITY : to_float(x[id]) - m - ln;
        }
        uint64_t next = 0;
        for (int i = threadIdx.x; i < n; i += kScoreThreads) {
            const uint64_t r = rank_of(to_float(x[i]), i);
            if (r < best) next = max(next, r);
        }
        best = block_max(next, shared_rank);
    }
}

}  // namespace

cudaError_t launch_token_logprobs(const void* logits, const void* tokens, float* logprob,
                                  float* entropy, int32_t* top_ids, float* top_logprobs,
                                  int64_t rows, int64_t vocabulary, int64_t row_stride, int type,
                                  int wide, int top, cudaStream_t stream, const DeviceCtx& ctx) {
    (void)ctx;
    ScoreArgs a{logits, tokens, logprob, entropy, top_logprobs, top_ids,
                rows, vocabulary, row_stride, wide, top};
    const unsigned grid = (unsigned)rows;
    if (type == W4A16_F16)
        score_kernel<__half><<<grid, kScoreThreads, 0, stream>>>(a);
    else if (type == W4A16_BF16)
        score_kernel<__nv_bfloat16><<<grid, kScoreThreads, 0, stream>>>(a);
    else
        score_kernel<float><<<grid, kScoreThreads, 0, stream>>>(a);
    return cudaGetLastError();
}

}  // namespace w4a16
