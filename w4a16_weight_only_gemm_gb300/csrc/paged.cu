// paged.cu -- the paged key-value cache: new tokens into their pages, and the
// attention of one new token over them.
#include <cuda_bf16.h>

#include "common.cuh"
#include "kernels.h"

namespace w4a16 {
namespace {

// A cache's geometry; strides in elements (2 bytes).
struct Cache {
    int64_t pages, page_stride, slot_stride, head_stride, table_stride;
    int page_size, kv_heads, head_dim, batch, width;
};

Cache cache_of(const w4a16_cache_shape& c) {
    return {c.pages,          c.page_stride,    c.slot_stride, c.head_stride,
            c.table_stride,   (int)c.page_size, (int)c.kv_heads, (int)c.head_dim,
            (int)c.batch,     (int)c.table_width};
}

// ---------------------------------------------------------------------------
// Append
// ---------------------------------------------------------------------------
constexpr int kAppendThreads = 256;

struct AppendArgs {
    const uint16_t *k, *v;
    uint16_t *k_pool, *v_pool;
    const int32_t *tables, *starts, *offsets;
    int64_t tokens, k_token, k_head, v_token, v_head;
    Cache c;
};

// The row whose [offsets[b], offsets[b + 1]) holds the token; -1: none does.
__device__ int row_of(const AppendArgs& a, int64_t token) {
    if (!a.offsets) return (int)token;
    int lo = 0, hi = a.c.batch;  // the last row that starts at or before the token
    while (lo < hi) {
        const int mid = (lo + hi) / 2;
        if (a.offsets[mid] <= token)
            lo = mid + 1;
        else
            hi = mid;
    }
    return lo - 1 >= 0 && token < a.offsets[lo] ? lo - 1 : -1;
}

__global__ void __launch_bounds__(kAppendThreads) append_kernel(AppendArgs a) {
    const int vectors = a.c.head_dim / 8, per = a.c.kv_heads * vectors;
    for (int64_t t = blockIdx.x; t < a.tokens; t += gridDim.x) {
        const int b = row_of(a, t);
        if (b < 0) continue;
        const int64_t p = (int64_t)a.starts[b] + t - (a.offsets ? a.offsets[b] : t);
        if (p < 0 || p >= (int64_t)a.c.width * a.c.page_size) continue;
        const int64_t page = a.tables[b * a.c.table_stride + p / a.c.page_size];
        if (page < 0 || page >= a.c.pages) continue;
        const int64_t to = page * a.c.page_stride + p % a.c.page_size * a.c.slot_stride;
        for (int i = threadIdx.x; i < 2 * per; i += kAppendThreads) {
            const bool value = i >= per;
            const int h = i % per / vectors, x = i % per % vectors * 8;
            const uint16_t* from = value ? a.v + t * a.v_token + h * a.v_head
                                         : a.k + t * a.k_token + h * a.k_head;
            uint16_t* dst = (value ? a.v_pool : a.k_pool) + to + h * a.c.head_stride;
            *reinterpret_cast<uint4*>(dst + x) = *reinterpret_cast<const uint4*>(from + x);
        }
    }
}

// ---------------------------------------------------------------------------
// Attention
// ---------------------------------------------------------------------------
template <typename T>
__device__ __forceinline__ float to_float(T v);
template <>
__device__ __forceinline__ float to_float(__half v) { return __half2float(v); }
template <>
__device__ __forceinline__ float to_float(__nv_bfloat16 v) { return __bfloat162float(v); }
template <typename T>
__device__ __forceinline__ T from_float(float v);
template <>
__device__ __forceinline__ __half from_float(float v) { return __float2half_rn(v); }
template <>
__device__ __forceinline__ __nv_bfloat16 from_float(float v) { return __float2bfloat16_rn(v); }

constexpr int kAttendWarps = 4;
constexpr int kMaxDim = 256;

template <typename T>
struct AttendArgs {
    const T *q, *k_pool, *v_pool;
    const int32_t *tables, *lengths;
    T* out;
    float* lse;
    int q_heads, group;
    int64_t q_row, q_head, out_row, out_head;
    float scale;
    Cache c;
};

// One block a (row, query head); a warp takes every fourth position, a lane
// every 32nd element, with a running maximum and sum; the warps join at the end.
template <typename T>
__global__ void __launch_bounds__(32 * kAttendWarps) attend_kernel(AttendArgs<T> a) {
    __shared__ float part[kAttendWarps][kMaxDim], top[kAttendWarps], total[kAttendWarps];
    const int h = blockIdx.x, b = blockIdx.y, warp = threadIdx.x / 32, lane = threadIdx.x % 32;
    const int d = a.c.head_dim;
    const int64_t most = (int64_t)a.c.width * a.c.page_size;
    const int64_t n = min((int64_t)max(a.lengths[b], 0), most);
    float q[kMaxDim / 32], o[kMaxDim / 32], m = -INFINITY, l = 0.f;
#pragma unroll
    for (int i = 0; i < kMaxDim / 32; ++i) {
        const int x = 32 * i + lane;
        q[i] = x < d ? to_float(a.q[b * a.q_row + h * a.q_head + x]) * a.scale : 0.f;
        o[i] = 0.f;
    }
    for (int64_t p = warp; p < n; p += kAttendWarps) {
        const int64_t page = a.tables[b * a.c.table_stride + p / a.c.page_size];
        if (page < 0 || page >= a.c.pages) continue;
        const int64_t at = page * a.c.page_stride + p % a.c.page_size * a.c.slot_stride +
                           h / a.group * a.c.head_stride;
        float s = 0.f;
#pragma unroll
        for (int i = 0; i < kMaxDim / 32; ++i)
            if (32 * i + lane < d) s += q[i] * to_float(a.k_pool[at + 32 * i + lane]);
#pragma unroll
        for (int x = 16; x > 0; x /= 2) s += __shfl_xor_sync(~0u, s, x);
        const float higher = fmaxf(m, s);
        if (higher == -INFINITY) continue;
        const float keep = __expf(m - higher), w = __expf(s - higher);
        l = l * keep + w;
        m = higher;
#pragma unroll
        for (int i = 0; i < kMaxDim / 32; ++i)
            if (32 * i + lane < d)
                o[i] = o[i] * keep + w * to_float(a.v_pool[at + 32 * i + lane]);
    }
#pragma unroll
    for (int i = 0; i < kMaxDim / 32; ++i) part[warp][32 * i + lane] = o[i];
    if (lane == 0) top[warp] = m, total[warp] = l;
    __syncthreads();
    m = -INFINITY, l = 0.f;
    for (int w = 0; w < kAttendWarps; ++w) m = fmaxf(m, top[w]);
    float keep[kAttendWarps];
    for (int w = 0; w < kAttendWarps; ++w) {
        keep[w] = top[w] == -INFINITY ? 0.f : __expf(top[w] - m);
        l += total[w] * keep[w];
    }
    for (int x = threadIdx.x; x < d; x += 32 * kAttendWarps) {
        float v = 0.f;
        for (int w = 0; w < kAttendWarps; ++w) v += part[w][x] * keep[w];
        a.out[b * a.out_row + h * a.out_head + x] = from_float<T>(l > 0.f ? v / l : 0.f);
    }
    if (a.lse && threadIdx.x == 0) a.lse[(int64_t)b * a.q_heads + h] = l > 0.f ? m + logf(l) : -INFINITY;
}

template <typename T>
cudaError_t attend(const void* q, const void* k_pool, const void* v_pool, const int32_t* tables,
                   const int32_t* lengths, void* out, float* lse, const w4a16_cache_shape& cache,
                   const w4a16_query_shape& query, cudaStream_t stream) {
    AttendArgs<T> a;
    a.q = static_cast<const T*>(q);
    a.k_pool = static_cast<const T*>(k_pool);
    a.v_pool = static_cast<const T*>(v_pool);
    a.tables = tables;
    a.lengths = lengths;
    a.out = static_cast<T*>(out);
    a.lse = lse;
    a.q_heads = (int)query.q_heads;
    a.group = (int)(query.q_heads / cache.kv_heads);
    a.q_row = query.q_row_stride;
    a.q_head = query.q_head_stride;
    a.out_row = query.out_row_stride;
    a.out_head = query.out_head_stride;
    a.scale = (float)query.scale;
    a.c = cache_of(cache);
    attend_kernel<T><<<dim3((unsigned)query.q_heads, (unsigned)cache.batch), 32 * kAttendWarps, 0,
                       stream>>>(a);
    return cudaGetLastError();
}

}  // namespace

cudaError_t launch_paged_append(const void* k, const void* v, void* k_pool, void* v_pool,
                                const int32_t* tables, const int32_t* starts,
                                const int32_t* offsets, const w4a16_cache_shape& cache,
                                int64_t tokens, int64_t k_token, int64_t k_head, int64_t v_token,
                                int64_t v_head, cudaStream_t stream, const DeviceCtx& ctx) {
    if (tokens == 0) return cudaSuccess;
    AppendArgs a{static_cast<const uint16_t*>(k), static_cast<const uint16_t*>(v),
                 static_cast<uint16_t*>(k_pool),  static_cast<uint16_t*>(v_pool),
                 tables, starts, offsets, tokens, k_token, k_head, v_token, v_head,
                 cache_of(cache)};
    const int64_t ctas = min(tokens, (int64_t)8 * ctx.num_sms);
    append_kernel<<<(unsigned)ctas, kAppendThreads, 0, stream>>>(a);
    return cudaGetLastError();
}

int64_t paged_attention_workspace(const w4a16_cache_shape& cache, int64_t q_heads,
                                  const DeviceCtx& ctx) {
    (void)cache, (void)q_heads, (void)ctx;
    return 16;
}

cudaError_t launch_paged_attention(const void* q, const void* k_pool, const void* v_pool,
                                   const int32_t* tables, const int32_t* lengths, void* out,
                                   float* lse, void* workspace, const w4a16_cache_shape& cache,
                                   const w4a16_query_shape& query, cudaStream_t stream,
                                   const DeviceCtx& ctx) {
    (void)workspace, (void)ctx;
    return cache.type == W4A16_BF16
               ? attend<__nv_bfloat16>(q, k_pool, v_pool, tables, lengths, out, lse, cache, query, stream)
               : attend<__half>(q, k_pool, v_pool, tables, lengths, out, lse, cache, query, stream);
}

}  // namespace w4a16
