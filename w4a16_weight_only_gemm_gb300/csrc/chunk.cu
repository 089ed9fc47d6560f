// chunk.cu -- attention of chunks of new tokens over the paged cache.
#include <cuda_bf16.h>

#include "common.cuh"
#include "kernels.h"
#include "paged.cuh"

namespace w4a16 {
namespace {

constexpr int kWarps = 4;

struct ChunkArgs {
    const uint16_t *q, *k_pool, *v_pool;
    const int32_t *tables, *lengths, *offsets;
    uint16_t* out;
    float* lse;
    int64_t tokens, q_row, q_head, out_row, out_head;
    int q_heads, group;
    float scale;
    Cache c;
};

// A warp has one head of one token: 32 positions at a time, a lane's score each, then the lanes
// take eight dimensions of V each.
template <typename T>
__global__ void __launch_bounds__(32 * kWarps) chunk_kernel(ChunkArgs a) {
    __shared__ float query[kWarps][256];
    grid_dependency_wait();
    grid_launch_dependents();
    const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
    const int64_t unit = (int64_t)blockIdx.x * kWarps + warp;
    if (unit >= a.tokens * a.q_heads) return;
    const int64_t t = unit / a.q_heads;
    const int h = (int)(unit % a.q_heads), dim = a.c.head_dim;
    const int b = row_of(a.offsets, a.c.batch, t);
    int64_t limit = 0;  // positions that the token sees
    if (b >= 0) {
        const int64_t length = min(max((int64_t)a.lengths[b], (int64_t)0),
                                   (int64_t)a.c.width * a.c.page_size.value);
        limit = max(length - a.offsets[b + 1] + t + 1, (int64_t)0);
    }
    const T* q = reinterpret_cast<const T*>(a.q) + t * a.q_row + h * a.q_head;
    for (int x = lane; x < dim; x += 32) query[warp][x] = (float)q[x];
    __syncwarp();
    const int64_t head = (int64_t)(h / a.group) * a.c.head_stride;
    float m = -INFINITY, l = 0.f, o[8] = {};
    for (int64_t first = 0; first < limit; first += 32) {
        const int64_t p = first + lane;
        int64_t at = -1;
        if (p < limit) {
            const int j = a.c.page_size.quotient((int)p);
            const int64_t page = a.tables[b * a.c.table_stride + j];
            if (page >= 0 && page < a.c.pages)
                at = page * a.c.page_stride + (p - j * a.c.page_size.value) * a.c.slot_stride + head;
        }
        float s = -INFINITY;
        if (at >= 0) {
            s = 0.f;
            const T* k = reinterpret_cast<const T*>(a.k_pool) + at;
            for (int x = 0; x < dim; x += 8) {
                const uint4 piece = *reinterpret_cast<const uint4*>(k + x);
                const T* v = reinterpret_cast<const T*>(&piece);
#pragma unroll
                for (int y = 0; y < 8; ++y) s = fmaf((float)v[y], query[warp][x + y], s);
            }
            s *= a.scale;
        }
        float top = s;
#pragma unroll
        for (int d = 16; d > 0; d /= 2) top = fmaxf(top, __shfl_xor_sync(~0u, top, d));
        top = fmaxf(top, m);
        const float base = top == -INFINITY ? 0.f : top;
        const float keep = expf(m - base), w = expf(s - base);
        m = top;
        l = l * keep + w;
#pragma unroll
        for (int y = 0; y < 8; ++y) o[y] *= keep;
        for (int i = 0; i < 32; ++i) {
            const float weight = __shfl_sync(~0u, w, i);
            const int64_t from = __shfl_sync(~0u, at, i);
            if (from < 0 || 8 * lane >= dim) continue;
            const uint4 piece =
                *reinterpret_cast<const uint4*>(reinterpret_cast<const T*>(a.v_pool) + from + 8 * lane);
            const T* v = reinterpret_cast<const T*>(&piece);
#pragma unroll
            for (int y = 0; y < 8; ++y) o[y] = fmaf(weight, (float)v[y], o[y]);
        }
    }
#pragma unroll
    for (int d = 16; d > 0; d /= 2) l += __shfl_xor_sync(~0u, l, d);
    const float inv = l == 0.f ? 0.f : 1.f / l;
    if (8 * lane < dim) {
        T* to = reinterpret_cast<T*>(a.out) + t * a.out_row + h * a.out_head + 8 * lane;
#pragma unroll
        for (int y = 0; y < 8; ++y) to[y] = (T)(o[y] * inv);
    }
    if (a.lse && lane == 0) a.lse[t * a.q_heads + h] = l == 0.f ? -INFINITY : m + logf(l);
}

}  // namespace

int64_t paged_chunk_workspace(const w4a16_cache_shape&, int64_t, int64_t, const DeviceCtx&) { return 0; }

cudaError_t launch_paged_chunk_attention(const void* q, const void* k_pool, const void* v_pool,
                                         const int32_t* tables, const int32_t* lengths,
                                         const int32_t* offsets, void* out, float* lse, void*,
                                         const w4a16_cache_shape& cache,
                                         const w4a16_query_shape& query, int64_t tokens,
                                         cudaStream_t stream, const DeviceCtx&) {
    ChunkArgs a;
    a.q = static_cast<const uint16_t*>(q);
    a.k_pool = static_cast<const uint16_t*>(k_pool);
    a.v_pool = static_cast<const uint16_t*>(v_pool);
    a.tables = tables;
    a.lengths = lengths;
    a.offsets = offsets;
    a.out = static_cast<uint16_t*>(out);
    a.lse = lse;
    a.tokens = tokens;
    a.q_row = query.q_row_stride;
    a.q_head = query.q_head_stride;
    a.out_row = query.out_row_stride;
    a.out_head = query.out_head_stride;
    a.q_heads = (int)query.q_heads;
    a.group = (int)(query.q_heads / cache.kv_heads);
    a.scale = (float)query.scale;
    a.c = cache_of(cache);
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)((tokens * a.q_heads + kWarps - 1) / kWarps));
    cfg.blockDim = dim3(32 * kWarps);
    cfg.stream = stream;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cache.type == W4A16_BF16 ? cudaLaunchKernelEx(&cfg, chunk_kernel<__nv_bfloat16>, a)
                                    : cudaLaunchKernelEx(&cfg, chunk_kernel<__half>, a);
}

}  // namespace w4a16
