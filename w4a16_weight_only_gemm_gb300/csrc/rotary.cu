// rotary.cu -- rotary positions, alone and on the way into the paged cache.
//
// A pair (a, b) of a head's values at position p becomes
//   m (a cos pw - b sin pw),  m (a sin pw + b cos pw)
// with the pair's rate w and the rotation's magnitude m.  A rate is held as its
// fraction of a turn, w / 2 pi, in 64-bit fixed point: times the position modulo
// 2^64 that is the angle's own fraction of a turn, exactly reduced for any
// position of 32 bits (off by 2^-33 turns at most, from the rate's last bit).
// An angle in FP32 would be off by 2^-8 radians at position 131071.
//
// Bound by HBM: 3 FLOPs a value.  A block takes a few tokens, finds their
// positions (and places in the cache), fills a table of their cosines and
// sines, which all heads share, and then works through units of 2 V values,
// the two halves of V pairs: 16-byte pieces where a head has a multiple of 8
// pairs.  Values of dimensions that are not rotated, and V's heads, are copied.
#include <cuda_bf16.h>

#include <algorithm>
#include <type_traits>

#include "common.cuh"
#include "kernels.h"
#include "paged.cuh"

namespace w4a16 {
namespace {

constexpr int kThreads = 256;
constexpr int kMostTokens = 16;  // of a block
constexpr int kMostPairs = 128;
constexpr int kUnroll = 2;       // units of a thread in flight

struct RotaryArgs {
    const void *q, *k, *v;
    void *out, *k_pool, *v_pool;
    const uint64_t* turns;                       // [pairs]
    const int32_t *positions;                    // of the tokens, or NULL: from starts and offsets
    const int32_t *tables, *starts, *offsets;
    int64_t tokens, q_token, q_head, out_token, out_head, k_token, k_head, v_token, v_head;
    int q_heads, kv_heads, dim, pairs, interleaved;
    float magnitude;
    Cache c;
    int block_tokens;
    // units: of a token, of its rotated heads, and of one head that is rotated or copied
    int rotated_units;
    Divisor token_units, head_units, copy_units;
};

template <typename T>
__device__ __forceinline__ float to_float(T v) {
    return (float)v;
}
template <typename T>
__device__ __forceinline__ T from_float(float v) {
    return (T)v;
}

// V consecutive values, as wide as their bytes allow.
template <typename T, int V>
struct alignas(sizeof(T) * V < 16 ? sizeof(T) * V : 16) Piece {
    T x[V];
};

template <typename T, int V>
__global__ void __launch_bounds__(kThreads) rotary_kernel(RotaryArgs a) {
    using P = Piece<T, V>;
    __shared__ int64_t place[kMostTokens];     // where a token's heads start in the pools, -1: nowhere
    __shared__ int64_t position[kMostTokens];
    __shared__ int claimed[kMostTokens];
    __shared__ __align__(16) float2 table[kMostTokens * kMostPairs];  // cosines and sines
    grid_dependency_wait();
    grid_launch_dependents();
    const int64_t first = (int64_t)blockIdx.x * a.block_tokens;
    const int tokens = (int)min((int64_t)a.block_tokens, a.tokens - first);
    if (a.positions) {
        if (threadIdx.x < tokens) {
            position[threadIdx.x] = a.positions[first + threadIdx.x];
            claimed[threadIdx.x] = 1;
        }
    } else {
        for (int i = threadIdx.x / 32; i < tokens; i += kThreads / 32) {
            const int64_t t = first + i;
            const int b = row_of(a.offsets, a.c.batch, t);
            int64_t at = -1, p = 0;
            if (b >= 0) {
                p = (int64_t)a.starts[b] + t - (a.offsets ? a.offsets[b] : t);
                if (p >= 0 && p < (int64_t)a.c.width * a.c.page_size.value) {
                    const int j = a.c.page_size.quotient((int)p);
                    const int64_t page = a.tables[b * a.c.table_stride + j];
                    if (page >= 0 && page < a.c.pages)
                        at = page * a.c.page_stride + (p - j * a.c.page_size.value) * a.c.slot_stride;
                }
            }
            if (threadIdx.x % 32 == 0) place[i] = at, position[i] = p, claimed[i] = b >= 0;
        }
    }
    __syncthreads();
    for (int i = threadIdx.x; i < tokens * a.pairs; i += kThreads) {
        const int t = i / a.pairs, j = i - t * a.pairs;
        const int64_t turn = (int64_t)((uint64_t)position[t] * a.turns[j]);  // of 2^64
        float s, c;
        sincospif((float)turn * 0x1p-63f, &s, &c);
        table[t * kMostPairs + j] = make_float2(c * a.magnitude, s * a.magnitude);
    }
    __syncthreads();
    const int units = tokens * a.token_units.value;
    for (int u = threadIdx.x; u < units; u += kUnroll * kThreads) {
        P lo[kUnroll], hi[kUnroll];
        T *to[kUnroll], *to_hi[kUnroll];
        const float2* turn[kUnroll];
        bool zero[kUnroll];
#pragma unroll
        for (int n = 0; n < kUnroll; ++n) {
            const int w = u + n * kThreads;
            to[n] = to_hi[n] = nullptr;
            turn[n] = nullptr;
            zero[n] = false;
            if (w >= units) continue;
            const int i = a.token_units.quotient(w);
            int y = w - i * a.token_units.value;
            const bool copied = y >= a.rotated_units;
            if (copied) y -= a.rotated_units;
            const Divisor& per = copied ? a.copy_units : a.head_units;
            int h = per.quotient(y);
            y -= h * per.value;
            // the unit's two pieces begin at x0 and x1 of the head
            int x0, x1;
            if (!copied && y * V < a.pairs) {
                turn[n] = table + i * kMostPairs + y * V;
                x0 = a.interleaved ? 2 * V * y : V * y;
                x1 = a.interleaved ? x0 + V : x0 + a.pairs;
            } else {
                x0 = (copied ? 0 : 2 * a.pairs) + 2 * V * (copied ? y : y - a.pairs / V);
                x1 = x0 + V;
            }
            const T* from;
            if (!copied && h < a.q_heads) {
                from = static_cast<const T*>(a.q) + (first + i) * a.q_token + h * a.q_head;
                to[n] = static_cast<T*>(a.out) + (first + i) * a.out_token + h * a.out_head;
                zero[n] = !claimed[i];
            } else {
                if (place[i] < 0) continue;
                if (!copied) h -= a.q_heads;
                from = copied ? static_cast<const T*>(a.v) + (first + i) * a.v_token + h * a.v_head
                              : static_cast<const T*>(a.k) + (first + i) * a.k_token + h * a.k_head;
                to[n] = static_cast<T*>(copied ? a.v_pool : a.k_pool) + place[i] + h * a.c.head_stride;
            }
            if (x1 < a.dim) to_hi[n] = to[n] + x1;
            to[n] += x0;
            lo[n] = *reinterpret_cast<const P*>(from + x0);
            if (to_hi[n]) hi[n] = *reinterpret_cast<const P*>(from + x1);
        }
#pragma unroll
        for (int n = 0; n < kUnroll; ++n) {
            if (!to[n]) continue;
            if (turn[n]) {
#pragma unroll
                for (int j = 0; j < V; ++j) {
                    // the pair's places in the two pieces, in either layout
                    const float2 z = turn[n][j];
                    if (a.interleaved) {
                        T& x = 2 * j < V ? lo[n].x[2 * j % V] : hi[n].x[2 * j % V];
                        T& y = 2 * j + 1 < V ? lo[n].x[(2 * j + 1) % V] : hi[n].x[(2 * j + 1) % V];
                        const float p = to_float(x), q = to_float(y);
                        x = from_float<T>(p * z.x - q * z.y);
                        y = from_float<T>(p * z.y + q * z.x);
                    } else {
                        const float p = to_float(lo[n].x[j]), q = to_float(hi[n].x[j]);
                        lo[n].x[j] = from_float<T>(p * z.x - q * z.y);
                        hi[n].x[j] = from_float<T>(p * z.y + q * z.x);
                    }
                }
            }
            if (zero[n]) {
#pragma unroll
                for (int j = 0; j < V; ++j) lo[n].x[j] = hi[n].x[j] = from_float<T>(0.f);
            }
            *reinterpret_cast<P*>(to[n]) = lo[n];
            if (to_hi[n]) *reinterpret_cast<P*>(to_hi[n]) = hi[n];
        }
    }
}

template <typename T, int V>
cudaError_t launch(RotaryArgs a, cudaStream_t stream, const DeviceCtx& ctx) {
    const int head = a.pairs / V + (a.dim - 2 * a.pairs + 2 * V - 1) / (2 * V);
    const int copied = (a.dim + 2 * V - 1) / (2 * V);
    a.rotated_units = (a.q_heads + a.kv_heads) * head;
    const int units = a.rotated_units + (a.v ? a.kv_heads : 0) * copied;
    a.head_units = Divisor(head);
    a.copy_units = Divisor(copied);
    a.token_units = Divisor(units);
    // up to 16 tokens a block and four units a thread, while that leaves four blocks an SM
    const int64_t most = (int64_t)4 * kThreads / units;
    a.block_tokens = (int)std::max<int64_t>(
        1, std::min({(int64_t)kMostTokens, a.tokens / (4 * ctx.num_sms), most}));
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)((a.tokens + a.block_tokens - 1) / a.block_tokens));
    cfg.blockDim = dim3(kThreads);
    cfg.stream = stream;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, rotary_kernel<T, V>, a);
}

template <typename T>
cudaError_t launch(const RotaryArgs& a, cudaStream_t stream, const DeviceCtx& ctx) {
    if (a.pairs % 8 == 0) return launch<T, 8>(a, stream, ctx);
    if (a.pairs % 4 == 0) return launch<T, 4>(a, stream, ctx);
    if (a.pairs % 2 == 0) return launch<T, 2>(a, stream, ctx);
    return launch<T, 1>(a, stream, ctx);
}

cudaError_t launch(const RotaryArgs& a, int64_t type, cudaStream_t stream, const DeviceCtx& ctx) {
    if (type == W4A16_BF16) return launch<__nv_bfloat16>(a, stream, ctx);
    return type == W4A16_F16 ? launch<__half>(a, stream, ctx) : launch<float>(a, stream, ctx);
}

}  // namespace

cudaError_t launch_rotate(const void* x, const int32_t* positions, const uint64_t* turns, void* out,
                          const w4a16_rotary_shape& rotary, const w4a16_heads_shape& heads,
                          cudaStream_t stream, const DeviceCtx& ctx) {
    RotaryArgs a = {};
    a.q = x;
    a.out = out;
    a.turns = turns;
    a.positions = positions;
    a.tokens = heads.tokens;
    a.q_token = heads.token_stride;
    a.q_head = heads.head_stride;
    a.out_token = heads.out_token_stride;
    a.out_head = heads.out_head_stride;
    a.q_heads = (int)heads.heads;
    a.dim = (int)heads.head_dim;
    a.pairs = (int)(rotary.dims / 2);
    a.interleaved = (int)rotary.interleaved;
    a.magnitude = (float)rotary.magnitude;
    return launch(a, heads.type, stream, ctx);
}

cudaError_t launch_paged_append_rotary(const void* k, const void* v, const uint64_t* turns,
                                       void* k_pool, void* v_pool, const int32_t* tables,
                                       const int32_t* starts, const int32_t* offsets, const void* q,
                                       void* out, const w4a16_cache_shape& cache,
                                       const w4a16_rotary_shape& rotary,
                                       const w4a16_heads_shape& queries, int64_t k_token,
                                       int64_t k_head, int64_t v_token, int64_t v_head,
                                       cudaStream_t stream, const DeviceCtx& ctx) {
    RotaryArgs a = {};
    a.q = q;
    a.k = k;
    a.v = v;
    a.out = out;
    a.k_pool = k_pool;
    a.v_pool = v_pool;
    a.turns = turns;
    a.tables = tables;
    a.starts = starts;
    a.offsets = offsets;
    a.tokens = queries.tokens;
    a.q_token = queries.token_stride;
    a.q_head = queries.head_stride;
    a.out_token = queries.out_token_stride;
    a.out_head = queries.out_head_stride;
    a.k_token = k_token;
    a.k_head = k_head;
    a.v_token = v_token;
    a.v_head = v_head;
    a.q_heads = q ? (int)queries.heads : 0;
    a.kv_heads = (int)cache.kv_heads;
    a.dim = (int)cache.head_dim;
    a.pairs = (int)(rotary.dims / 2);
    a.interleaved = (int)rotary.interleaved;
    a.magnitude = (float)rotary.magnitude;
    a.c = cache_of(cache);
    return launch(a, cache.type, stream, ctx);
}

}  // namespace w4a16
