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
// positions (and places in the cache) and fills a table of their cosines and
// sines.  Its threads are dealt out over tokens, over every so manieth head, and
// over units of 2 V values of a head, the two halves of V pairs: 16-byte pieces
// where a head has a multiple of 8 pairs.  So a thread has its pairs' cosines and
// sines in registers and steps from head to head by an addition.  Values of
// dimensions that are not rotated, and V's heads, are copied.
//
// Measured: 16381 tokens of 40 heads of 128, 64 dimensions of each, bf16, 54 us,
// 6.2 TB/s (0.91 of a plain copy); 32749 tokens of 8 + 8 heads into the pages and
// of 32 heads of queries, 123 us, 6.6 TB/s (0.97).  One token 2.4 us, 16 tokens
// into the pages 3.9: launches and dependent reads.  Threads without pairs of
// their own, which read the table for each head, took 82 and 209 us; six blocks an
// SM and more heads in flight were slower.  The 16381 tokens in fp32 111 us (halves
// paired, 6.0 TB/s) and 127 (neighbours): eight pairs of 32 bits and their angles
// spill (68 bytes of stores, 148 of loads a thread).
#include <cuda_bf16.h>

#include <algorithm>
#include <type_traits>

#include "common.cuh"
#include "kernels.h"
#include "paged.cuh"

namespace w4a16 {
namespace {

constexpr int kThreads = 256;    // of a block at most
constexpr int kMostTokens = 16;  // of a block
constexpr int kMostPairs = 128;
constexpr int kUnroll = 2;       // heads of a thread in flight

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
    int units;                        // of a head
    int block_tokens, block_heads;    // tokens of a block, and heads that it takes at a time
    Divisor token_threads, head_units;
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

template <typename T>
__device__ __forceinline__ uint32_t pack2(float2 v) {
    if constexpr (std::is_same<T, __half>::value) {
        const __half2 h = __float22half2_rn(v);
        return *reinterpret_cast<const uint32_t*>(&h);
    } else {
        const __nv_bfloat162 h = __float22bfloat162_rn(v);
        return *reinterpret_cast<const uint32_t*>(&h);
    }
}
template <typename T>
__device__ __forceinline__ float2 unpack2(uint32_t v) {
    if constexpr (std::is_same<T, __half>::value)
        return __half22float2(*reinterpret_cast<const __half2*>(&v));
    else
        return __bfloat1622float2(*reinterpret_cast<const __nv_bfloat162*>(&v));
}

// The turned pieces.  16-bit values are taken in twos (a conversion at a time runs on a pipe of a
// quarter of the rate).
template <typename T, int V>
__device__ __forceinline__ void turn(Piece<T, V>& lo, Piece<T, V>& hi, const float2 (&cs)[V],
                                     bool interleaved) {
    if constexpr (sizeof(T) == 2 && V >= 2) {
        uint32_t* a = reinterpret_cast<uint32_t*>(&lo);
        uint32_t* b = reinterpret_cast<uint32_t*>(&hi);
        if (interleaved) {
#pragma unroll
            for (int j = 0; j < V; ++j) {
                uint32_t& w = j < V / 2 ? a[j] : b[j - V / 2];
                const float2 v = unpack2<T>(w), z = cs[j];
                w = pack2<T>(make_float2(v.x * z.x - v.y * z.y, v.x * z.y + v.y * z.x));
            }
        } else {
#pragma unroll
            for (int j = 0; j < V / 2; ++j) {
                const float2 x = unpack2<T>(a[j]), y = unpack2<T>(b[j]), z = cs[2 * j], n = cs[2 * j + 1];
                a[j] = pack2<T>(make_float2(x.x * z.x - y.x * z.y, x.y * n.x - y.y * n.y));
                b[j] = pack2<T>(make_float2(x.x * z.y + y.x * z.x, x.y * n.y + y.y * n.x));
            }
        }
    } else {
#pragma unroll
        for (int j = 0; j < V; ++j) {
            const float2 z = cs[j];
            // the pair's places in the two pieces
            T& x = !interleaved ? lo.x[j] : 2 * j < V ? lo.x[2 * j % V] : hi.x[2 * j % V];
            T& y = !interleaved ? hi.x[j] : 2 * j + 1 < V ? lo.x[(2 * j + 1) % V] : hi.x[(2 * j + 1) % V];
            const float p = to_float(x), q = to_float(y);
            x = from_float<T>(p * z.x - q * z.y);
            y = from_float<T>(p * z.y + q * z.x);
        }
    }
}

// One unit of heads first, first + every, ... below `heads`, from `from` to `to` (of head 0, with
// their strides); turned by cs where `turned`, else copied.  x0, x1: where its pieces begin (x1 < 0:
// there is no second one).
template <typename T, int V>
__device__ __forceinline__ void move_heads(const T* from, int64_t from_head, T* to, int64_t to_head,
                                           int first, int heads, int every, int x0, int x1, bool turned,
                                           bool interleaved, bool zero, const float2 (&cs)[V]) {
    using P = Piece<T, V>;
    for (int h = first; h < heads; h += kUnroll * every) {
        P lo[kUnroll], hi[kUnroll];
#pragma unroll
        for (int n = 0; n < kUnroll; ++n) {
            if (h + n * every >= heads) break;
            const T* at = from + (h + n * every) * from_head;
            lo[n] = *reinterpret_cast<const P*>(at + x0);
            if (x1 >= 0) hi[n] = *reinterpret_cast<const P*>(at + x1);
        }
#pragma unroll
        for (int n = 0; n < kUnroll; ++n) {
            if (h + n * every >= heads) break;
            if (turned) turn<T, V>(lo[n], hi[n], cs, interleaved);
            if (zero) {
#pragma unroll
                for (int j = 0; j < V; ++j) lo[n].x[j] = hi[n].x[j] = from_float<T>(0.f);
            }
            T* at = to + (h + n * every) * to_head;
            *reinterpret_cast<P*>(at + x0) = lo[n];
            if (x1 >= 0) *reinterpret_cast<P*>(at + x1) = hi[n];
        }
    }
}

template <typename T, int V>
__global__ void __launch_bounds__(kThreads, 4) rotary_kernel(RotaryArgs a) {
    __shared__ int64_t place[kMostTokens];     // where a token's heads start in the pools, -1: nowhere
    __shared__ int64_t position[kMostTokens];
    __shared__ int claimed[kMostTokens];
    __shared__ __align__(16) float2 table[kMostTokens * kMostPairs];  // cosines and sines
    grid_dependency_wait();
    grid_launch_dependents();
    const int64_t first = (int64_t)blockIdx.x * a.block_tokens;
    const int tokens = (int)min((int64_t)a.block_tokens, a.tokens - first), threads = blockDim.x;
    if (a.positions) {
        if (threadIdx.x < tokens) {
            position[threadIdx.x] = a.positions[first + threadIdx.x];
            claimed[threadIdx.x] = 1;
        }
    } else {
        for (int i = threadIdx.x / 32; i < tokens; i += threads / 32) {
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
    for (int i = threadIdx.x; i < tokens * a.pairs; i += threads) {
        const int t = i / a.pairs, j = i - t * a.pairs;
        const int64_t turn = (int64_t)((uint64_t)position[t] * a.turns[j]);  // of 2^64
        float s, c;
        sincospif((float)turn * 0x1p-63f, &s, &c);
        table[t * kMostPairs + j] = make_float2(c * a.magnitude, s * a.magnitude);
    }
    __syncthreads();
    const int i = a.token_threads.quotient((int)threadIdx.x);
    if (i >= tokens) return;
    const int in_token = threadIdx.x - i * a.token_threads.value;
    const int h = a.head_units.quotient(in_token), u = in_token - h * a.units;
    const int64_t t = first + i;
    const bool turned = u * V < a.pairs;
    float2 cs[V];
#pragma unroll
    for (int j = 0; j < V; ++j) cs[j] = turned ? table[i * kMostPairs + u * V + j] : make_float2(0.f, 0.f);
    // a copied unit is 2 V values in a row; V's heads are copied throughout
    const int copied = 2 * V * u, copied_hi = copied + V < a.dim ? copied + V : -1;
    const int x0 = turned && !a.interleaved ? V * u : copied;
    const int x1 = turned && !a.interleaved ? V * u + a.pairs : copied_hi;
    move_heads<T, V>(static_cast<const T*>(a.q) + t * a.q_token, a.q_head,
                     static_cast<T*>(a.out) + t * a.out_token, a.out_head, h, a.q_heads, a.block_heads, x0,
                     x1, turned, a.interleaved, !claimed[i], cs);
    if (a.kv_heads == 0 || place[i] < 0) return;
    move_heads<T, V>(static_cast<const T*>(a.k) + t * a.k_token, a.k_head,
                     static_cast<T*>(a.k_pool) + place[i], a.c.head_stride, h, a.kv_heads, a.block_heads, x0,
                     x1, turned, a.interleaved, false, cs);
    move_heads<T, V>(static_cast<const T*>(a.v) + t * a.v_token, a.v_head,
                     static_cast<T*>(a.v_pool) + place[i], a.c.head_stride, h, a.kv_heads, a.block_heads,
                     copied, copied_hi, false, false, false, cs);
}

template <typename T, int V>
cudaError_t launch(RotaryArgs a, cudaStream_t stream, const DeviceCtx& ctx) {
    a.units = (a.dim + 2 * V - 1) / (2 * V);
    // Tokens of a block: as many as leave a block two for each SM, and four threads for a unit's heads;
    // the rest of the threads go over the heads.
    const int64_t most = std::max(1, std::min(kMostTokens, kThreads / (4 * a.units)));
    a.block_tokens = (int)std::max<int64_t>(1, std::min(most, a.tokens / (2 * ctx.num_sms)));
    a.block_heads = std::max(1, std::min(std::max(a.q_heads, a.kv_heads),
                                         kThreads / (a.units * a.block_tokens)));
    a.token_threads = Divisor(a.units * a.block_heads);
    a.head_units = Divisor(a.units);
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)((a.tokens + a.block_tokens - 1) / a.block_tokens));
    cfg.blockDim = dim3((unsigned)((a.units * a.block_heads * a.block_tokens + 31) / 32 * 32));
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
