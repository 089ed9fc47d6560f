// paged.cu -- the paged key-value cache: new tokens into their pages, and the
// attention of one new token over them.
#include <cuda_bf16.h>

#include <algorithm>
#include <mutex>
#include <type_traits>

#include "common.cuh"
#include "kernels.h"
#include "paged.cuh"

namespace w4a16 {
namespace {

// ---------------------------------------------------------------------------
// Append
//
// A copy, bound by HBM.  A block first finds the places of its few tokens, a
// warp each in turn (the row by a 32-way search of the offsets, then its
// start, then its page: three loads that depend on one another), and then
// copies their 16-byte pieces, four of a thread in flight.
// ---------------------------------------------------------------------------
constexpr int kAppendThreads = 256;
constexpr int kAppendTokens = 16;  // of a block at most
constexpr int kAppendUnroll = 4;

struct AppendArgs {
    const uint16_t *k, *v;
    uint16_t *k_pool, *v_pool;
    const int32_t *tables, *starts, *offsets;
    int64_t tokens, k_token, k_head, v_token, v_head;
    Cache c;
    int block_tokens;
    Divisor token_pieces, head_pieces;  // 16-byte pieces of a token's keys, of a head
};

__global__ void __launch_bounds__(kAppendThreads) append_kernel(AppendArgs a) {
    __shared__ int64_t place[kAppendTokens];  // where a token's heads start in the pools, -1: nowhere
    grid_dependency_wait();
    grid_launch_dependents();
    const int64_t first = (int64_t)blockIdx.x * a.block_tokens;
    const int tokens = (int)min((int64_t)a.block_tokens, a.tokens - first);
    for (int i = threadIdx.x / 32; i < tokens; i += kAppendThreads / 32) {
        const int64_t t = first + i;
        const int b = row_of(a.offsets, a.c.batch, t);
        int64_t at = -1;
        if (b >= 0) {
            const int64_t p = (int64_t)a.starts[b] + t - (a.offsets ? a.offsets[b] : t);
            if (p >= 0 && p < (int64_t)a.c.width * a.c.page_size.value) {
                const int j = a.c.page_size.quotient((int)p);
                const int64_t page = a.tables[b * a.c.table_stride + j];
                if (page >= 0 && page < a.c.pages)
                    at = page * a.c.page_stride + (p - j * a.c.page_size.value) * a.c.slot_stride;
            }
        }
        if (threadIdx.x % 32 == 0) place[i] = at;
    }
    __syncthreads();
    const int units = tokens * a.token_pieces.value;  // of keys, and as many of values
    for (int u = threadIdx.x; u < 2 * units; u += kAppendUnroll * kAppendThreads) {
        uint4 data[kAppendUnroll];
        uint16_t* to[kAppendUnroll];
#pragma unroll
        for (int k = 0; k < kAppendUnroll; ++k) {
            const int w = u + k * kAppendThreads;
            const bool value = w >= units;
            const int x = value ? w - units : w;
            const int i = a.token_pieces.quotient(x), y = x - i * a.token_pieces.value;
            const int h = a.head_pieces.quotient(y), d = (y - h * a.head_pieces.value) * 8;
            const int64_t at = w < 2 * units ? place[i] : -1;
            to[k] = nullptr;
            if (at < 0) continue;
            data[k] = *reinterpret_cast<const uint4*>(
                value ? a.v + (first + i) * a.v_token + h * a.v_head + d
                      : a.k + (first + i) * a.k_token + h * a.k_head + d);
            to[k] = (value ? a.v_pool : a.k_pool) + at + h * a.c.head_stride + d;
        }
#pragma unroll
        for (int k = 0; k < kAppendUnroll; ++k)
            if (to[k]) *reinterpret_cast<uint4*>(to[k]) = data[k];
    }
}

// ---------------------------------------------------------------------------
// Attention
//
// A step is 64 positions of one item (a row's key-value head with up to 16 of
// its query heads); the items' steps, one item after the other, form one line
// that the blocks cut into equal parts, so rows of any lengths load every SM
// alike and one long row is split over all of them.  A block that has all of
// an item writes its output; the others leave (max, sum, unnormalised output)
// in the workspace, and a join kernel adds those up.
//
// Bound by HBM: each key and value is read once and meets `group` FLOPs a
// byte, so what counts is bytes in flight and few instructions a tile.  Each
// warp has a ring of its own in shared memory, filled by cp.async with whole
// 128-byte lines by eight lanes (lines cut in halves cost 1.5 times the traffic
// between L2 and the SM), so it waits for its own copies only and the block
// meets at the end of an item.  Scores are taken transposed, S^T = K Q^T: 16
// positions are the rows of an MMA and 8 query heads its columns, with the
// dimension permuted alike in K and Q so that a lane's operands are 16
// consecutive bytes.  P^T becomes the right operand of O^T = V^T P^T by an 8x8
// transposition between lanes; V^T comes from transposing matrix loads.  The
// 16-byte pieces of a row are swizzled against bank conflicts, K's for the
// lanes' 16-byte reads and V's for the matrix loads.
// P is split in two 16-bit parts, its value and what rounding that left over,
// so that the probabilities keep 22 (fp16) or 16 (bf16) bits: the MMAs are
// far from the bound, and the output is then rounded only once.  The first part
// is rounded down and the second never 0 beside it, so both have the sign of
// the weight: an infinite value meets no zero and no opposite sign, which would
// turn it into NaN.
//
// On one GB300 (6790 GB/s copied), 8 key-value heads of 128 and 4 query heads
// to each: one row of 131071 positions 86.1 us (6240 GB/s), 128 rows of up to
// 8191 318 us (6700 GB/s), one row of 512 4.8 us.  16 rows of up to 4093 with 4
// key-value heads 17.7 us (4030 GB/s): a launch and three reads that depend on
// one another (length, page, keys) before the first tile, the longest rows'
// blocks after the others are done, and the join, about 7 us in all.  32 rows of
// 4096 take 90 us by pages of 16 to 128, 91 by pages of 8, 13 and 24, 89 by 1.
// ---------------------------------------------------------------------------
constexpr int kAttendWarps = 4;
constexpr int kAttendThreads = 32 * kAttendWarps;
constexpr int kTile = 16;                       // positions of a warp in a step
constexpr int kStep = kTile * kAttendWarps;     // positions of a step
constexpr float kLn2 = 0.6931471805599453f;
// Weights are held times 2^12 (2^15 at most): FP16 has nothing between 0 and 2^-24, and many small
// weights in a warp's part would each be rounded to one or the other beside a weight of 1.
constexpr float kHeadroom = 12.f, kMostWeight = 15.f;
constexpr int kMaxCluster = 8;                  // blocks to an item, without the line,
constexpr int kFewSteps = 8, kMostSteps = 32;   // and the most steps of such a block

// What is left for the join: an item that begins in block `first` and is ended
// by the `count` blocks after it (count 0: none).  The place of an item's joint
// is its own number where there are no more items than blocks, so that few
// items need few join blocks, else its first block's.
struct Joint {
    int row, item, count, first;
};

struct AttendArgs {
    const uint16_t *q, *k_pool, *v_pool;
    const int32_t *tables, *lengths;
    uint16_t* out;
    float* lse;
    float* partial;     // [blocks][2][heads of an item][padded dim]
    float2* partial_ml; // [blocks][2][heads of an item]
    Joint* joints;      // [min(blocks, items in all)]
    int by_item;        // whether joints are placed by their items
    int cluster;        // blocks to an item, a cluster, where tables are short; 0: the line is cut
    int q_heads, group;
    int items;          // of a row: kv_heads * blocks of heads
    int head_blocks;    // per key-value head
    int block_heads;    // query heads of an item (the last block may have fewer)
    int64_t q_row, q_head, out_row, out_head;
    float scale_log2;
    Cache c;

    __device__ int length(int row) const {
        return min(max(lengths[row], 0), c.width * c.page_size.value);
    }
    __device__ int64_t head_offset(int item) const {
        return (int64_t)(item / head_blocks) * c.head_stride;
    }
    __device__ int first_head(int item) const {
        return item / head_blocks * group + item % head_blocks * block_heads;
    }
    __device__ int heads_of(int item) const {
        return min(block_heads, group - item % head_blocks * block_heads);
    }
};

template <typename T>
__device__ __forceinline__ uint32_t pack2(float lo, float hi);
template <>
__device__ __forceinline__ uint32_t pack2<__half>(float lo, float hi) {
    const __half2 v = __floats2half2_rn(lo, hi);
    return *reinterpret_cast<const uint32_t*>(&v);
}
template <>
__device__ __forceinline__ uint32_t pack2<__nv_bfloat16>(float lo, float hi) {
    const __nv_bfloat162 v = __floats2bfloat162_rn(lo, hi);
    return *reinterpret_cast<const uint32_t*>(&v);
}
// The same, rounded towards zero.
template <typename T>
__device__ __forceinline__ uint32_t pack2_down(float lo, float hi) {
    uint32_t r;
    if constexpr (std::is_same<T, __half>::value)
        asm("cvt.rz.f16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
    else
        asm("cvt.rz.bf16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
    return r;
}
template <typename T>
__device__ __forceinline__ float2 unpack2(uint32_t v);
template <>
__device__ __forceinline__ float2 unpack2<__half>(uint32_t v) {
    return __half22float2(*reinterpret_cast<const __half2*>(&v));
}
template <>
__device__ __forceinline__ float2 unpack2<__nv_bfloat16>(uint32_t v) {
    return __bfloat1622float2(*reinterpret_cast<const __nv_bfloat162*>(&v));
}

// c += A(16x16) * B(16x8)
template <typename T>
__device__ __forceinline__ void mma(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2,
                                    uint32_t a3, uint32_t b0, uint32_t b1) {
    if constexpr (std::is_same<T, __half>::value)
        asm(
            "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, "
            "{%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, %3};"
            : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
            : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
    else
        asm(
            "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, "
            "{%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, %3};"
            : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
            : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

__device__ __forceinline__ uint32_t transpose8x8(uint32_t v) {
    uint32_t r;
    asm("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(r) : "r"(v));
    return r;
}

// Four 8x8 matrices, transposed; lane i names row i % 8 of matrix i / 8.
__device__ __forceinline__ void load_transposed(uint32_t (&r)[4], uint32_t addr) {
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0, %1, %2, %3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
                 : "r"(addr)
                 : "memory");
}

__device__ __forceinline__ void copy16(uint32_t dst, const void* src) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst), "l"(src) : "memory");
}

// 16 bytes to shared memory, or 16 zero bytes when `there` is false.
__device__ __forceinline__ void copy16(uint32_t dst, const void* src, bool there) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src),
                 "r"(there ? 16 : 0)
                 : "memory");
}

__device__ __forceinline__ void copy_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void copy_wait() {
    asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}

__device__ __forceinline__ float exp2_fast(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

template <int DP, int NT>
struct AttendShape {
    static constexpr int kRowBytes = 2 * DP;
    static constexpr int kHalf = kTile * kRowBytes;     // a warp's keys of 16 positions
    static constexpr int kTileBytes = 2 * kHalf;        // and values
    static constexpr int kStageBytes = kTileBytes * kAttendWarps;
    // 192 KB of ring an SM: as many blocks as registers allow
    static constexpr int kBlocksPerSm =
        DP == 64 ? (NT == 1 ? 4 : 3) : DP == 128 ? (NT == 1 ? 3 : 2) : 1;
    static constexpr int kStages = 192 * 1024 / kBlocksPerSm / kStageBytes;
    // behind the ring, the queries of as many items
    static constexpr int kQueryBytes = 8 * NT * kRowBytes;
    static constexpr int kSmem = kStages * (kStageBytes + kQueryBytes);
};

// A place on the line of steps.
struct Place {
    int row, item, tile, steps, length;
    int64_t head;  // of the item's keys and values in their pools
};

// (unsigned: lengths go up to 2^31 - 1)
__device__ __forceinline__ int steps_of(int length) {
    return (int)(((uint32_t)length + kStep - 1) / kStep);
}

__device__ __forceinline__ void advance(const AttendArgs& a, Place& p) {
    if (++p.tile < p.steps) return;
    p.tile = 0;
    p.item = p.item + 1 == a.items ? 0 : p.item + 1;
    p.head = a.head_offset(p.item);
    if (p.item) return;
    p.steps = 0;
    while (++p.row < a.c.batch) {
        p.length = a.length(p.row);
        p.steps = steps_of(p.length);
        if (p.steps) return;
    }
}

// Four values of a head's output, of sum `l` under the maximum `m` of binary exponents.
template <typename T>
__device__ __forceinline__ void write_out(const AttendArgs& a, int row, int head, int x,
                                          const float4& v, float m, float l) {
    const float inv = l == 0.f ? 0.f : 1.f / l;
    if (x < a.c.head_dim)
        *reinterpret_cast<uint2*>(a.out + row * a.out_row + head * a.out_head + x) =
            make_uint2(pack2<T>(v.x * inv, v.y * inv), pack2<T>(v.z * inv, v.w * inv));
    if (x == 0 && a.lse)
        a.lse[(int64_t)row * a.q_heads + head] = l == 0.f ? -INFINITY : (m + log2f(l)) * kLn2;
}

__device__ __forceinline__ float2 ld_cluster_f2(uint32_t addr) {
    float2 v;
    asm volatile("ld.shared::cluster.v2.f32 {%0, %1}, [%2];"
                 : "=f"(v.x), "=f"(v.y) : "r"(addr) : "memory");
    return v;
}
__device__ __forceinline__ float4 ld_cluster_f4(uint32_t addr) {
    float4 v;
    asm volatile("ld.shared::cluster.v4.f32 {%0, %1, %2, %3}, [%4];"
                 : "=f"(v.x), "=f"(v.y), "=f"(v.z), "=f"(v.w) : "r"(addr) : "memory");
    return v;
}

// The part [lo, hi) of the line that block `index` of `blocks` takes.
__device__ __forceinline__ int64_t cut(int64_t total, int64_t index, int64_t blocks) {
    return total * index / blocks;
}

template <typename T, int DP, int NT, bool kTilePage>
__global__ void __launch_bounds__(kAttendThreads, AttendShape<DP, NT>::kBlocksPerSm)
    attend_kernel(AttendArgs a) {
    using S = AttendShape<DP, NT>;
    constexpr int kHeads = 8 * NT;
    // the least a part of a weight can be: FP16's smallest number, BF16's smallest normal one
    constexpr float kLeast = std::is_same<T, __half>::value ? 0x1p-24f : 0x1p-126f;
    extern __shared__ __align__(16) unsigned char ring[];
    __shared__ int64_t scan[kAttendWarps];
    __shared__ Place begin;
    __shared__ float2 warp_ml[kAttendWarps][kHeads], block_ml[kHeads];
    const int tid = threadIdx.x, warp = tid / 32, lane = tid % 32, g = lane / 4, t = lane % 4;
    const int dim = a.c.head_dim;

    grid_dependency_wait();
    grid_launch_dependents();

    // The line: its length, and where this block's part begins.
    int64_t total = 0, blocks = 0, lo = 0, hi = 0;
    if (a.cluster) {
        const int item = blockIdx.x / a.cluster, rank = blockIdx.x % a.cluster;
        const int row = item / a.items, length = a.length(row), n = steps_of(length);
        lo = cut(n, rank, a.cluster);
        hi = cut(n, rank + 1, a.cluster);
        if (tid == 0)
            begin = {row, item % a.items, (int)lo, n, length, a.head_offset(item % a.items)};
        // a sum below 0: no step, and nothing written at this block's ring's start
        if (tid < kHeads) block_ml[tid] = make_float2(-INFINITY, -1.f);
    } else {
        const int per = (a.c.batch + kAttendThreads - 1) / kAttendThreads;
        const int r0 = min(tid * per, a.c.batch), r1 = min(r0 + per, a.c.batch);
        int64_t mine = 0;
        for (int r = r0; r < r1; ++r) mine += steps_of(a.length(r));
        int64_t upto = mine;
#pragma unroll
        for (int d = 1; d < 32; d *= 2) {
            const int64_t o = __shfl_up_sync(~0u, upto, d);
            if (lane >= d) upto += o;
        }
        if (lane == 31) scan[warp] = upto;
        __syncthreads();
#pragma unroll
        for (int w = 0; w < kAttendWarps; ++w) {
            if (w < warp) upto += scan[w];
            total += scan[w];
        }
        total *= a.items;
        blocks = min((int64_t)gridDim.x, total);
        if (blockIdx.x < blocks) {
            lo = cut(total, blockIdx.x, blocks);
            hi = cut(total, blockIdx.x + 1, blocks);
        }
        if (lo < hi && (upto - mine) * a.items <= lo && lo < upto * a.items) {
            int r = r0;
            int64_t at = (upto - mine) * a.items;
            int n = steps_of(a.length(r));
            while (at + (int64_t)n * a.items <= lo) at += (int64_t)n * a.items, n = steps_of(a.length(++r));
            const int item = (int)((lo - at) / n);
            begin = {r, item, (int)((lo - at) % n), n, a.length(r), a.head_offset(item)};
        }
    }
    if (!a.by_item && !a.cluster && tid == 0) a.joints[blockIdx.x] = {0, 0, 0, 0};
    // rows without a position
    for (int r = blockIdx.x; r < a.c.batch; r += gridDim.x) {
        if (a.length(r) != 0) continue;
        if (a.by_item && !a.cluster)
            for (int i = tid; i < a.items; i += kAttendThreads)
                a.joints[r * a.items + i] = {0, 0, 0, 0};
        for (int h = warp; h < a.q_heads; h += kAttendWarps) {
            for (int x = lane * 8; x < dim; x += 256)
                *reinterpret_cast<uint4*>(a.out + r * a.out_row + h * a.out_head + x) =
                    make_uint4(0, 0, 0, 0);
            if (a.lse && lane == 0) a.lse[(int64_t)r * a.q_heads + h] = -INFINITY;
        }
    }
    __syncthreads();
    if (lo == hi && (a.cluster <= 1 || begin.steps == 0)) return;

    Place ahead = begin, here = begin;
    const uint32_t warp_ring = smem_u32(ring) + warp * S::kTileBytes;
    uint32_t flags = 0;      // two bits a tile in flight: whether positions g and g + 8 count
    const int count = (int)(hi - lo);
    int left = count;        // steps to issue
    int next_page = -1;      // of the tile to issue next: the warp's, or of position `lane`

    const auto load_page = [&]() {
        const int p = ahead.tile * kStep + warp * kTile + (kTilePage ? 0 : lane % kTile);
        next_page = -1;
        if (p < ahead.length) next_page = a.tables[ahead.row * a.c.table_stride + a.c.page_size.quotient(p)];
    };
    // Copies: lane's piece `piece` of rows row0, row0 + kRows, ...
    constexpr int kPieces = DP / 8, kRows = 32 / kPieces;
    const int piece = lane % kPieces, row0 = lane / kPieces;
    const bool in_dim = piece * 8 < dim;
    // The queries of an item come with its first tile: every warp copies all of them to the same
    // place, and each waits for its own copies only.  (Read from memory at the item's start they
    // held up its first tile.)
    const uint32_t queries = smem_u32(ring) + S::kStages * S::kStageBytes;
    int ahead_item = 0, here_item = 0;  // places of the items being issued and taken
    bool ahead_fresh = true;
    const auto issue_queries = [&]() {
        const int heads = a.heads_of(ahead.item);
        const uint16_t* src = a.q + ahead.row * a.q_row +
                              (int64_t)a.first_head(ahead.item) * a.q_head + 8 * piece;
        const uint32_t dst = queries + ahead_item * S::kQueryBytes + row0 * S::kRowBytes;
#pragma unroll
        for (int r = 0; r < kHeads; r += kRows) {
            const int h = row0 + r;
            const bool in = h < heads && in_dim;
            copy16(dst + r * S::kRowBytes + ((piece ^ ((h & 1) << 2 | (h >> 1 & 3))) << 4),
                   in ? src + h * a.q_head : a.q, in);
        }
    };
    const auto issue = [&](int stage) {
        flags <<= 2;
        if (left > 0) {
            --left;
            if (ahead_fresh) issue_queries();
            const int first = ahead.tile * kStep + warp * kTile;
            const bool there = (uint32_t)next_page < (uint32_t)a.c.pages;
            const uint32_t dst = warp_ring + stage * S::kStageBytes + row0 * S::kRowBytes;
            // the swizzle of row r: K's pieces meet 4 to a row in a read, V's 8 to a row
            const auto k_at = [&](int r) {
                const int y = row0 + r;
                return dst + r * S::kRowBytes + ((piece ^ ((y & 1) << 2 | (y >> 1 & 3))) << 4);
            };
            const auto v_at = [&](int r) {
                return dst + S::kHalf + r * S::kRowBytes + ((piece ^ (row0 + r & 7)) << 4);
            };
            if (kTilePage) {
                const int slot = a.c.page_size.remainder(first);
                const int64_t at =
                    next_page * a.c.page_stride + (slot + row0) * a.c.slot_stride + ahead.head + 8 * piece;
                const int n = there ? ahead.length - first : 0;  // positions that count
                const uint16_t *k = a.k_pool + at, *v = a.v_pool + at;
                const int64_t next = kRows * a.c.slot_stride;
                flags |= (uint32_t)(g < n) | (uint32_t)(g + 8 < n) << 1;
                if (n >= kTile && dim == DP) {
#pragma unroll
                    for (int r = 0; r < kTile; r += kRows, k += next, v += next)
                        copy16(k_at(r), k), copy16(v_at(r), v);
                } else {
#pragma unroll
                    for (int r = 0; r < kTile; r += kRows, k += next, v += next) {
                        const bool in = row0 + r < n && in_dim;
                        copy16(k_at(r), in ? k : a.k_pool, in);
                        copy16(v_at(r), in ? v : a.v_pool, in);
                    }
                }
            } else {
                // where position `lane` starts; a page number is looked up below the length only
                const int p = first + lane % kTile;
                const int64_t at = there ? next_page * a.c.page_stride +
                                               a.c.page_size.remainder(p) * a.c.slot_stride +
                                               ahead.head
                                         : -1;
                flags |= (uint32_t)(__shfl_sync(~0u, at, g) >= 0) |
                         (uint32_t)(__shfl_sync(~0u, at, g + 8) >= 0) << 1;
#pragma unroll
                for (int r = 0; r < kTile; r += kRows) {
                    const int64_t o = __shfl_sync(~0u, at, row0 + r);
                    const bool in = o >= 0 && in_dim;
                    copy16(k_at(r), a.k_pool + (in ? o + 8 * piece : 0), in);
                    copy16(v_at(r), a.v_pool + (in ? o + 8 * piece : 0), in);
                }
            }
            advance(a, ahead);
            ahead_fresh = ahead.tile == 0;
            if (ahead_fresh) ahead_item = ahead_item + 1 == S::kStages ? 0 : ahead_item + 1;
            if (left > 0) load_page();
        }
        copy_commit();
    };
    // Reads: K's row g (and g + 8, alike in the swizzle), pieces 4j + t; V's transposed matrices.
    const int k_swizzle = (g & 1) << 2 | (g >> 1 & 3);
    const uint32_t k_lane = warp_ring + g * S::kRowBytes, k_xor = (t ^ k_swizzle) << 4;
    const uint32_t v_lane =
        warp_ring + S::kHalf + ((lane >> 4) * 8 + lane % 8) * S::kRowBytes;
    const uint32_t v_xor = ((lane >> 3 & 1) ^ lane % 8) << 4;

    if (left > 0) load_page();
#pragma unroll 1
    for (int s = 0; s < S::kStages; ++s) issue(s);

    uint4 q[NT][DP / 32];
    float o[NT][DP / 16][4], top[NT][2], sum[NT][2];
    bool fresh = true;
    int first_tile = 0, stage = 0;
#pragma unroll 1
    for (int step = 0; step < count; ++step) {
        copy_wait<S::kStages - 1>();
        __syncwarp();
        if (fresh) {
            fresh = false;
            first_tile = here.tile;
#pragma unroll
            for (int n = 0; n < NT; ++n) {
#pragma unroll
                for (int j = 0; j < DP / 32; ++j)
                    q[n][j] = lds128(queries + here_item * S::kQueryBytes +
                                     (8 * n + g) * S::kRowBytes + (k_xor ^ (64 * j)));
                top[n][0] = top[n][1] = -INFINITY;
                sum[n][0] = sum[n][1] = 0.f;
#pragma unroll
                for (int i = 0; i < DP / 16; ++i)
#pragma unroll
                    for (int x = 0; x < 4; ++x) o[n][i][x] = 0.f;
            }
            here_item = here_item + 1 == S::kStages ? 0 : here_item + 1;
        }
        const uint32_t at = stage * S::kStageBytes;
        float c[NT][4], c2[NT][4];  // two chains
#pragma unroll
        for (int n = 0; n < NT; ++n)
#pragma unroll
            for (int x = 0; x < 4; ++x) c[n][x] = c2[n][x] = 0.f;
#pragma unroll
        for (int j = 0; j < DP / 32; ++j) {
            const uint32_t row = at + k_lane + (k_xor ^ (64 * j));
            const uint4 k0 = lds128(row), k1 = lds128(row + 8 * S::kRowBytes);
#pragma unroll
            for (int n = 0; n < NT; ++n) {
                mma<T>(c[n], k0.x, k1.x, k0.y, k1.y, q[n][j].x, q[n][j].y);
                mma<T>(c2[n], k0.z, k1.z, k0.w, k1.w, q[n][j].z, q[n][j].w);
            }
        }
#pragma unroll
        for (int n = 0; n < NT; ++n)
#pragma unroll
            for (int x = 0; x < 4; ++x) c[n][x] += c2[n][x];
        const uint32_t bits = flags >> (2 * (S::kStages - 1));
        // binary exponents over `top`, the maximum so far less the headroom; masked: -infinity
        bool low = true;
#pragma unroll
        for (int n = 0; n < NT; ++n)
#pragma unroll
            for (int x = 0; x < 4; ++x) {
                const float y = fmaf(c[n][x], a.scale_log2, -top[n][x & 1]);
                c2[n][x] = bits >> (x >> 1) & 1 ? y : -INFINITY;
                low = low && c2[n][x] <= kMostWeight;
            }
        if (!__all_sync(~0u, low)) {
            // A new maximum.  One up to 2^3 above the old is let be, so after a row's first
            // tiles this is rarely entered.
#pragma unroll
            for (int n = 0; n < NT; ++n) {
                float keep[2];
#pragma unroll
                for (int x = 0; x < 2; ++x) {  // heads 2t and 2t + 1
                    const float s0 = bits & 1 ? c[n][x] * a.scale_log2 : -INFINITY;
                    const float s1 = bits & 2 ? c[n][x + 2] * a.scale_log2 : -INFINITY;
                    float m = fmaxf(s0, s1);
                    m = fmaxf(m, __shfl_xor_sync(~0u, m, 4));
                    m = fmaxf(m, __shfl_xor_sync(~0u, m, 8));
                    m = fmaxf(m, __shfl_xor_sync(~0u, m, 16));
                    m = fmaxf(m - kHeadroom, top[n][x]);
                    const float base = m == -INFINITY ? 0.f : m;  // nothing yet: every weight is 0
                    keep[x] = exp2_fast(top[n][x] - base);
                    top[n][x] = m;
                    sum[n][x] *= keep[x];
                    c2[n][x] = s0 - base;
                    c2[n][x + 2] = s1 - base;
                }
#pragma unroll
                for (int i = 0; i < DP / 16; ++i) {
                    o[n][i][0] *= keep[0], o[n][i][1] *= keep[1];
                    o[n][i][2] *= keep[0], o[n][i][3] *= keep[1];
                }
            }
        }
        uint32_t p_hi[NT][2], p_lo[NT][2];
#pragma unroll
        for (int n = 0; n < NT; ++n) {
#pragma unroll
            for (int x = 0; x < 4; ++x) c[n][x] = exp2_fast(c2[n][x]);
            sum[n][0] += c[n][0] + c[n][2];
            sum[n][1] += c[n][1] + c[n][3];
#pragma unroll
            for (int r = 0; r < 2; ++r) {  // positions g and g + 8
                const float p0 = c[n][2 * r], p1 = c[n][2 * r + 1];
                const uint32_t hi16 = pack2_down<T>(p0, p1);
                const float2 back = unpack2<T>(hi16);
                p_hi[n][r] = transpose8x8(hi16);
                // a weight below kLeast has no first part and stays what it is
                p_lo[n][r] = transpose8x8(pack2<T>(fmaxf(p0 - back.x, fminf(p0, kLeast)),
                                                   fmaxf(p1 - back.y, fminf(p1, kLeast))));
            }
        }
#pragma unroll
        for (int i = 0; i < DP / 16; ++i) {
            uint32_t v[4];
            load_transposed(v, at + v_lane + (v_xor ^ (32 * i)));
#pragma unroll
            for (int n = 0; n < NT; ++n) {
                mma<T>(o[n][i], v[0], v[1], v[2], v[3], p_hi[n][0], p_hi[n][1]);
                mma<T>(o[n][i], v[0], v[1], v[2], v[3], p_lo[n][0], p_lo[n][1]);
            }
        }
        __syncwarp();  // the tile is read: its slot may be filled again

        const bool ends = here.tile == here.steps - 1;
        if (ends || step == count - 1) {
            // The warps' parts meet in the slots of the tiles just read.
            // (dims 16i + g and 16i + g + 8 of heads 2t, 2t + 1; swizzled by the head)
            float* mine_out = reinterpret_cast<float*>(ring + stage * S::kStageBytes +
                                                       warp * S::kTileBytes);
#pragma unroll
            for (int n = 0; n < NT; ++n) {
#pragma unroll
                for (int x = 0; x < 2; ++x) {
                    float l = sum[n][x];
                    l += __shfl_xor_sync(~0u, l, 4);
                    l += __shfl_xor_sync(~0u, l, 8);
                    l += __shfl_xor_sync(~0u, l, 16);
                    const int h = 8 * n + 2 * t + x;
                    if (g == 0) warp_ml[warp][h] = make_float2(top[n][x], l);
#pragma unroll
                    for (int i = 0; i < DP / 16; ++i) {
                        mine_out[h * DP + ((16 * i + g) ^ 8 * t)] = o[n][i][x];
                        mine_out[h * DP + ((16 * i + g + 8) ^ 8 * t)] = o[n][i][x + 2];
                    }
                }
            }
            __syncthreads();
            const bool whole = ends && first_tile == 0 && a.cluster <= 1;
            const int heads = a.heads_of(here.item), side = first_tile == 0 ? 1 : 0;
            const float* parts = reinterpret_cast<const float*>(ring + stage * S::kStageBytes);
            for (int i = tid; i < heads * (DP / 4); i += kAttendThreads) {
                const int h = i / (DP / 4), x = i % (DP / 4) * 4;
                float m = -INFINITY, l = 0.f;
#pragma unroll
                for (int w = 0; w < kAttendWarps; ++w) m = fmaxf(m, warp_ml[w][h].x);
                const float base = m == -INFINITY ? 0.f : m;
                float4 v = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
                for (int w = 0; w < kAttendWarps; ++w) {
                    const float e = exp2_fast(warp_ml[w][h].x - base);
                    const float4 u = *reinterpret_cast<const float4*>(
                        parts + w * (S::kTileBytes / 4) + h * DP + (x ^ 8 * (h / 2 % 4)));
                    l += e * warp_ml[w][h].y;
                    v.x += e * u.x, v.y += e * u.y, v.z += e * u.z, v.w += e * u.w;
                }
                if (whole) {
                    write_out<T>(a, here.row, a.first_head(here.item) + h, x, v, m, l);
                } else if (a.cluster) {
                    // at the ring's start, which only this thread still reads there, if any does
                    *reinterpret_cast<float4*>(reinterpret_cast<float*>(ring) + h * DP +
                                               (x ^ 8 * (h / 2 % 4))) = v;
                    if (x == 0) block_ml[h] = make_float2(m, l);
                } else {
                    const int64_t slot = ((int64_t)blockIdx.x * 2 + side) * kHeads + h;
                    *reinterpret_cast<float4*>(a.partial + slot * DP + x) = v;
                    if (x == 0) a.partial_ml[slot] = make_float2(m, l);
                }
            }
            if (side == 1 && tid == 0 && (!ends || a.by_item) && !a.cluster) {
                int64_t owner = blockIdx.x;
                if (!ends) {
                    const int64_t last = lo + step + (here.steps - 1 - here.tile);  // the item's last step
                    owner = last * blocks / total;
                    while (cut(total, owner + 1, blocks) <= last) ++owner;
                    while (cut(total, owner, blocks) > last) --owner;
                }
                a.joints[a.by_item ? here.row * a.items + here.item : blockIdx.x] = {
                    here.row, here.item, (int)(owner - blockIdx.x), (int)blockIdx.x};
            }
            __syncthreads();
            fresh = true;
        }
        advance(a, here);
        issue(stage);
        stage = stage + 1 == S::kStages ? 0 : stage + 1;
    }
    copy_wait<0>();

    if (a.cluster > 1) {
        // Each block adds up a part of the item's output, read from all of them.
        cluster_sync_all();
        const int heads = a.heads_of(begin.item);
        const uint32_t my_ml = smem_u32(block_ml), my_out = smem_u32(ring);
        for (int i = (int)cluster_cta_rank() * kAttendThreads + tid; i < heads * (DP / 4);
             i += a.cluster * kAttendThreads) {
            const int h = i / (DP / 4), x = i % (DP / 4) * 4;
            const uint32_t offset = (h * DP + (x ^ 8 * (h / 2 % 4))) * 4;
            float2 ml[kMaxCluster];
            float4 u[kMaxCluster];
            float m = -INFINITY, l = 0.f;
#pragma unroll
            for (int r = 0; r < kMaxCluster; ++r) {
                ml[r] = make_float2(-INFINITY, 0.f);
                u[r] = make_float4(0.f, 0.f, 0.f, 0.f);
                if (r < a.cluster) {
                    ml[r] = ld_cluster_f2(map_to_cta(my_ml + h * 8, r));
                    u[r] = ld_cluster_f4(map_to_cta(my_out + offset, r));
                    m = fmaxf(m, ml[r].x);
                }
            }
            const float base = m == -INFINITY ? 0.f : m;
            float4 v = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
            for (int r = 0; r < kMaxCluster; ++r) {
                if (ml[r].y < 0.f) continue;  // no step; a maximum of -infinity may have a sum of NaN
                const float e = exp2_fast(ml[r].x - base);
                l += e * ml[r].y;
                v.x += e * u[r].x, v.y += e * u[r].y, v.z += e * u[r].z, v.w += e * u[r].w;
            }
            write_out<T>(a, begin.row, a.first_head(begin.item) + h, x, v, m, l);
        }
        cluster_sync_all();  // the others have read this block's part
    }
}

// Adds up items' parts, where an item has few: block (x, y) has joint x, a thread
// four dimensions of a head, eight parts on their way at a time.
constexpr int kFewThreads = 128;
template <typename T, int DP>
__global__ void __launch_bounds__(kFewThreads) join_few_kernel(AttendArgs a, int heads_padded) {
    constexpr int kAhead = 8;
    grid_dependency_wait();
    grid_launch_dependents();
    const Joint joint = a.joints[blockIdx.x];
    if (joint.count == 0) return;
    const int heads = a.heads_of(joint.item);
    for (int t = blockIdx.y * kFewThreads + threadIdx.x; t < heads * (DP / 4);
         t += gridDim.y * kFewThreads) {
        const int h = t / (DP / 4), x = t % (DP / 4) * 4;
        float m = -INFINITY, l = 0.f;
        float4 v = make_float4(0.f, 0.f, 0.f, 0.f);
        for (int first = 0; first <= joint.count; first += kAhead) {
            float2 ml[kAhead];
            float4 u[kAhead];
            float higher = m;
#pragma unroll
            for (int k = 0; k < kAhead; ++k) {
                const int i = first + k;
                ml[k] = make_float2(-INFINITY, 0.f);
                u[k] = make_float4(0.f, 0.f, 0.f, 0.f);
                if (i <= joint.count) {
                    // the first block's second slot, then the first slots of the blocks after it
                    const int64_t slot = ((int64_t)(joint.first + i) * 2 + (i == 0)) * heads_padded + h;
                    ml[k] = a.partial_ml[slot];
                    u[k] = *reinterpret_cast<const float4*>(a.partial + slot * DP + x);
                }
            }
#pragma unroll
            for (int k = 0; k < kAhead; ++k) higher = fmaxf(higher, ml[k].x);
            const float base = higher == -INFINITY ? 0.f : higher, keep = exp2_fast(m - base);
            m = higher;
            l *= keep;
            v.x *= keep, v.y *= keep, v.z *= keep, v.w *= keep;
#pragma unroll
            for (int k = 0; k < kAhead; ++k) {
                const float e = exp2_fast(ml[k].x - base);
                l += e * ml[k].y;
                v.x += e * u[k].x, v.y += e * u[k].y, v.z += e * u[k].z, v.w += e * u[k].w;
            }
        }
        write_out<T>(a, joint.row, a.first_head(joint.item) + h, x, v, m, l);
    }
}

// The same where an item has many parts: block (x, y) has head y of joint x.  A
// row split over the whole GPU has some sixty parts a head: a thread group's first
// eight are read before the weights are settled, and no part waits for another.  (One part at a time with running
// maxima in between took 13 us of a 131071-position call.)
constexpr int kJoinThreads = 256;
constexpr int kMaxParts = 1024;  // blocks of attend_kernel: num_sms * kBlocksPerSm at most
template <typename T, int DP>
__global__ void __launch_bounds__(kJoinThreads) join_many_kernel(AttendArgs a, int heads_padded) {
    constexpr int kGroups = kJoinThreads / (DP / 4);
    __shared__ float weight[kMaxParts + 1];
    __shared__ float4 part[kGroups][DP / 4];
    __shared__ float2 warp_ml[kJoinThreads / 32];
    const int h = blockIdx.y, x = threadIdx.x % (DP / 4), group = threadIdx.x / (DP / 4);
    grid_dependency_wait();
    grid_launch_dependents();
    const Joint joint = a.joints[blockIdx.x];
    if (joint.count == 0 || h >= a.heads_of(joint.item)) return;
    // part i: the first block's second slot, then the first slots of the blocks after it
    const auto slot = [&](int i) {
        return ((int64_t)(joint.first + i) * 2 + (i == 0)) * heads_padded + h;
    };
    constexpr int kAhead = 8;
    float4 u[kAhead];
#pragma unroll
    for (int k = 0; k < kAhead; ++k) {
        const int i = group + k * kGroups;
        if (i <= joint.count)
            u[k] = *reinterpret_cast<const float4*>(a.partial + slot(i) * DP + 4 * x);
    }
    float m = -INFINITY, l = 0.f;
    for (int i = threadIdx.x; i <= joint.count; i += kJoinThreads) {
        const float2 ml = a.partial_ml[slot(i)];
        const float higher = fmaxf(m, ml.x), base = higher == -INFINITY ? 0.f : higher;
        l = l * exp2_fast(m - base) + ml.y * exp2_fast(ml.x - base);
        m = higher;
        weight[i] = ml.x;
    }
    const float own = m;
#pragma unroll
    for (int d = 16; d > 0; d /= 2) m = fmaxf(m, __shfl_xor_sync(~0u, m, d));
    l *= exp2_fast(own - (m == -INFINITY ? 0.f : m));
#pragma unroll
    for (int d = 16; d > 0; d /= 2) l += __shfl_xor_sync(~0u, l, d);
    if (threadIdx.x % 32 == 0) warp_ml[threadIdx.x / 32] = make_float2(m, l);
    __syncthreads();
    m = -INFINITY, l = 0.f;
#pragma unroll
    for (int w = 0; w < kJoinThreads / 32; ++w) m = fmaxf(m, warp_ml[w].x);
    const float base = m == -INFINITY ? 0.f : m;
#pragma unroll
    for (int w = 0; w < kJoinThreads / 32; ++w) l += warp_ml[w].y * exp2_fast(warp_ml[w].x - base);
    float4 v = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
    for (int k = 0; k < kAhead; ++k) {
        const int i = group + k * kGroups;
        if (i > joint.count) break;
        const float e = exp2_fast(weight[i] - base);
        v.x += e * u[k].x, v.y += e * u[k].y, v.z += e * u[k].z, v.w += e * u[k].w;
    }
#pragma unroll 4
    for (int i = group + kAhead * kGroups; i <= joint.count; i += kGroups) {
        const float e = exp2_fast(weight[i] - base);
        const float4 w = *reinterpret_cast<const float4*>(a.partial + slot(i) * DP + 4 * x);
        v.x += e * w.x, v.y += e * w.y, v.z += e * w.z, v.w += e * w.w;
    }
    part[group][x] = v;
    __syncthreads();
    if (group) return;
#pragma unroll
    for (int i = 1; i < kGroups; ++i) {
        const float4 u = part[i][x];
        v.x += u.x, v.y += u.y, v.z += u.z, v.w += u.w;
    }
    write_out<T>(a, joint.row, a.first_head(joint.item) + h, 4 * x, v, m, l);
}

// Query heads of an item and their tiles of 8: one tile up to 8 heads to a
// key-value head, else two; more than 16 are dealt out evenly over blocks.
struct HeadPlan {
    int tiles, blocks, heads;
};
HeadPlan plan_heads(int64_t group) {
    HeadPlan p;
    p.tiles = group <= 8 ? 1 : 2;  // 16 heads by items of 8 read all keys twice: 1.8 times as long
    p.blocks = (int)((group + 8 * p.tiles - 1) / (8 * p.tiles));
    p.heads = (int)((group + p.blocks - 1) / p.blocks);
    return p;
}

int padded_dim(int64_t dim) { return dim <= 64 ? 64 : dim <= 128 ? 128 : 256; }

int attend_blocks(int64_t dim, int tiles, const DeviceCtx& ctx) {
    const int per_sm[3][2] = {{AttendShape<64, 1>::kBlocksPerSm, AttendShape<64, 2>::kBlocksPerSm},
                              {AttendShape<128, 1>::kBlocksPerSm, AttendShape<128, 2>::kBlocksPerSm},
                              {AttendShape<256, 1>::kBlocksPerSm, AttendShape<256, 2>::kBlocksPerSm}};
    return std::min(kMaxParts, ctx.num_sms * per_sm[dim <= 64 ? 0 : dim <= 128 ? 1 : 2][tiles - 1]);
}

// Clusters of 1 .. 8 blocks of an attention kernel that the device has room for at once.
struct Room {
    cudaError_t error = cudaSuccess;
    int clusters[kMaxCluster + 1] = {};
};

template <typename T, int DP, int NT, bool kTilePage>
const Room& room_of(int device) {
    static std::once_flag once[64];
    static Room room[64];
    const auto kernel = attend_kernel<T, DP, NT, kTilePage>;
    std::call_once(once[device], [&]() {
        Room& r = room[device];
        r.error = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                       AttendShape<DP, NT>::kSmem);
        cudaLaunchAttribute attr;
        attr.id = cudaLaunchAttributeClusterDimension;
        cudaLaunchConfig_t cfg = {};
        cfg.blockDim = dim3(kAttendThreads);
        cfg.dynamicSmemBytes = AttendShape<DP, NT>::kSmem;
        cfg.attrs = &attr;
        cfg.numAttrs = 1;
        for (int n = 1; n <= kMaxCluster && r.error == cudaSuccess; ++n) {
            cfg.gridDim = dim3((unsigned)n);
            attr.val.clusterDim.x = (unsigned)n;
            attr.val.clusterDim.y = attr.val.clusterDim.z = 1;
            r.error = cudaOccupancyMaxActiveClusters(&r.clusters[n], kernel, &cfg);
        }
    });
    return room[device];
}

// The room of the kernel that a cache's geometry takes.
template <typename T, int DP, int NT>
const Room& room_of(bool tile_page, int device) {
    return tile_page ? room_of<T, DP, NT, true>(device) : room_of<T, DP, NT, false>(device);
}
template <typename T>
const Room& room_of(int dim, int tiles, bool tile_page, int device) {
    if (dim <= 64)
        return tiles == 1 ? room_of<T, 64, 1>(tile_page, device) : room_of<T, 64, 2>(tile_page, device);
    if (dim <= 128)
        return tiles == 1 ? room_of<T, 128, 1>(tile_page, device) : room_of<T, 128, 2>(tile_page, device);
    return tiles == 1 ? room_of<T, 256, 1>(tile_page, device) : room_of<T, 256, 2>(tile_page, device);
}

// Blocks to an item where tables are short, a cluster that joins its parts in
// shared memory: no second launch and no workspace.  As many as the device has
// room for at once (a cluster stays within a part of the GPU, so 8 fit less
// often than 6: 64 items of 8 steps by clusters of 7 take 10.9 us, by 6 7.1),
// and a step each.  0, and the line is cut instead, where that leaves a block
// too many steps, as a row may be that much longer than the others (such a step
// takes 0.7 us): 32 where the blocks fill half the places or more, else 8.
// Clusters / the line, 8 key-value heads: 56 rows of 2048 73 / 81 us, from short
// ones to 2048 44 / 48, 14 rows to 4096 27.7 / 27.9, 8 rows to 4096 17.7 / 19.3,
// of 512 7.0 / 9.2, one row of 512 4.8 / 6.8, one of 8192 15.9 / 10.9.
// What counts is the room of the tables: the lengths are on the device.  So one row
// of 512 takes the line where its table has room for more than 4096 positions.
int item_cluster(const w4a16_cache_shape& c, int64_t group, const DeviceCtx& ctx, cudaError_t* error) {
    const HeadPlan heads = plan_heads(group);
    const int64_t items = c.batch * c.kv_heads * heads.blocks;
    const int64_t places = attend_blocks(c.head_dim, heads.tiles, ctx);
    const int64_t steps = (c.table_width * c.page_size + kStep - 1) / kStep;
    if (items > places || steps > kMaxCluster * kMostSteps) return 0;
    int device = 0;
    if ((*error = cudaGetDevice(&device)) != cudaSuccess) return 0;
    const bool tile_page = c.page_size % kTile == 0;
    const Room& room = c.type == W4A16_BF16
                           ? room_of<__nv_bfloat16>((int)c.head_dim, heads.tiles, tile_page, device)
                           : room_of<__half>((int)c.head_dim, heads.tiles, tile_page, device);
    if ((*error = room.error) != cudaSuccess) return 0;
    int n = (int)std::min<int64_t>(kMaxCluster, steps);
    while (n > 0 && items > room.clusters[n]) --n;
    return steps <= n * (2 * items * n >= places ? kMostSteps : kFewSteps) ? n : 0;
}

// The workspace: partial outputs, their maxima and sums, the joints.
struct Workspace {
    int64_t partial, ml, joints, bytes;
};
Workspace plan_workspace(int64_t dim, int64_t group, const DeviceCtx& ctx) {
    const int tiles = plan_heads(group).tiles;
    const int64_t blocks = attend_blocks(dim, tiles, ctx), slots = 2 * blocks * 8 * tiles;
    Workspace w;
    w.partial = 0;
    w.ml = slots * padded_dim(dim) * 4;
    w.joints = w.ml + slots * 8;
    w.bytes = w.joints + blocks * (int64_t)sizeof(Joint);
    return w;
}

template <typename T, int DP, int NT, bool kTilePage>
cudaError_t attend(AttendArgs a, cudaStream_t stream, const DeviceCtx& ctx) {
    using S = AttendShape<DP, NT>;
    int device = 0;
    cudaError_t e = cudaGetDevice(&device);
    if (e != cudaSuccess) return e;
    if ((e = room_of<T, DP, NT, kTilePage>(device).error) != cudaSuccess) return e;
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.x = (unsigned)a.cluster;
    attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
    cudaLaunchConfig_t cfg = {};
    const unsigned blocks = (unsigned)attend_blocks(DP, NT, ctx);
    a.by_item = (int64_t)a.c.batch * a.items <= blocks;
    cfg.gridDim = dim3(a.cluster ? (unsigned)(a.c.batch * a.items * a.cluster) : blocks);
    cfg.blockDim = dim3(kAttendThreads);
    cfg.dynamicSmemBytes = S::kSmem;
    cfg.stream = stream;
    cfg.attrs = attr;
    cfg.numAttrs = a.cluster > 1 ? 2 : 1;
    e = cudaLaunchKernelEx(&cfg, attend_kernel<T, DP, NT, kTilePage>, a);
    if (e != cudaSuccess || a.cluster) return e;
    cfg.numAttrs = 1;
    cfg.dynamicSmemBytes = 0;
    const int64_t items = (int64_t)a.c.batch * a.items;
    // Few joints, so several parts an item: 64 items of 7 heads (16 rows to 4093, 4 key-value
    // heads, wide tables) 19.2 us, 20.0 by the other form.  Many joints, mostly of two parts: 512
    // items of 4 heads (64 rows of 1024, 8 key-value heads) 51 us, 53.3 by this form.
    if (items * a.block_heads <= blocks) {
        cfg.gridDim = dim3((unsigned)items, (unsigned)a.block_heads);
        cfg.blockDim = dim3(kJoinThreads);
        return cudaLaunchKernelEx(&cfg, join_many_kernel<T, DP>, a, 8 * NT);
    }
    cfg.gridDim = dim3(a.by_item ? (unsigned)items : blocks,
                       (unsigned)((a.block_heads * (DP / 4) + kFewThreads - 1) / kFewThreads));
    cfg.blockDim = dim3(kFewThreads);
    return cudaLaunchKernelEx(&cfg, join_few_kernel<T, DP>, a, 8 * NT);
}

// Tiles of 16 positions lie within a page where the page size is a multiple of
// 16: one page number a tile then, else one a position.
template <typename T, int DP, int NT>
cudaError_t attend(const AttendArgs& a, cudaStream_t stream, const DeviceCtx& ctx) {
    return a.c.page_size.value % kTile == 0 ? attend<T, DP, NT, true>(a, stream, ctx)
                                      : attend<T, DP, NT, false>(a, stream, ctx);
}

template <typename T, int DP>
cudaError_t attend(const AttendArgs& a, int tiles, cudaStream_t stream, const DeviceCtx& ctx) {
    return tiles == 1 ? attend<T, DP, 1>(a, stream, ctx) : attend<T, DP, 2>(a, stream, ctx);
}

template <typename T>
cudaError_t attend(const AttendArgs& a, int tiles, cudaStream_t stream, const DeviceCtx& ctx) {
    switch (padded_dim(a.c.head_dim)) {
        case 64: return attend<T, 64>(a, tiles, stream, ctx);
        case 128: return attend<T, 128>(a, tiles, stream, ctx);
        default: return attend<T, 256>(a, tiles, stream, ctx);
    }
}

}  // namespace

cudaError_t launch_paged_append(const void* k, const void* v, void* k_pool, void* v_pool,
                                const int32_t* tables, const int32_t* starts,
                                const int32_t* offsets, const w4a16_cache_shape& cache,
                                int64_t tokens, int64_t k_token, int64_t k_head, int64_t v_token,
                                int64_t v_head, cudaStream_t stream, const DeviceCtx& ctx) {
    const int64_t pieces = cache.head_dim / 8;
    // four pieces a thread, up to 16 tokens a block, while that leaves four blocks an SM: 32749
    // tokens of 8 heads of 128 take 42.0 us by 4 tokens a block, 44.6 by 16 and 51 by 2
    const int64_t block = std::max<int64_t>(
        1, std::min({(int64_t)kAppendTokens, tokens / (4 * ctx.num_sms),
                     kAppendThreads * kAppendUnroll / (2 * cache.kv_heads * pieces)}));
    const AppendArgs a{static_cast<const uint16_t*>(k),
                       static_cast<const uint16_t*>(v),
                       static_cast<uint16_t*>(k_pool),
                       static_cast<uint16_t*>(v_pool),
                       tables, starts, offsets, tokens, k_token, k_head, v_token, v_head,
                       cache_of(cache), (int)block, Divisor(cache.kv_heads * pieces),
                       Divisor(pieces)};
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)((tokens + block - 1) / block));
    cfg.blockDim = dim3(kAppendThreads);
    cfg.stream = stream;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, append_kernel, a);
}

int64_t paged_attention_workspace(const w4a16_cache_shape& cache, int64_t q_heads,
                                  const DeviceCtx& ctx) {
    const int64_t group = q_heads / cache.kv_heads;
    cudaError_t e = cudaSuccess;
    const int cluster = item_cluster(cache, group, ctx, &e);
    if (e != cudaSuccess) return -1;
    return cluster ? 0 : plan_workspace(cache.head_dim, group, ctx).bytes;
}

cudaError_t launch_paged_attention(const void* q, const void* k_pool, const void* v_pool,
                                   const int32_t* tables, const int32_t* lengths, void* out,
                                   float* lse, void* workspace, const w4a16_cache_shape& cache,
                                   const w4a16_query_shape& query, cudaStream_t stream,
                                   const DeviceCtx& ctx) {
    AttendArgs a;
    a.q = static_cast<const uint16_t*>(q);
    a.k_pool = static_cast<const uint16_t*>(k_pool);
    a.v_pool = static_cast<const uint16_t*>(v_pool);
    a.tables = tables;
    a.lengths = lengths;
    a.out = static_cast<uint16_t*>(out);
    a.lse = lse;
    a.q_heads = (int)query.q_heads;
    a.group = (int)(query.q_heads / cache.kv_heads);
    const HeadPlan heads = plan_heads(a.group);
    a.head_blocks = heads.blocks;
    a.block_heads = heads.heads;
    a.items = (int)cache.kv_heads * heads.blocks;
    cudaError_t e = cudaSuccess;
    a.cluster = item_cluster(cache, a.group, ctx, &e);
    if (e != cudaSuccess) return e;
    const Workspace w = plan_workspace(cache.head_dim, a.group, ctx);
    char* base = static_cast<char*>(workspace);
    a.partial = reinterpret_cast<float*>(base + w.partial);
    a.partial_ml = reinterpret_cast<float2*>(base + w.ml);
    a.joints = reinterpret_cast<Joint*>(base + w.joints);
    a.q_row = query.q_row_stride;
    a.q_head = query.q_head_stride;
    a.out_row = query.out_row_stride;
    a.out_head = query.out_head_stride;
    a.scale_log2 = (float)(query.scale * 1.4426950408889634);
    a.c = cache_of(cache);
    return cache.type == W4A16_BF16 ? attend<__nv_bfloat16>(a, heads.tiles, stream, ctx)
                                    : attend<__half>(a, heads.tiles, stream, ctx);
}

}  // namespace w4a16
