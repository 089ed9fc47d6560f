// paged.cuh -- the geometry of a paged cache, for the kernels that read and write it.
#pragma once

#include "common.cuh"
#include "kernels.h"

namespace w4a16 {
namespace {

// x / divisor for 0 <= x < 2^31: with l = ceil(log2 divisor) and
// m = floor(2^(31 + l) / divisor) + 1, m * divisor exceeds 2^(31 + l) by at most
// divisor <= 2^l, so x * m / 2^(31 + l) is off by less than 1 / divisor.
struct Divisor {
    int value;
    uint32_t mul, shift;

    Divisor() : Divisor(1) {}
    explicit Divisor(int64_t divisor) : value((int)divisor) {
        uint32_t l = 0;
        while (((int64_t)1 << l) < divisor) ++l;
        shift = 31 + l;
        mul = (uint32_t)(((uint64_t)1 << shift) / (uint64_t)divisor + 1);
    }
    __device__ __forceinline__ int quotient(int x) const {
        return (int)(((uint64_t)(uint32_t)x * mul) >> shift);
    }
    __device__ __forceinline__ int remainder(int x) const { return x - quotient(x) * value; }
};

// A cache's geometry; strides in elements (2 bytes).
struct Cache {
    int64_t pages, page_stride, slot_stride, head_stride, table_stride;
    int kv_heads, head_dim, batch, width;
    Divisor page_size;
};

inline Cache cache_of(const w4a16_cache_shape& c) {
    return {c.pages,         c.page_stride,    c.slot_stride,    c.head_stride,
            c.table_stride,  (int)c.kv_heads,  (int)c.head_dim,  (int)c.batch,
            (int)c.table_width, Divisor(c.page_size)};
}

// The row with offsets[b] <= token < offsets[b + 1], -1 if none (the token itself without
// offsets); by a whole warp.
inline __device__ int row_of(const int32_t* offsets, int batch, int64_t token) {
    if (!offsets) return (int)token;
    const int lane = threadIdx.x % 32;
    int lo = 0, step = batch;  // rows before lo end at or before the token
    do {
        step = (step + 31) / 32;
        const int last = lo + (lane + 1) * step - 1;  // of the lane's part
        const bool before = last < batch && offsets[last + 1] <= token;
        lo += __popc(__ballot_sync(~0u, before)) * step;
    } while (step > 1 && lo < batch);
    return lo < batch && offsets[lo] <= token && token < offsets[lo + 1] ? lo : -1;
}

}  // namespace
}  // namespace w4a16
