// logprobs.cu -- the scores of given tokens under rows of logits: log
// probability, entropy and the likeliest alternatives.
//
// With m the row's maximum, s = sum e^(x - m) and t = sum e^(x - m) (x - m):
//   logprob = x[token] - m - ln s,   entropy = ln s - t / s,
// so one pass over the logits gives everything but the alternatives.  Each
// thread keeps (m, s, t) of its own 16-byte pieces and takes a new maximum
// once a batch of them; parts with other maxima are added up as
//   s = sum s_i e^(m_i - m),   t = sum e^(m_i - m) (t_i + s_i (m_i - m)).
//
// The sums run in pairs (f32x2) with y = (x - m) log2(e), t in units of ln 2.
//
// The alternatives come from the maxima that the pass leaves anyway.  The
// k-th largest of the maxima of 64 groups of threads is at most the k-th
// largest logit, and few logits are above it (k = 20: 24 of 128256 independent
// ones); only the batches of pieces whose maximum reaches it are read again,
// and the few logits found are ranked by counting.  Where they are not few
// (masks leave fewer than k logits, so the cut is the mask's value), those
// above the cut are kept and the lowest indices at it added in order.
//
// A row is a block's, or, for few rows, a cluster's, whose first block joins
// the others' sums and alternatives through shared memory: no workspace, one
// launch.  Bound by HBM for many rows, short of it by what a block does after
// its pass: on one GB300 (6790 GB/s copied) 2047 rows of 128256 take 88 us in
// fp16 (5985 GB/s), 1023 in fp32 80 us (6560 GB/s).  One row takes 8.2 us, all
// of it latency: a launch, a pass, six barriers of a block with alternatives
// (two without), two of the cluster and three in its first block.
#include <cuda_bf16.h>

#include <stddef.h>

#include <type_traits>

#include "common.cuh"
#include "kernels.h"

namespace w4a16 {
namespace {

constexpr int kSmThreads = 1024;            // of blocks side by side on an SM
constexpr int kGroups = 64;                 // of threads, for the first cut of the alternatives
constexpr int kBatch = 8;                   // 16-byte pieces a thread has in flight
constexpr int kCandidates = 1024;
constexpr int kAheadBytes = 32768;          // of a row to come, asked into L2
constexpr int kMaxCluster = 4;
constexpr int kKept = 16;                   // batches of a thread whose maxima are kept
constexpr float kLog2e = 1.4426950408889634f;
constexpr float kLn2 = 0.6931471805599453f;

struct ScoreArgs {
    const void *logits, *tokens;
    float *logprob, *entropy, *top_logprobs;
    int32_t* top_ids;
    int64_t rows, vocabulary, row_stride;
    int wide, top;
};

__device__ __forceinline__ float to_float(__half v) { return __half2float(v); }
__device__ __forceinline__ float to_float(__nv_bfloat16 v) { return __bfloat162float(v); }
__device__ __forceinline__ float to_float(float v) { return v; }

__device__ __forceinline__ __half from_float(float v, __half) { return __float2half_rn(v); }
__device__ __forceinline__ __nv_bfloat16 from_float(float v, __nv_bfloat16) {
    return __float2bfloat16_rn(v);
}
__device__ __forceinline__ float from_float(float v, float) { return v; }

// Two FP32 values, for the paired instructions.
__device__ __forceinline__ uint64_t pair(float lo, float hi) {
    uint64_t r;
    asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(lo), "f"(hi));
    return r;
}
__device__ __forceinline__ void unpair(uint64_t v, float& lo, float& hi) {
    asm("mov.b64 {%0, %1}, %2;" : "=f"(lo), "=f"(hi) : "l"(v));
}
__device__ __forceinline__ uint64_t fma2(uint64_t a, uint64_t b, uint64_t c) {
    uint64_t r;
    asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
    return r;
}
__device__ __forceinline__ uint64_t add2(uint64_t a, uint64_t b) {
    uint64_t r;
    asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
    return r;
}
__device__ __forceinline__ uint64_t mul2(uint64_t a, uint64_t b) {
    uint64_t r;
    asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
    return r;
}
__device__ __forceinline__ float exp2_fast(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

// The larger, NaN if one is: of a word's values at once.
__device__ __forceinline__ uint32_t max_words(uint32_t a, uint32_t b, __half) {
    uint32_t r;
    asm("max.NaN.f16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
    return r;
}
__device__ __forceinline__ uint32_t max_words(uint32_t a, uint32_t b, __nv_bfloat16) {
    uint32_t r;
    asm("max.NaN.bf16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
    return r;
}
__device__ __forceinline__ float max_nan(float a, float b) {
    float r;
    asm("max.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(a), "f"(b));
    return r;
}
__device__ __forceinline__ uint32_t max_words(uint32_t a, uint32_t b, float) {
    return __float_as_uint(max_nan(__uint_as_float(a), __uint_as_float(b)));
}

// A 32-bit word's values.
__device__ __forceinline__ void word_values(uint32_t w, float (&v)[2], __half) {
    const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&w));
    v[0] = f.x, v[1] = f.y;
}
__device__ __forceinline__ void word_values(uint32_t w, float (&v)[2], __nv_bfloat16) {
    v[0] = __uint_as_float(w << 16), v[1] = __uint_as_float(w & 0xFFFF0000u);
}
__device__ __forceinline__ void word_values(uint32_t w, float (&v)[1], float) {
    v[0] = __uint_as_float(w);
}

template <typename T>
__device__ __forceinline__ uint32_t lowest_word() {  // -infinity
    return sizeof(T) == 4 ? 0xFF800000u : std::is_same<T, __half>::value ? 0xFC00FC00u : 0xFF80FF80u;
}

__device__ __forceinline__ float exp_fast(float x) { return exp2_fast(x * kLog2e); }

// Whole numbers in the order of the values, NaN above all, -0 equal to 0; none is 0.
__device__ __forceinline__ uint32_t key_of(float x) {
    const int bits = __float_as_int(x + 0.f);
    const uint32_t key = (uint32_t)(bits ^ ((bits >> 31) & 0x7FFFFFFF)) ^ 0x80000000u;
    return x != x ? 0xFFFFFFFFu : key;
}
__device__ __forceinline__ float value_of(uint32_t key) {
    const int bits = (int)(key ^ 0x80000000u);
    return __int_as_float(bits ^ ((bits >> 31) & 0x7FFFFFFF));  // all ones gives a NaN
}
// The same with the index: of equal values the lower index first.
__device__ __forceinline__ uint64_t rank_of(uint32_t key, int index) {
    return (uint64_t)key << 32 | (uint32_t)~index;
}

// Part of a row's sums.  worst: the key of a NaN or +infinity seen, else 0.
struct Sums {
    float m, s, t;
    uint32_t worst;
};

__device__ __forceinline__ Sums add(const Sums& a, const Sums& b) {
    Sums r;
    r.m = fmaxf(a.m, b.m);
    r.worst = max(a.worst, b.worst);
    const float da = a.m == -INFINITY ? 0.f : a.m - r.m, db = b.m == -INFINITY ? 0.f : b.m - r.m;
    const float ea = exp_fast(da), eb = exp_fast(db);  // s = t = 0 where m is -infinity
    // far below, e is 0 and e * d is not to be 0 * infinity
    r.s = a.s * ea + b.s * eb;
    r.t = (ea > 0.f ? ea * (a.t + a.s * da) : 0.f) + (eb > 0.f ? eb * (b.t + b.s * db) : 0.f);
    return r;
}

template <typename T, int kThreads>
struct ScoreShared {
    T batch_top[kKept][kThreads];       // the largest logit of a thread's batch
    int batches;
    uint32_t batch[kThreads];      // those that reach the cut: thread | batch << 16
    Sums part[kThreads / 32];
    Sums sums;                      // of the block
    uint32_t group_key[kGroups];
    uint32_t cut, higher;
    int listed, found;
    uint16_t list[kThreads];   // threads whose maximum reaches the cut
    uint64_t best[W4A16_MAX_TOP];   // the block's alternatives, in order
    int bests;
    uint64_t candidate[kCandidates];
    uint64_t warp_best[kThreads / 32];
    int equal[kThreads / 32];
};

__device__ __forceinline__ uint64_t ld_cluster_u64(uint32_t addr) {
    uint64_t v;
    asm volatile("ld.shared::cluster.u64 %0, [%1];" : "=l"(v) : "r"(addr) : "memory");
    return v;
}
__device__ __forceinline__ uint32_t ld_cluster_u32(uint32_t addr) {
    uint32_t v;
    asm volatile("ld.shared::cluster.u32 %0, [%1];" : "=r"(v) : "r"(addr) : "memory");
    return v;
}

template <typename T, int kThreads>
__global__ void __launch_bounds__(kThreads, kSmThreads / kThreads)
    score_kernel(ScoreArgs a, int blocks, int64_t ahead) {
    constexpr int kPer = 16 / sizeof(T), kWord = 4 / sizeof(T);
    constexpr int kWarps = kThreads / 32, kGroupThreads = kThreads / kGroups;
    using Shared = ScoreShared<T, kThreads>;
    __shared__ Shared sh;
    const int tid = threadIdx.x, warp = tid / 32, lane = tid % 32;
    const int64_t row = blockIdx.x / blocks;
    const int rank = (int)(blockIdx.x % blocks);
    const T* x = static_cast<const T*>(a.logits) + row * a.row_stride;
    const int n = (int)a.vocabulary;
    grid_dependency_wait();
    grid_launch_dependents();

    // The row: values before the first 16-byte boundary, pieces, values after the last.
    const int head = min(n, (int)((16 - (reinterpret_cast<uintptr_t>(x) & 15)) % 16 / sizeof(T)));
    const int pieces = (n - head) / kPer;
    const int loose = rank == 0 ? n - pieces * kPer : 0;  // < 2 * kPer, one a thread
    const int loose_at = tid < head ? tid : tid + pieces * kPer;
    const int first = (int)((int64_t)pieces * rank / blocks);
    const int count = (int)((int64_t)pieces * (rank + 1) / blocks) - first;
    const uint4* piece = reinterpret_cast<const uint4*>(x + head) + first;

    int64_t token = -1;
    float token_logit = 0.f;
    if (rank == 0 && tid == 0) {
        token = a.wide ? static_cast<const int64_t*>(a.tokens)[row]
                       : static_cast<const int32_t*>(a.tokens)[row];
        if (token >= 0 && token < n) token_logit = to_float(x[token]);
    }
    if (tid == 0) sh.listed = sh.found = sh.batches = 0;

    Sums own{-INFINITY, 0.f, 0.f, 0u};
    const bool some = tid < loose || tid < count;
    float s = 0.f, t = 0.f;
    const auto take = [&](const uint4 (&v)[kBatch], int batch) {
        uint32_t top = v[0].x;
#pragma unroll
        for (int b = 0; b < kBatch; ++b) {
            top = max_words(top, v[b].x, T());
            top = max_words(top, v[b].y, T());
            top = max_words(top, v[b].z, T());
            top = max_words(top, v[b].w, T());
        }
        float f[kWord];
        word_values(top, f, T());
        const float higher = kWord == 2 ? max_nan(f[0], f[kWord - 1]) : f[0];
        if (batch < kKept) sh.batch_top[batch][tid] = from_float(higher, T());
        if (!(higher <= own.m)) {  // a new maximum, or no number
            if (higher < INFINITY) {
                const float d = own.m == -INFINITY ? 0.f : fmaxf((own.m - higher) * kLog2e, -200.f);
                const float e = exp2_fast(d);  // e' = e 2^d, y' = y + d
                t = e * (t + s * d);
                s *= e;
                own.m = higher;
            } else {
                own.worst = max(own.worst, key_of(higher));
            }
        }
        uint64_t s2 = 0, t2 = 0;  // pairs of +0
        const float base = own.m == -INFINITY ? 0.f : -own.m;
        const uint64_t l2 = pair(kLog2e, kLog2e), m2 = pair(base, base);
#pragma unroll
        for (int b = 0; b < kBatch; ++b) {
            const uint32_t w[4] = {v[b].x, v[b].y, v[b].z, v[b].w};
#pragma unroll
            for (int i = 0; i < 4; i += 2 / kWord) {
                float g[2];
                if (kWord == 2) {
                    word_values(w[i], f, T());
                    g[0] = f[0], g[1] = f[kWord - 1];
                } else {
                    g[0] = __uint_as_float(w[i]), g[1] = __uint_as_float(w[i + 2 / kWord - 1]);
                }
                float y0, y1;
                unpair(mul2(add2(pair(g[0], g[1]), m2), l2), y0, y1);
                // at least -150, where e is 0: so a masked logit adds 0 and not 0 * infinity
                y0 = fmaxf(y0, -150.f), y1 = fmaxf(y1, -150.f);
                const uint64_t e2 = pair(exp2_fast(y0), exp2_fast(y1));
                s2 = add2(s2, e2);
                t2 = fma2(e2, pair(y0, y1), t2);
            }
        }
        float lo, hi;
        unpair(s2, lo, hi);
        s += lo + hi;
        unpair(t2, lo, hi);
        t += lo + hi;
    };
    int j = tid, batch = 0;
    for (; j + (kBatch - 1) * kThreads < count; j += kBatch * kThreads, ++batch) {
        uint4 v[kBatch];
#pragma unroll
        for (int b = 0; b < kBatch; ++b) v[b] = __ldg(piece + j + b * kThreads);
        take(v, batch);
    }
    if (j < count) {
        uint4 v[kBatch];
#pragma unroll
        for (int b = 0; b < kBatch; ++b) {
            const int at = j + b * kThreads;
            v[b] = make_uint4(lowest_word<T>(), lowest_word<T>(), lowest_word<T>(), lowest_word<T>());
            if (at < count) v[b] = __ldg(piece + at);
        }
        take(v, batch);
    }
    own.s = s;
    own.t = t * kLn2;
    // What follows reads little: meanwhile, the start of the row that a block of the next wave has
    // comes to L2 (2047 rows 89.1 us without, 86.7 with 32 KB, 87.6 with 64, 92.9 with 128).
    if (tid == 0 && row + ahead < a.rows && count >= 2 * kAheadBytes / 16) {
        const uintptr_t next = reinterpret_cast<uintptr_t>(x + ahead * a.row_stride);
        bulk_prefetch_l2(reinterpret_cast<const void*>((next + 15) & ~(uintptr_t)15), kAheadBytes);
    }
    if (tid < loose) {
        const float v = to_float(x[loose_at]);
        if (!(v < INFINITY))
            own.worst = max(own.worst, key_of(v));
        else if (v > -INFINITY)
            own = add(own, Sums{v, 1.f, 0.f, 0u});
    }
    const uint32_t own_key = some ? max(key_of(own.m), own.worst) : 0u;

    // The block's sums, and the maxima of its groups of two or four threads.
    uint32_t key = max(own_key, __shfl_xor_sync(~0u, own_key, 1));
    if (kGroupThreads == 4) key = max(key, __shfl_xor_sync(~0u, key, 2));
    if (lane % kGroupThreads == 0) sh.group_key[tid / kGroupThreads] = key;
#pragma unroll
    for (int d = 16; d > 0; d /= 2) {
        const Sums o{__shfl_xor_sync(~0u, own.m, d), __shfl_xor_sync(~0u, own.s, d),
                     __shfl_xor_sync(~0u, own.t, d), __shfl_xor_sync(~0u, own.worst, d)};
        own = add(own, o);
    }
    if (lane == 0) sh.part[warp] = own;
    __syncthreads();
    if (warp == kWarps - 1) {
        Sums p = lane < kWarps ? sh.part[lane] : Sums{-INFINITY, 0.f, 0.f, 0u};
#pragma unroll
        for (int d = kWarps / 2; d > 0; d /= 2) {
            const Sums o{__shfl_xor_sync(~0u, p.m, d), __shfl_xor_sync(~0u, p.s, d),
                         __shfl_xor_sync(~0u, p.t, d), __shfl_xor_sync(~0u, p.worst, d)};
            p = add(p, o);
        }
        if (lane == 0) sh.sums = p;
    }
    if (a.top > 0) {
        // the cut: the group maximum with top - 1 others before it
        if (tid < kGroups) {
            const uint32_t mine = sh.group_key[tid];
            int before = 0;
#pragma unroll 16
            for (int i = 0; i < kGroups; ++i)
                before += sh.group_key[i] > mine || (sh.group_key[i] == mine && i < tid);
            if (before == a.top - 1) sh.cut = mine;
            if (before == kGroups * 3 / 4) sh.higher = mine;  // as many groups are above it
        }
        __syncthreads();
        const uint32_t cut = sh.cut;
        // the batches with a maximum of at least `least`, then their logits
        const auto collect = [&](uint32_t least) {
            const auto offer = [&](float v, int index) {
                const uint32_t k = key_of(v);
                if (k < least) return;
                const int at = atomicAdd(&sh.found, 1);
                if (at < kCandidates) sh.candidate[at] = rank_of(k, index);
            };
            const auto offer_piece = [&](int at) {
                if (at >= count) return;
                const uint4 v = __ldg(piece + at);
                const uint32_t w[4] = {v.x, v.y, v.z, v.w};
                const int index = head + (first + at) * kPer;
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    float f[kWord];
                    word_values(w[i], f, T());
#pragma unroll
                    for (int k = 0; k < kWord; ++k) offer(f[k], index + i * kWord + k);
                }
            };
            constexpr int kTurn = kBatch * kThreads;
            if (own_key != 0u && own_key >= least)
                sh.list[atomicAdd(&sh.listed, 1)] = (uint16_t)tid;
            __syncthreads();
            const int listed = sh.listed, turns = (count + kTurn - 1) / kTurn;
            for (int u = tid; u < listed * turns; u += kThreads) {
                const int who = sh.list[u % listed], turn = u / listed;
                if (turn < kKept) {
                    if (turn * kTurn + who >= count ||
                        key_of(to_float(sh.batch_top[turn][who])) < least)
                        continue;
                    const int at = atomicAdd(&sh.batches, 1);
                    if (at < kThreads) {
                        sh.batch[at] = (uint32_t)who | (uint32_t)turn << 16;
                        continue;
                    }
                }
                // not kept, or too many for the list: here and now
                for (int b = 0; b < kBatch; ++b) offer_piece(turn * kTurn + b * kThreads + who);
            }
            if (tid < loose) offer(to_float(x[loose_at]), loose_at);
            __syncthreads();
            const int batches = min(sh.batches, kThreads);
            for (int u = tid; u < batches * kBatch; u += kThreads) {
                const uint32_t what = sh.batch[u / kBatch];
                offer_piece((int)(what >> 16) * kTurn + u % kBatch * kThreads +
                            (int)(what & 0xFFFFu));
            }
            __syncthreads();
            return sh.found;
        };
        // logit e of the block's part, in ascending order
        const int before_pieces = rank == 0 ? head : 0, in_pieces = count * kPer;
        const int part = loose + in_pieces;
        const auto index_of = [&](int e) {
            return e < before_pieces               ? e
                   : e < before_pieces + in_pieces ? head + first * kPer + e - before_pieces
                                                   : head + pieces * kPer + e - before_pieces - in_pieces;
        };
        // where most groups reach the cut, they do so at its value: a mask's
        bool above = sh.higher >= cut;
        int found = above ? 0 : collect(cut);
        if (found > kCandidates) {
            above = true;
            __syncthreads();
            if (tid == 0) sh.listed = sh.found = sh.batches = 0;
            __syncthreads();
        }
        if (above) {
            found = cut == 0xFFFFFFFFu ? 0 : collect(cut + 1);
            for (int base = 0; found < a.top && base < part; base += kThreads) {
                const int index = index_of(min(base + tid, part - 1));
                const bool equal = base + tid < part && key_of(to_float(x[index])) == cut;
                const uint32_t mask = __ballot_sync(~0u, equal);
                if (lane == 0) sh.equal[warp] = __popc(mask);
                __syncthreads();
                int at = found + __popc(mask & ((1u << lane) - 1));
                for (int w = 0; w < kWarps; ++w) {
                    if (w < warp) at += sh.equal[w];
                    found += sh.equal[w];
                }
                if (equal && at < a.top) sh.candidate[at] = rank_of(cut, index);
                __syncthreads();
                found = min(found, a.top);
            }
        }
        if (found <= kCandidates) {
            for (int i = tid; i < found; i += kThreads) {
                const uint64_t mine = sh.candidate[i];
                int before = 0;
                for (int j = 0; j < found; ++j) before += sh.candidate[j] > mine;
                if (before < a.top) sh.best[before] = mine;
            }
            if (tid == 0) sh.bests = min(found, a.top);
        } else {
            // A thousand logits above the cut, in the pieces of few threads: a sweep of the
            // block's part for each alternative.
            uint64_t last = ~0ull;
            for (int k = 0; k < a.top; ++k) {
                uint64_t next = 0;
                for (int e = tid; e < part; e += kThreads) {
                    const int index = index_of(e);
                    const uint64_t r = rank_of(key_of(to_float(x[index])), index);
                    if (r < last) next = max(next, r);
                }
#pragma unroll
                for (int d = 16; d > 0; d /= 2) next = max(next, __shfl_xor_sync(~0u, next, d));
                if (lane == 0) sh.warp_best[warp] = next;
                __syncthreads();
                for (int w = 0; w < kWarps; ++w) next = max(next, sh.warp_best[w]);
                last = next;
                if (tid == 0) sh.best[k] = next;
                __syncthreads();
            }
            if (tid == 0) sh.bests = a.top;
        }
    }
    __syncthreads();

    // The first block joins the cluster's parts.
    Sums all = sh.sums;
    if (blocks > 1) {
        cluster_sync_all();
        if (rank == 0) {
            const uint32_t here = smem_u32(&sh);
            for (int r = 1; r < blocks; ++r) {
                const uint32_t there = map_to_cta(here, r) + (uint32_t)offsetof(Shared, sums);
                const Sums o{__uint_as_float(ld_cluster_u32(there)),
                             __uint_as_float(ld_cluster_u32(there + 4)),
                             __uint_as_float(ld_cluster_u32(there + 8)), ld_cluster_u32(there + 12)};
                all = add(all, o);
            }
            if (a.top > 0) {
                // thread (r, k) has alternative k of block r
                const int r = tid / W4A16_MAX_TOP, k = tid % W4A16_MAX_TOP;
                uint64_t mine = 0;
                if (r < blocks) {
                    const uint32_t there = map_to_cta(here, r);
                    const int held = (int)ld_cluster_u32(there + (uint32_t)offsetof(Shared, bests));
                    if (k < held)
                        mine = ld_cluster_u64(there + (uint32_t)offsetof(Shared, best) + 8 * k);
                }
                sh.candidate[tid] = mine;  // 0: none, below all
                __syncthreads();
                int before = 0;
                for (int j = 0; j < blocks * W4A16_MAX_TOP; ++j) before += sh.candidate[j] > mine;
                __syncthreads();
                if (mine != 0 && before < a.top) sh.best[before] = mine;
                __syncthreads();
            }
        }
        cluster_sync_all();  // the other blocks' shared memory has been read
        if (rank != 0) return;
    }
    const bool nothing = all.worst == 0 && all.m == -INFINITY;
    const float ln = logf(all.s);
    const auto score = [&](float v) {
        return all.worst ? NAN : nothing ? -INFINITY : v - all.m - ln;
    };
    if (tid == 0) {
        a.logprob[row] = token >= 0 && token < n ? score(token_logit) : NAN;
        a.entropy[row] = all.worst ? NAN : nothing ? 0.f : ln - all.t / all.s;
    }
    if (tid < a.top) {
        const uint64_t best = sh.best[tid];
        a.top_ids[row * a.top + tid] = (int)~(uint32_t)best;
        a.top_logprobs[row * a.top + tid] = score(value_of((uint32_t)(best >> 32)));
    }
}

// Blocks to a row: one where the rows are more than half the SMs, else up to
// four, as many as keep a piece of the row for every thread.  What a block does
// after its pass costs more than a shorter pass saves: one row of 128256 takes
// 9.0, 8.1 and 8.8 us by 2, 4 and 8 blocks, 64 rows 9.5 us by 2 and 16 us by 8,
// 153 rows 15.5 us by 1 and 22 us by 4.
int score_blocks(int64_t rows, int64_t vocabulary, int size, const DeviceCtx& ctx) {
    int blocks = 1;
    while (blocks < kMaxCluster && rows * blocks * 2 <= ctx.num_sms &&
           vocabulary * size / 16 >= (int64_t)blocks * 2 * 256)
        blocks *= 2;
    return blocks;
}

template <typename T, int kThreads>
cudaError_t score(const ScoreArgs& a, int blocks, cudaStream_t stream, const DeviceCtx& ctx) {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)(a.rows * blocks));
    cfg.blockDim = dim3(kThreads);
    cfg.stream = stream;
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.x = (unsigned)blocks;
    attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = blocks > 1 ? 2 : 1;
    // rows to a wave of blocks; clusters have one wave
    const int64_t ahead = blocks > 1 ? a.rows : (int64_t)(kSmThreads / kThreads) * ctx.num_sms;
    return cudaLaunchKernelEx(&cfg, score_kernel<T, kThreads>, a, blocks, ahead);
}

// Rows of less than two batches of pieces for 256 threads go by blocks of 128: what a block does
// after its pass then runs beside seven others' (2047 rows of 32000 fp16 logits 30.5 us, by 256
// threads 35.8; of 128256, top 20, 95 and 91).
template <typename T>
cudaError_t score(const ScoreArgs& a, cudaStream_t stream, const DeviceCtx& ctx) {
    const int blocks = score_blocks(a.rows, a.vocabulary, sizeof(T), ctx);
    return blocks == 1 && a.vocabulary * (int64_t)sizeof(T) / 16 < 2 * kBatch * 256
               ? score<T, 128>(a, blocks, stream, ctx)
               : score<T, 256>(a, blocks, stream, ctx);
}

}  // namespace

cudaError_t launch_token_logprobs(const void* logits, const void* tokens, float* logprob,
                                  float* entropy, int32_t* top_ids, float* top_logprobs,
                                  int64_t rows, int64_t vocabulary, int64_t row_stride, int type,
                                  int wide, int top, cudaStream_t stream, const DeviceCtx& ctx) {
    const ScoreArgs a{logits, tokens, logprob, entropy, top_logprobs, top_ids,
                      rows, vocabulary, row_stride, wide, top};
    return type == W4A16_F16    ? score<__half>(a, stream, ctx)
           : type == W4A16_BF16 ? score<__nv_bfloat16>(a, stream, ctx)
                                : score<float>(a, stream, ctx);
}

}  // namespace w4a16
