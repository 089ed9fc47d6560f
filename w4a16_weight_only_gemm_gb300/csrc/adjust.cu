// adjust.cu -- penalties, biases and masks on logits before a token is sampled.
//
// With c the times a token was generated, and r, f, p the row's repetition,
// frequency and presence penalties:
//   y = x, or where the prompt or the generation has the token x / r (x > 0), x r (else)
//   y = y - f c - p [c > 0] + bias,   -infinity where the mask's bit is 0.
//
// A copy of the logits under the mask, bound by HBM, and then the few tokens that a
// row has said or has biases for, one by one.  Those a block finds without a table
// in memory: it takes a slice of one row's vocabulary, holds a word of counts for
// each token of it in shared memory, and reads the whole history, which the row's
// other blocks find in L2 (4096 tokens are 16 KB, as many bytes as a slice of 8192
// logits of 16 bits).
// Counts are integers and a token's logit is its own, so the order of the atomics
// changes nothing.  A piece of 16 bytes that the mask has none of is not read, and in
// place only what changes is touched.
//
// Measured: 512 rows of 128256 bf16 logits under masks, histories of up to 8191 (4103 on
// average), 80 us: 43 for the copy, the rest for the histories (41 would be all bytes once at
// 6790 GB/s); instructions bound it, issue slots are 77 % full.  64 rows of fp32, histories of
// up to 4093, 18 us (9.8).  One row 4.0 us, which is latency.  The same with
//   slices of 16384, 512 threads       79, 21.4, 3.9 us: half as many reads of the histories, but
//                                      too few blocks for 64 rows
//   what is found by a bit a token, and from a list of the block's  90, 18, 4.0
//   logits staged in shared memory while the history is read        90, 23, 4.2
// Other calls, the same inputs again each time: the 512 rows in place 75 us, with int64 tokens 98
// (a load of 8 bytes each); 64 rows of bf16 with histories of up to 16383 tokens 23, 30000 33, 16
// rows of 100000 41, one 24.
#include <cuda_bf16.h>

#include <algorithm>
#include <mutex>
#include <type_traits>

#include "common.cuh"
#include "kernels.h"

namespace w4a16 {
namespace {

constexpr int kThreads = 256;
constexpr int kBlocksPerSm = 8;
constexpr int kAhead = 1;            // pieces of a thread on their way
constexpr int kWordBytes = 16384;    // of a slice's words at most
constexpr int kTogether = 3;         // said tokens of a thread on their way
// Places of the list for what a thread finds itself: with 6, one block in several ran out (99 us for
// 512 rows with 4, 89 with 6, 83 with 10); with 16 the list takes from L1 what it gives (90, and 86
// now that 10 take 78).  A block that runs out sweeps its words: where all of a row's history lies in one
// slice, 512 rows take 72 us for 78, 64 rows of fp32 16.1 for 13.4 (the same inputs again each time).
constexpr int kOwn = 10;
constexpr int kListed = kOwn * kThreads;
constexpr int kEach = 4, kSwept = kEach * kThreads;  // words of a thread and of a block, swept at a time
static_assert(kSwept <= kListed && 1024 % kSwept == 0, "a list of them, and slices are multiples of 1024");
constexpr int kMostBiases = W4A16_MAX_BIASES;

// A token's word: whether a bias is listed for it, whether the prompt has it, and in the other bits
// how often the generation has it.  Of 16 bits where histories are short enough, else of 32.
template <typename W>
struct Word {
    static constexpr int kBits = 8 * sizeof(W);
    static constexpr uint32_t kBiased = 1u << (kBits - 1), kPrompt = 1u << (kBits - 2),
                              kCount = kPrompt - 1;
    static constexpr int kSlice = kWordBytes / sizeof(W);
};

struct AdjustArgs {
    w4a16_adjust_tensors t;
    w4a16_adjust_shape s;
    int slice, slices;
    bool in_place;
    float repetition, presence, frequency;  // (converted by the host: FP64 units are few)
};

__device__ __forceinline__ float to_float(__half v) { return __half2float(v); }
__device__ __forceinline__ float to_float(__nv_bfloat16 v) { return __bfloat162float(v); }
__device__ __forceinline__ float to_float(float v) { return v; }
template <typename T>
__device__ __forceinline__ T from_float(float v) {
    return (T)v;
}

template <typename W>
struct Penalties {
    float repetition, presence, frequency;

    __device__ __forceinline__ float apply(float x, uint32_t word) const {
        if (word & ~Word<W>::kBiased) x = x > 0.f ? x / repetition : x * repetition;
        const uint32_t count = word & Word<W>::kCount;
        if (count) x = x - frequency * (float)count - presence;
        return x;
    }
};

template <typename T, int V>
struct alignas(sizeof(T) * V) Piece {
    T x[V];
};

// The values whose bit is 0 become -infinity; two of 16 bits at a time.
template <typename T, int V>
__device__ __forceinline__ void blank(Piece<T, V>& v, uint32_t bits) {
    if constexpr (sizeof(T) == 2 && V >= 2) {
        constexpr uint32_t kMasked = std::is_same<T, __half>::value ? 0xFC00FC00u : 0xFF80FF80u;
        uint32_t* two = reinterpret_cast<uint32_t*>(&v);
#pragma unroll
        for (int k = 0; k < V / 2; ++k, bits >>= 2) {
            const uint32_t keep = ((bits | bits << 15) & 0x00010001u) * 0xFFFFu;
            two[k] = (two[k] & keep) | (kMasked & ~keep);
        }
    } else {
#pragma unroll
        for (int k = 0; k < V; ++k)
            if (!(bits >> k & 1)) v.x[k] = from_float<T>(-INFINITY);
    }
}

// Whether the row's mask allows token j (all of them without a mask).
__device__ __forceinline__ bool allowed(const uint32_t* mask, int64_t j) {
    return !mask || (mask[j >> 5] >> (j & 31) & 1);
}

// V: logits of a piece, 16 bytes where the rows of logits and out lie alike to that boundary, else 1.
template <typename T, int V, typename W>
__global__ void __launch_bounds__(kThreads, kBlocksPerSm) adjust_kernel(AdjustArgs a) {
    // words of the slice's tokens, the list, the biases' tokens
    extern __shared__ __align__(16) uint32_t space[];
    W* words = reinterpret_cast<W*>(space);
    __shared__ int listed;  // tokens on the list
    __shared__ int twice;   // whether some token has two biases
    uint16_t* list = reinterpret_cast<uint16_t*>(words + a.slice);
    int32_t* bias_ids = reinterpret_cast<int32_t*>(list + kListed);
    const int64_t row = blockIdx.x / a.slices;
    const int vocabulary = (int)a.s.vocabulary;
    grid_dependency_wait();
    grid_launch_dependents();
    const T* x = static_cast<const T*>(a.t.logits) + row * a.s.logits_stride;
    T* out = static_cast<T*>(a.t.out) + row * a.s.out_stride;
    const uint32_t* mask = a.t.mask ? a.t.mask + row * a.s.mask_stride : nullptr;
    // The slice begins where a piece does: `shift` values before the row's first one are passed over.
    const int shift = (int)(reinterpret_cast<uintptr_t>(x) / sizeof(T) % V);
    const int begin = (int)(blockIdx.x % a.slices) * a.slice - shift;
    const int from = max(begin, 0), to = (int)min((int64_t)begin + a.slice, (int64_t)vocabulary);
    if (from >= to) return;
    const uint32_t span = (uint32_t)(to - from), skip = (uint32_t)(from - begin);

    const int length = a.t.tokens ? (int)(a.t.lengths ? min(max((int64_t)a.t.lengths[row], (int64_t)0), a.s.width)
                                                      : a.s.width)
                                  : 0;
    const int prompt = a.t.prompts ? a.t.prompts[row] : 0;
    const int biases = a.t.bias_ids ? (int)a.s.biases : 0;
    for (int i = threadIdx.x; i < biases; i += kThreads)
        bias_ids[i] = a.t.bias_ids[row * a.s.bias_stride + i];
    for (int i = threadIdx.x; i < a.slice * (int)sizeof(W) / 16; i += kThreads)
        reinterpret_cast<uint4*>(space)[i] = make_uint4(0, 0, 0, 0);
    if (threadIdx.x == 0) listed = twice = 0;
    __syncthreads();

    // The history: first what the prompt has, then what the generation has.  Each thread also writes
    // down what it finds in the slice, which is little.  (Predicated, and nothing waits for it: with
    // branches, or with the old word returned to see who is first, this took longer than all the rest.
    // A number before the row's first token counts in a word that stands for none.)
    const uint32_t word0 = smem_u32(words), own0 = smem_u32(list) + 2 * threadIdx.x;
    const uint32_t own_end = own0 + kOwn * (2 * kThreads), size = (uint32_t)(to - begin);
    uint32_t next = own0;  // where the thread's next find goes
    const auto note = [&](auto said, int32_t token) {
        constexpr bool kSaid = decltype(said)::value;  // by the prompt
        const uint32_t at = (uint32_t)token - (uint32_t)begin;
        const uint32_t address = sizeof(W) == 2 ? word0 + (2 * at & ~3u) : word0 + 4 * at;
        const uint32_t unit = kSaid ? Word<W>::kPrompt : 1u;
        const uint32_t value = sizeof(W) == 2 && (at & 1) ? unit << 16 : unit;
#define NOTE(OPERATION)                                          \
    asm volatile(                                                \
        "{\n\t.reg .pred p, q;\n\t"                              \
        "setp.lt.u32 p, %1, %2;\n\t"                             \
        "@p red.shared." OPERATION " [%3], %4;\n\t"              \
        "setp.lt.and.u32 q, %0, %5, p;\n\t"                      \
        "@q st.shared.u16 [%0], %1;\n\t"                         \
        "@p add.u32 %0, %0, %6;\n\t}"                            \
        : "+r"(next)                                             \
        : "r"(at), "r"(size), "r"(address), "r"(value), "r"(own_end), "n"(2 * kThreads) \
        : "memory")
        if constexpr (kSaid) NOTE("or.b32"); else NOTE("add.u32");
#undef NOTE
    };
    // tokens first .. last - 1 of the row
    const auto read = [&](auto said, int first, int last) {
        if (a.s.wide) {
            const int64_t* tokens = static_cast<const int64_t*>(a.t.tokens) + row * a.s.token_stride;
#pragma unroll 2
            for (int i = first + threadIdx.x; i < last; i += kThreads) {
                const int64_t token = tokens[i];
                note(said, token >= 0 && token < vocabulary ? (int32_t)token : INT32_MIN);
            }
            return;
        }
        const int32_t* tokens = static_cast<const int32_t*>(a.t.tokens) + row * a.s.token_stride;
        // fours that begin at a 16-byte boundary, and single ones before and behind them
        const int shift = (int)(reinterpret_cast<uintptr_t>(tokens) / 4 % 4);
        const int begin4 = min((first + shift + 3) / 4 * 4 - shift, last);
        const int end4 = max((last + shift) / 4 * 4 - shift, begin4);
#pragma unroll 2
        for (int i = begin4 + threadIdx.x * 4; i < end4; i += kThreads * 4) {
            const int4 four = *reinterpret_cast<const int4*>(tokens + i);
            note(said, four.x);
            note(said, four.y);
            note(said, four.z);
            note(said, four.w);
        }
        const int singles = begin4 - first + last - end4;
        if (threadIdx.x < singles) {
            const int i = first + threadIdx.x;
            note(said, tokens[i < begin4 ? i : i - begin4 + end4]);
        }
    };
    if (length) {
        read(std::true_type(), 0, min(max(prompt, 0), length));
        read(std::false_type(), min(max(prompt, 0), length), length);
    }
    // Tokens that a bias is listed for are marked: they are their biases' business.
    for (int i = threadIdx.x; i < biases; i += kThreads) {
        const uint32_t at = (uint32_t)bias_ids[i] - (uint32_t)from;
        if (at >= span) continue;
        const uint32_t by = sizeof(W) == 2 ? 16 * ((at + skip) & 1) : 0;
        const uint32_t old = atomicOr(space + (at + skip) * sizeof(W) / 4, Word<W>::kBiased << by);
        if (old & Word<W>::kBiased << by) twice = 1;
    }

    // The copy, under the mask.
    constexpr uint32_t kAll = (1u << V) - 1;
    const T masked = from_float<T>(-INFINITY);
    for (int first = 0; first < a.slice; first += kAhead * kThreads * V) {
        uint32_t bits[kAhead];  // the mask's for each piece; kAll + 1: no whole piece
        Piece<T, V> v[kAhead];
#pragma unroll
        for (int n = 0; n < kAhead; ++n) {
            const int i = first + (n * kThreads + threadIdx.x) * V, j = begin + i;
            bits[n] = kAll + 1;
            if (i >= a.slice || j < 0 || j + V > to) continue;
            bits[n] = kAll;
            if (!mask) continue;
            // the V bits from token j on, which may lie in two words
            const int word = j >> 5, last = (j + V - 1) >> 5;
            const uint32_t low = mask[word], high = last > word ? mask[last] : 0;
            bits[n] = __funnelshift_r(low, high, j & 31) & kAll;
        }
#pragma unroll
        for (int n = 0; n < kAhead; ++n) {
            const int i = first + (n * kThreads + threadIdx.x) * V;
            if (bits[n] && bits[n] <= kAll && !(a.in_place && bits[n] == kAll))
                v[n] = *reinterpret_cast<const Piece<T, V>*>(x + begin + i);
        }
#pragma unroll
        for (int n = 0; n < kAhead; ++n) {
            const int i = first + (n * kThreads + threadIdx.x) * V, j = begin + i;
            if (bits[n] <= kAll) {
                if (bits[n] != kAll) {
                    blank<T, V>(v[n], bits[n]);
                } else if (a.in_place) {
                    continue;
                }
                *reinterpret_cast<Piece<T, V>*>(out + j) = v[n];
            } else if (i < a.slice && j + V > 0 && j < to) {  // the row's ends
                for (int k = 0; k < V; ++k)
                    if (j + k >= 0 && j + k < to && !(a.in_place && allowed(mask, j + k)))
                        out[j + k] = allowed(mask, j + k) ? x[j + k] : masked;
            }
        }
    }
    const Penalties<W> p = {a.t.repetition ? a.t.repetition[row] : a.repetition,
                            a.t.presence ? a.t.presence[row] : a.presence,
                            a.t.frequency ? a.t.frequency[row] : a.frequency};
    const int found = (int)((next - own0) / (2 * kThreads));
    const bool own = !__syncthreads_or(found > kOwn);

    // Biased tokens.  One with several biases is its first listing's, with the biases added in the
    // order of the list.
    const float* value = a.t.biases + row * a.s.bias_stride;
    for (int i = threadIdx.x; i < biases; i += kThreads) {
        const int id = bias_ids[i];
        if ((uint32_t)id - (uint32_t)from >= span || !allowed(mask, id)) continue;
        float y = p.apply(to_float(x[id]), words[id - begin]) + value[i];
        bool later = false;
        for (int j = 0; twice && j < biases; ++j)
            if (bias_ids[j] == id && j != i) {
                later = later || j < i;
                y += value[j];
            }
        // (in place a later listing's thread may read what the first has written, and is dropped)
        if (!later) out[id] = from_float<T>(y);
    }
    // Said tokens: each thread's own, where all had places for what they found.  One that several
    // threads found is written by each of them, alike; in place it is the first's to mark its word.
    if (own) {
#pragma unroll 1
        for (int first = 0; first < found; first += kTogether) {
            int at[kTogether];
            T was[kTogether];
            uint32_t bits[kTogether];
#pragma unroll
            for (int n = 0; n < kTogether; ++n) {
                at[n] = -1;
                if (first + n >= found) continue;
                const int there = list[(first + n) * kThreads + threadIdx.x], id = begin + there;
                const uint32_t mark = Word<W>::kBiased << (sizeof(W) == 2 ? 16 * (there & 1) : 0);
                if (id < 0 || words[there] >= Word<W>::kBiased ||
                    (a.in_place && atomicOr(space + there * sizeof(W) / 4, mark) & mark)) continue;
                at[n] = there;
                was[n] = x[id];
                bits[n] = mask ? mask[id >> 5] : ~0u;
            }
#pragma unroll
            for (int n = 0; n < kTogether; ++n) {
                const int id = begin + at[n];
                if (at[n] >= 0 && bits[n] >> (id & 31) & 1)
                    out[id] = from_float<T>(p.apply(to_float(was[n]), words[at[n]]));
            }
        }
        return;
    }
    // Else those of kSwept words at a time are listed, and then taken one by one, so that all threads
    // have their share.
#pragma unroll 1
    for (int first = 0; first < a.slice; first += kSwept) {
        __syncthreads();
        if (threadIdx.x == 0) listed = 0;
        __syncthreads();
        const int i = first + threadIdx.x * kEach;
        uint32_t set = 0;
#pragma unroll
        for (int k = 0; k < kEach; ++k)
            if (words[i + k] != 0 && words[i + k] < Word<W>::kBiased) set |= 1u << k;
        int at = set ? atomicAdd(&listed, __popc(set)) : 0;
        for (; set; set &= set - 1) list[at++] = (uint16_t)(i + __ffs(set) - 1);
        __syncthreads();
        for (int n = threadIdx.x; n < listed; n += kThreads) {
            const int id = begin + list[n];
            if (id >= 0 && allowed(mask, id)) out[id] = from_float<T>(p.apply(to_float(x[id]), words[list[n]]));
        }
    }
}

template <typename T, int V, typename W>
cudaError_t launch(AdjustArgs a, cudaStream_t stream, const DeviceCtx& ctx) {
    static std::once_flag once[64];
    static cudaError_t set[64];
    int device = 0;
    cudaError_t e = cudaGetDevice(&device);
    if (e != cudaSuccess) return e;
    std::call_once(once[device], [&]() {
        set[device] =
            cudaFuncSetAttribute(adjust_kernel<T, V, W>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                 kWordBytes + 2 * kListed + 4 * kMostBiases);
    });
    if (set[device] != cudaSuccess) return set[device];
    // as large a slice as there are words for, less where that leaves fewer than four blocks an SM
    const int64_t padded = a.s.vocabulary + V - 1;  // a row may begin inside a piece
    int64_t slice = std::min<int64_t>(Word<W>::kSlice, padded * a.s.rows / (4 * ctx.num_sms));
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
    cfg.dynamicSmemBytes = slice * sizeof(W) + 2 * kListed + (a.t.bias_ids ? 4 * a.s.biases : 0);
    cfg.stream = stream;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, adjust_kernel<T, V, W>, a);
}

template <typename T, int V>
cudaError_t launch(const AdjustArgs& a, cudaStream_t stream, const DeviceCtx& ctx) {
    return a.s.width <= (int64_t)Word<uint16_t>::kCount ? launch<T, V, uint16_t>(a, stream, ctx)
                                                        : launch<T, V, uint32_t>(a, stream, ctx);
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
    a.repetition = (float)shape.repetition;
    a.presence = (float)shape.presence;
    a.frequency = (float)shape.frequency;
    if (shape.rows == 1) a.s.logits_stride = a.s.out_stride = 0;
    if (shape.type == W4A16_BF16) return launch<__nv_bfloat16>(a, stream, ctx);
    return shape.type == W4A16_F16 ? launch<__half>(a, stream, ctx) : launch<float>(a, stream, ctx);
}

}  // namespace w4a16
