// chunk.cu -- attention of chunks of new tokens over the paged cache, on the
// tcgen05 tensor cores.
//
// A row's new tokens and the query heads that share a key-value head are one list
// of queries, token by token.  As many whole tokens as make 128 queries at most are
// the rows of an MMA tile, and two such tiles (one with heads above 128) an item: so
// no number of heads to a key-value head wastes much.  An item walks the positions that its last query sees in steps
// of 128 (64): S = Q K^T, P = exp(S - max), O += P V, with S and O in tensor memory
// and P written over S as the 16-bit left operand of the second product.
//
// Bound by the tensor cores: 4 dim FLOPs a query and position, where a step's 64 KB
// of keys and values serve 256 queries.  The two tiles take turns, so that the
// tensor cores work on one while the other's softmax runs:
//   warps 0-3, 4-7   softmax of the first and second tile, a thread a query
//   warps 8-11       copy queries, keys and values: by tensor maps, a box for a
//                    page's rows, or row by row (cp.async) with zeros where a
//                    position has no page, and for pages of odd sizes
//   warp 12          one thread issues the MMAs
//   warp 13          takes the next unit of work
//   warps 14, 15     look for values that are not finite where some queries see a
//                    step in part
// An item of one tile has both softmax groups all the same: they take its steps in turn, and
// what the second has is added to the first's at the end.
// The work is cut by a plan kernel, as only the device knows the lengths: items are
// split into parts where that levels the load, and a join kernel adds those up.
// Blocks take units from a counter, the longest first, an item's heads and parts side by
// side: blocks at work at the same time read the same keys and values, through L2.
//
// Weights are rounded to 16 bits once, for the product with V (two 16-bit parts would make it
// two products): off by up to 2^-11 (fp16) or 2^-8 (bf16) of themselves.  The sums that divide it
// are of the weights before that.  So an average of equal values is not always that value: weights
// that are alike all round alike, as those of 1244 positions with scores of 4.94 behind 256 of 0, over
// which equal bf16 values came out up to 0.6 % off, their own rounding in it (fp16 0.05 %).  Summing
// the rounded weights too, to divide by, gave the value itself, and took 187 us for 162 (prompts),
// 160 for 153.5 (a mixed step), 2.84 to 2.95 ms for 2.61 to 2.67 (2048 after 129023) and with heads of
// 64 397 for 317 (2048 after 16384).  It is not done: the error is the bound that each weight's
// rounding has by itself.
//
// Measured (8 key-value heads of 128, 4 query heads to each): one row of 2048 tokens after
// 129023, bf16, 2.56 to 2.87 ms, 1520 to 1700 TFLOP/s, as the power allows; 23 prompts of up to
// 1531 tokens, fp16, 161 us, 970 TFLOP/s, the rest being the ends of units, 2 to 3 us
// each, 15.7 of them a block; 5 tokens after 700, 15 us: the plan 6, the attention and the join.
#include <cuda_bf16.h>

#include <algorithm>
#include <cmath>
#include <mutex>
#include <type_traits>

#include "common.cuh"
#include "kernels.h"
#include "paged.cuh"
#include "tcgen05.cuh"

namespace w4a16 {
namespace {

constexpr float kLn2 = 0.6931471805599453f;
constexpr int kQueryTile = 128;   // queries of an MMA
constexpr int kSoftmaxWarps = 8, kCopyWarps = 4;
constexpr int kMmaWarp = kSoftmaxWarps + kCopyWarps, kUnitWarp = kMmaWarp + 1;
constexpr int kLookWarp = kUnitWarp + 1, kLookWarps = 2;
constexpr int kThreads = 32 * (kLookWarp + kLookWarps);
// Registers of a thread: launched with 128, a softmax thread holds a row of scores.  The four
// warpgroups' shares, 2 x 184 + 2 x 72, are what the block was launched with.
constexpr int kSoftmaxRegisters = 184, kOtherRegisters = 72;
constexpr int kSlots = 4;         // of the ring: keys, values, keys, values
constexpr int kWanted = 4;        // steps of a unit left to copy when the next one is asked for
constexpr int kUnits = 4;         // places for units' notes of values that are not finite
constexpr int kPlanThreads = 1024;
constexpr int kJoinThreads = 128, kJoinAhead = 4;  // parts on their way
constexpr int kPartsPerSm = 4;    // of the workspace

// Sizes by the padded head size: queries of an item, positions of a step.
template <int DP>
struct Shape {
    static constexpr int kTiles = DP <= 128 ? 2 : 1;
    static constexpr int kRows = kTiles * kQueryTile;
    static constexpr int kStep = DP <= 128 ? 128 : 64;
    static constexpr int kTileBytes = kQueryTile * DP * 2;
    static constexpr int kSlotBytes = kStep * DP * 2;
    static constexpr int kOffRing = kTiles * kTileBytes;
    static constexpr int kOffRest = kOffRing + kSlots * kSlotBytes;
    static constexpr int kSmem = 1024 + kOffRest + 16384;
    static constexpr int kOutColumn = 256;                      // of tensor memory
};
constexpr int tiles_of(int64_t dim) { return dim <= 128 ? 2 : 1; }
constexpr int tile_rows_of(int64_t group) {
    return (int)(group <= kQueryTile ? kQueryTile / group * group : kQueryTile);
}
constexpr int step_of(int64_t dim) { return dim <= 128 ? 128 : 64; }

// What the plan leaves, for each key-value head: `whole` units that are items, then `parts` that
// are parts of `joints` items.
struct Plan {
    int whole, parts, joints;
    unsigned next;  // unit to hand out after each block's first
};
// An item: its row, the row's first token and its position (below 0 for a row with more tokens than
// positions), the row's length, and its queries, first and count, in the row's list.
struct Item {
    int row, token0, position0, length, lin0, lins;
};
struct Entry {
    Item item;
    int first, steps;  // steps first .. first + steps - 1
    int part;          // its place among the parts, -1: a whole item
    int unused[3];
};
struct Joint {
    Item item;
    int part, count;
};
struct Slot {
    Item item;
    int steps, unused;
};

struct ChunkArgs {
    const uint16_t *q, *k_pool, *v_pool;
    const int32_t *tables, *lengths, *offsets;
    uint16_t* out;
    float* lse;
    Plan* plan;
    Entry* entries;
    Joint* joints;
    Slot* slots;
    float* partial;      // [part][head][tile][dim / 4][query][4]
    float2* partial_ml;  // [part][head][query of the item]
    int64_t tokens, q_row, q_head, out_row, out_head;
    int64_t slot_count, most_parts;
    int q_heads, sms;
    float scale_log2;    // of the scale's magnitude; its sign:
    int negative;
    unsigned* status;
    uint64_t timeout_ns;
    Cache c;
    Divisor group;
    int tile_rows;       // queries of a tile: as many whole tokens as 128 rows hold
    // Tensor maps serve: of the queries [tokens, heads, dim], of the pools [pages, heads, slots, dim]
    // with boxes of box_rows slots.  0: they do not, and cp.async copies row by row.
    int q_map, box_rows;

    __device__ int64_t offset(int b) const {
        return min(max((int64_t)offsets[b], (int64_t)0), tokens);
    }
    __device__ int64_t length(int b) const {
        return min(max((int64_t)lengths[b], (int64_t)0), (int64_t)c.width * c.page_size.value);
    }
};

// ---------------------------------------------------------------------------
// The plan
//
// Item j of row b takes slot offsets[b] group / rows + b + j (rows of an item): as
// offsets do not descend, no two items share one, and an item's row is found by a
// search.  Some of the items are handed out whole, first and by their length, the longest
// before the others; the rest, and any longer than a block's share, are cut into
// ceil(n / u) parts of nearly equal length.  Tried are 32 lengths u, with none whole or as
// many as make full rounds of the blocks; taken is what makes the estimated time least: a
// unit costs its steps and three more (four where it is a part), and the blocks end within
// half of one of the last units, those that the blocks take last being the shortest; or
// they take rounds of units that are alike.  (Whole ones are counted in slots, from the last;
// slots that no item took count among them, so that a last round may lack a few.  48 rows, 8
// of them with chunks of up to 509 tokens and positions from few to 8191: with items in the
// order of their rows the last block ended 207 us after the start, the mean one after 138.)
// ---------------------------------------------------------------------------
constexpr int kUnitCost = 3, kStaged = 2048, kLengths = 64;

// ceil(steps / unit), or one more for very many (steps are at most 2^25).
__device__ __forceinline__ int parts_of(int steps, int unit, float inverse) {
    int k = (int)((float)steps * inverse);
    k += k * unit < steps;
    return k + (k * unit < steps);
}

// (Loops are not unrolled: it runs once, and its time is mostly that of fetching its code.)
__global__ void __launch_bounds__(kPlanThreads) plan_kernel(ChunkArgs a, Divisor rows, int step_bits) {
    static_assert(kPlanThreads == 1024, "32 warps: one for each length tried");
    __shared__ int64_t sums[32];
    __shared__ int longests[32], ints[32];
    __shared__ int shortests[32];  // (of their own: nothing waits for all to have read them)
    __shared__ int32_t staged[kStaged + 1], staged_steps[kStaged];
    __shared__ float costs[32];
    __shared__ int units[32], keeps[32];
    __shared__ int of_length[kLengths];  // items by their length, then where those go
    const int tid = threadIdx.x, lane = tid % 32, warp = tid / 32;
    grid_dependency_wait();
    grid_launch_dependents();
    const int heads = a.c.kv_heads, batch = a.c.batch, group = a.group.value;
    const int slots = (int)a.slot_count;
    const bool short_batch = batch <= kStaged;
    if (tid < kLengths) of_length[tid] = 0;
    if (short_batch)
#pragma unroll 1
        for (int b = tid; b <= batch; b += kPlanThreads) staged[b] = (int32_t)a.offset(b);
    __syncthreads();
    const auto offset = [&](int b) { return short_batch ? staged[b] : (int)a.offset(b); };
    // (tokens * group is below 2^31)
    const auto key = [&](int b) { return rows.quotient(offset(b) * group) + b; };
    int64_t total = 0;
    int longest = 0, shortest = INT32_MAX, items = 0;
#pragma unroll 1
    for (int s = tid; s < slots; s += kPlanThreads) {
        int lo = 0, hi = batch;  // key(lo) <= s < key(hi)
#pragma unroll 1
        while (hi - lo > 1) {
            const int mid = (lo + hi) / 2;
            if (key(mid) <= s) lo = mid; else hi = mid;
        }
        const int from = offset(lo), count = max(offset(lo + 1) - from, 0), length = (int)a.length(lo);
        const int tile = s - key(lo), lins = count * group;
        Slot slot = {{lo, from, length - count, length, 0, 0}, 0, 0};
        if (tile >= 0 && (int64_t)tile * rows.value < lins) {
            slot.item.lin0 = tile * rows.value;
            slot.item.lins = min(rows.value, lins - slot.item.lin0);
            // positions of the item's last query
            const int last = a.group.quotient(slot.item.lin0 + slot.item.lins - 1);
            const int64_t seen = (int64_t)slot.item.position0 + last + 1;
            slot.steps = seen > 0 ? (int)((seen + (1 << step_bits) - 1) >> step_bits) : 0;
        }
        a.slots[s] = slot;
        if (s < kStaged) staged_steps[s] = slot.steps;
        total += slot.steps;
        items += slot.steps > 0;
        longest = max(longest, slot.steps);
        if (slot.steps) shortest = min(shortest, slot.steps);
    }
#pragma unroll 1
    for (int level = 0; level < 2; ++level) {  // over the warp, then over the warps
#pragma unroll
        for (int d = 16; d > 0; d /= 2) {
            total += __shfl_xor_sync(~0u, total, d);
            items += __shfl_xor_sync(~0u, items, d);
            longest = max(longest, __shfl_xor_sync(~0u, longest, d));
            shortest = min(shortest, __shfl_xor_sync(~0u, shortest, d));
        }
        if (level) break;
        if (lane == 0) {
            sums[warp] = total, ints[warp] = items;
            longests[warp] = longest, shortests[warp] = shortest;
        }
        __syncthreads();
        total = sums[lane], items = ints[lane], longest = longests[lane];
        shortest = shortests[lane];
    }
    total *= heads;
    // Slots are gone through from the last to the first.  Cut are those from the `keep`-th on, and
    // those longer than `cap`.
    const float sms = (float)a.sms, share = (float)total / sms;
    const int cap = (int)fmaxf(share, 1.f);
    const float by_length = (float)(kLengths - 1) / (float)max(longest, 1);
    const auto steps_of_slot = [&](int s) { return s < kStaged ? staged_steps[s] : a.slots[s].steps; };
    int unit = max(longest, 1), keep = slots;
    // (An item that is a sixth of a block's share or less is not worth a cut, nor the search for one.
    // With an eighth, 128 rows of a token after 500 took 66.7 us for 62.5, after 4000 340.8 for 336.5;
    // 30 ragged ones of up to 400 new tokens 211.7 for 216.5.)
    if ((float)longest * 6.f > share && a.most_parts > 0) {
        // The longest of the last units, where none is cut: as many of the shortest items as there
        // are blocks.
        int last = longest;
        const bool many = (float)items * (float)heads > sms;
        if (many) {
#pragma unroll 1
            for (int s = tid; s < slots; s += kPlanThreads) {
                const int n = steps_of_slot(s);
                if (n) atomicAdd(&of_length[(int)((float)n * by_length)], heads);
            }
            __syncthreads();
            static_assert(kLengths == 64, "two lengths a lane");
            const int x = of_length[2 * lane], y = of_length[2 * lane + 1];
            int upto = x + y;
#pragma unroll
            for (int d = 1; d < 32; d *= 2) {
                const int o = __shfl_up_sync(~0u, upto, d);
                if (lane >= d) upto += o;
            }
            const int enough = __ballot_sync(~0u, upto >= a.sms);
            const int at = enough ? 2 * (__ffs(enough) - 1) + 2 : kLengths;
            last = min(longest, (int)((float)at / by_length) + 1);
        }
        // as many as make full rounds of the blocks
        const int full_rounds = (int)(floorf((float)items * (float)heads / sms) * sms / (float)heads);
        // k = 1, 2, 3, ... 8, then some 2^(1/4) apart up to 512
        const int k = warp < 8 ? warp + 1 : (int)(8.f * exp2f((float)(warp - 7) * 0.25f));
        const int u = (longest + k - 1) / k;
        const float inverse = 1.f / (float)u;
        const bool alike = shortest * 5 >= longest * 4;
        float best = INFINITY;
        int best_keep = 0;
#pragma unroll 1
        for (int round = 0; round < (full_rounds ? 2 : 1); ++round) {
            const int kept = round ? full_rounds : 0;
            int whole = 0, parts = 0;
#pragma unroll 1
            for (int r = lane; r < slots; r += 32) {
                const int n = steps_of_slot(slots - 1 - r);
                int p = n > 0;
                if (r >= kept || n > cap) p = parts_of(n, u, inverse);
                parts += p > 1 ? p : 0;
                whole += p == 1;
            }
#pragma unroll
            for (int d = 16; d > 0; d /= 2) {
                whole += __shfl_xor_sync(~0u, whole, d);
                parts += __shfl_xor_sync(~0u, parts, d);
            }
            const float all_parts = (float)parts * (float)heads, all_whole = (float)whole * (float)heads;
            const float work = (float)total + kUnitCost * all_whole + (kUnitCost + 1) * all_parts;
            const float end = (float)(all_parts >= sms ? min(u, last) : last);
            float cost = work / sms + (end + kUnitCost) / 2;
            if (all_parts + all_whole <= sms)  // all at once
                cost = (float)((parts ? u : longest) + kUnitCost + (parts > 0));
            if (alike && whole == 0)
                cost = fminf(cost, ceilf(all_parts / sms) * (float)(u + kUnitCost + 1));
            if (alike && parts == 0)
                cost = ceilf(all_whole / sms) * (float)(longest + kUnitCost);
            if (parts) cost += 1.f;  // the join
            if ((int64_t)parts * heads <= a.most_parts && cost < best) best = cost, best_keep = kept;
        }
        if (lane == 0) costs[warp] = best, units[warp] = u, keeps[warp] = best_keep;
        __syncthreads();
        float least = costs[lane];
        int which = lane;
#pragma unroll
        for (int d = 16; d > 0; d /= 2) {
            const float o = __shfl_xor_sync(~0u, least, d);
            const int w = __shfl_xor_sync(~0u, which, d);
            if (o < least || (o == least && w < which)) least = o, which = w;
        }
        if (least < INFINITY) unit = units[which], keep = keeps[which];
        if (tid < kLengths) of_length[tid] = 0;
    }
    const auto parts_of_slot = [&](int r, int n) {
        return n == 0 ? 0 : r >= keep || n > cap ? (n + unit - 1) / unit : 1;
    };
    // Whole items by their length: how many there are, then where the longest of them begin.
    __syncthreads();
#pragma unroll 1
    for (int r = tid; r < slots; r += kPlanThreads) {
        const int n = steps_of_slot(slots - 1 - r);
        if (parts_of_slot(r, n) == 1) atomicAdd(&of_length[(int)((float)n * by_length)], 1);
    }
    __syncthreads();
    if (warp == 0) {
        const int x = of_length[2 * lane], y = of_length[2 * lane + 1];
        int from = x + y;  // of these lengths and longer ones
#pragma unroll
        for (int d = 1; d < 32; d *= 2) {
            const int o = __shfl_down_sync(~0u, from, d);
            if (lane + d < 32) from += o;
        }
        of_length[2 * lane] = from - x;
        of_length[2 * lane + 1] = from - x - y;
    }
    // The entries: whole ones from the table's start, parts from place `slots` on.
    int base_whole = 0, base_parts = 0, base_joints = 0;
#pragma unroll 1
    for (int first = 0; first < slots; first += kPlanThreads) {
        const int r = first + tid;
        Slot slot = {};
        if (r < slots) slot = a.slots[slots - 1 - r];
        const int n = slot.steps;
        const int k = parts_of_slot(r, n);
        // before this slot: whole ones, joints (16 bits each: 1024 slots at most), parts
        const int own = (k == 1) | (k > 1) << 16, own_parts = k > 1 ? k : 0;
        int upto = own, upto_parts = own_parts;
#pragma unroll
        for (int d = 1; d < 32; d *= 2) {
            const int o = __shfl_up_sync(~0u, upto, d), p = __shfl_up_sync(~0u, upto_parts, d);
            if (lane >= d) upto += o, upto_parts += p;
        }
        __syncthreads();
        if (lane == 31) ints[warp] = upto, longests[warp] = upto_parts;
        __syncthreads();
        int all = ints[lane], before = lane < warp ? all : 0;
        int all_parts = longests[lane], before_parts = lane < warp ? all_parts : 0;
#pragma unroll
        for (int d = 16; d > 0; d /= 2) {
            all += __shfl_xor_sync(~0u, all, d);
            before += __shfl_xor_sync(~0u, before, d);
            all_parts += __shfl_xor_sync(~0u, all_parts, d);
            before_parts += __shfl_xor_sync(~0u, before_parts, d);
        }
        upto += before - own;
        upto_parts += before_parts - own_parts;
        const int part = base_parts + upto_parts;
        if (k > 1) a.joints[base_joints + (upto >> 16)] = {slot.item, part, k};
        // (lengths of parts differ by a step at most)
        const int each = k > 1 ? n / k : n, more = n - each * k;
#pragma unroll 1
        for (int i = 0, at = 0; i < k; ++i) {
            const int steps = each + (i < more);
            a.entries[k > 1 ? slots + part + i : atomicAdd(&of_length[(int)((float)n * by_length)], 1)] = {
                slot.item, at, steps, k > 1 ? part + i : -1, {}};
            at += steps;
        }
        base_whole += all & 0xFFFF;
        base_parts += all_parts;
        base_joints += all >> 16;
    }
    if (tid == 0) *a.plan = {base_whole, base_parts, base_joints, 0};
}

// ---------------------------------------------------------------------------
// Helpers
// ---------------------------------------------------------------------------
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
// An arrival once every copy of this thread so far has landed.
__device__ __forceinline__ void copy_arrive(uint32_t bar) {
    asm volatile("cp.async.mbarrier.arrive.noinc.shared::cta.b64 [%0];" ::"r"(bar) : "memory");
}

// A whole warp's wait, in little code: there are two dozen of them, and code that is run once a
// unit comes from L2 each time.
__device__ __forceinline__ bool warp_wait(uint32_t bar, uint32_t phase, uint64_t timeout_ns,
                                          unsigned* status) {
    if (__all_sync(~0u, mbar_try_wait(bar, phase & 1))) return true;
    const uint64_t since = global_timer_ns();
#pragma unroll 1
    do {
        if (__all_sync(~0u, mbar_try_wait(bar, phase & 1))) return true;
    } while (__any_sync(~0u, global_timer_ns() - since < timeout_ns));
    atomicOr(status, kDevTimeout);
    return false;
}

// Tensor-map loads by one elected lane of a warp that is together (see the MMAs below).
__device__ __forceinline__ void box_load_3d(uint32_t dst, const CUtensorMap* map, int c0, int c1,
                                            int c2, uint32_t bar) {
    asm volatile(
        "{\n\t.reg .pred q;\n\telect.sync _|q, 0xffffffff;\n\t"
        "@q cp.async.bulk.tensor.3d.shared::cluster.global.tile.mbarrier::complete_tx::bytes "
        "[%0], [%1, {%2, %3, %4}], [%5];\n\t}" ::"r"(dst),
        "l"(reinterpret_cast<uint64_t>(map)), "r"(c0), "r"(c1), "r"(c2), "r"(bar)
        : "memory");
}
__device__ __forceinline__ void box_load_4d(uint32_t dst, const CUtensorMap* map, int c0, int c1,
                                            int c2, int c3, uint32_t bar) {
    asm volatile(
        "{\n\t.reg .pred q;\n\telect.sync _|q, 0xffffffff;\n\t"
        "@q cp.async.bulk.tensor.4d.shared::cluster.global.tile.mbarrier::complete_tx::bytes "
        "[%0], [%1, {%2, %3, %4, %5}], [%6];\n\t}" ::"r"(dst),
        "l"(reinterpret_cast<uint64_t>(map)), "r"(c0), "r"(c1), "r"(c2), "r"(c3), "r"(bar)
        : "memory");
}

__device__ __forceinline__ float max3(float x, float y, float z) {
    float m;
    asm("max.f32 %0, %1, %2, %3;" : "=f"(m) : "f"(x), "f"(y), "f"(z));
    return m;
}

__device__ __forceinline__ float exp2_fast(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

// Transposes the 4x4 pieces of four neighbouring lanes: v[j] of lane i and v[i] of lane j change places.
__device__ __forceinline__ void turn4(uint4 (&v)[4], int lane) {
#pragma unroll
    for (int d = 1; d < 4; d *= 2) {
        const bool high = lane & d;
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            if (j & d) continue;
            // the low lane keeps v[j] and gives v[j + d], the high one the other way round
            uint32_t* keep = reinterpret_cast<uint32_t*>(&v[j]);
            uint32_t* give = reinterpret_cast<uint32_t*>(&v[j + d]);
#pragma unroll
            for (int x = 0; x < 4; ++x) {
                const uint32_t got = __shfl_xor_sync(~0u, high ? keep[x] : give[x], d);
                if (high) keep[x] = got; else give[x] = got;
            }
        }
    }
}

template <typename T>
__device__ __forceinline__ uint32_t pack2(float lo, float hi) {
    if constexpr (std::is_same<T, __half>::value) {
        const __half2 v = __floats2half2_rn(lo, hi);
        return *reinterpret_cast<const uint32_t*>(&v);
    } else {
        const __nv_bfloat162 v = __floats2bfloat162_rn(lo, hi);
        return *reinterpret_cast<const uint32_t*>(&v);
    }
}

__device__ __forceinline__ void registers_up() {
    asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(kSoftmaxRegisters));
}
__device__ __forceinline__ void registers_down() {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kOtherRegisters));
}

// The MMAs.  The whole warp comes here together, with operands that are alike in all lanes, and
// one lane, elected in the same statement, issues them: so they stay in uniform registers.  (Under
// a branch on the lane, or by a predicate of the lane's, an MMA took some 100 cycles to issue.)  A
// matrix in shared memory is given by its descriptor's low word; the high word is that of the
// layouts below.
constexpr uint32_t kDescHigh = (1024 >> 4) | (1u << 14) | (2u << 29);

// D[tmem] (+)= A[smem] * B[smem]^T over 64 of K, K-major; 16-bit inputs, f32 accumulate.
__device__ __forceinline__ void mma_ss_64(uint32_t d, uint32_t a, uint32_t b, uint32_t idesc,
                                          uint32_t accumulate) {
    asm volatile(
        "{\n\t.reg .pred p, q;\n\t.reg .b64 x, y;\n\t.reg .b32 a, b;\n\t"
        "elect.sync _|q, 0xffffffff;\n\t"
        "setp.ne.b32 p, %5, 0;\n\t"
        "mov.b64 x, {%1, %3};\n\t"
        "mov.b64 y, {%2, %3};\n\t"
        "@q tcgen05.mma.cta_group::1.kind::f16 [%0], x, y, %4, p;\n\t"
        "add.u32 a, %1, 2;\n\t"
        "add.u32 b, %2, 2;\n\t"
        "mov.b64 x, {a, %3};\n\t"
        "mov.b64 y, {b, %3};\n\t"
        "@q tcgen05.mma.cta_group::1.kind::f16 [%0], x, y, %4, 1;\n\t"
        "add.u32 a, %1, 4;\n\t"
        "add.u32 b, %2, 4;\n\t"
        "mov.b64 x, {a, %3};\n\t"
        "mov.b64 y, {b, %3};\n\t"
        "@q tcgen05.mma.cta_group::1.kind::f16 [%0], x, y, %4, 1;\n\t"
        "add.u32 a, %1, 6;\n\t"
        "add.u32 b, %2, 6;\n\t"
        "mov.b64 x, {a, %3};\n\t"
        "mov.b64 y, {b, %3};\n\t"
        "@q tcgen05.mma.cta_group::1.kind::f16 [%0], x, y, %4, 1;\n\t}" ::"r"(d),
        "r"(a), "r"(b), "r"(kDescHigh), "r"(idesc), "r"(accumulate)
        : "memory");
}

// D[tmem] (+)= A[tmem] * B[smem] over 32 of K, B MN-major.
__device__ __forceinline__ void mma_ts_32(uint32_t d, uint32_t a, uint32_t b, uint32_t idesc,
                                          uint32_t accumulate) {
    asm volatile(
        "{\n\t.reg .pred p, q;\n\t.reg .b64 y;\n\t.reg .b32 a, b;\n\t"
        "elect.sync _|q, 0xffffffff;\n\t"
        "setp.ne.b32 p, %5, 0;\n\t"
        "mov.b64 y, {%2, %3};\n\t"
        "@q tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], y, %4, p;\n\t"
        "add.u32 a, %1, 8;\n\t"
        "add.u32 b, %2, 128;\n\t"
        "mov.b64 y, {b, %3};\n\t"
        "@q tcgen05.mma.cta_group::1.kind::f16 [%0], [a], y, %4, 1;\n\t}" ::"r"(d),
        "r"(a), "r"(b), "r"(kDescHigh), "r"(idesc), "r"(accumulate)
        : "memory");
}

__device__ __forceinline__ void mma_commit(uint32_t bar) {
    asm volatile(
        "{\n\t.reg .pred q;\n\t"
        "elect.sync _|q, 0xffffffff;\n\t"
        "@q tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];\n\t}" ::"r"(bar)
        : "memory");
}

// Low words of descriptors, 128-byte swizzle.  Queries and keys: dimensions along the rows of
// shared memory (K-major).  V as the right operand [positions x dims]: again dims along the rows,
// which is MN-major: 64 of them are a row, `block` bytes from one such block to the next, 1024
// bytes from eight positions to the next eight.
__device__ __forceinline__ uint32_t desc_k_major(uint32_t smem_addr) { return smem_addr >> 4 | 1u << 16; }
__device__ __forceinline__ uint32_t desc_mn_major(uint32_t smem_addr, uint32_t block) {
    return smem_addr >> 4 | block >> 4 << 16;
}

// tcgen05.ld; its registers are to be used behind tmem_ld_wait and tmem_loaded only.
__device__ __forceinline__ void tmem_load(uint32_t taddr, uint32_t (&r)[32]) {
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x32.b32 {"
        "%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, "
        "%16, %17, %18, %19, %20, %21, %22, %23, %24, %25, %26, %27, %28, %29, %30, %31 "
        "}, [%32];"
        : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]),
          "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15]),
          "=r"(r[16]), "=r"(r[17]), "=r"(r[18]), "=r"(r[19]), "=r"(r[20]), "=r"(r[21]), "=r"(r[22]), "=r"(r[23]),
          "=r"(r[24]), "=r"(r[25]), "=r"(r[26]), "=r"(r[27]), "=r"(r[28]), "=r"(r[29]), "=r"(r[30]), "=r"(r[31])
        : "r"(taddr)
        : "memory");
}
__device__ __forceinline__ void tmem_load(uint32_t taddr, uint32_t (&r)[64]) {
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x64.b32 {"
        "%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, "
        "%16, %17, %18, %19, %20, %21, %22, %23, %24, %25, %26, %27, %28, %29, %30, %31, "
        "%32, %33, %34, %35, %36, %37, %38, %39, %40, %41, %42, %43, %44, %45, %46, %47, "
        "%48, %49, %50, %51, %52, %53, %54, %55, %56, %57, %58, %59, %60, %61, %62, %63 "
        "}, [%64];"
        : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]),
          "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15]),
          "=r"(r[16]), "=r"(r[17]), "=r"(r[18]), "=r"(r[19]), "=r"(r[20]), "=r"(r[21]), "=r"(r[22]), "=r"(r[23]),
          "=r"(r[24]), "=r"(r[25]), "=r"(r[26]), "=r"(r[27]), "=r"(r[28]), "=r"(r[29]), "=r"(r[30]), "=r"(r[31]),
          "=r"(r[32]), "=r"(r[33]), "=r"(r[34]), "=r"(r[35]), "=r"(r[36]), "=r"(r[37]), "=r"(r[38]), "=r"(r[39]),
          "=r"(r[40]), "=r"(r[41]), "=r"(r[42]), "=r"(r[43]), "=r"(r[44]), "=r"(r[45]), "=r"(r[46]), "=r"(r[47]),
          "=r"(r[48]), "=r"(r[49]), "=r"(r[50]), "=r"(r[51]), "=r"(r[52]), "=r"(r[53]), "=r"(r[54]), "=r"(r[55]),
          "=r"(r[56]), "=r"(r[57]), "=r"(r[58]), "=r"(r[59]), "=r"(r[60]), "=r"(r[61]), "=r"(r[62]), "=r"(r[63])
        : "r"(taddr)
        : "memory");
}
// The wait for all loads so far.  What they loaded goes through `loaded` behind it, so that nothing
// uses it before.
template <int N>
__device__ __forceinline__ void tmem_loaded(uint32_t (&r)[N]) {
#pragma unroll
    for (int i = 0; i < N; ++i) asm volatile("" : "+r"(r[i]));
}

__device__ __forceinline__ void tmem_st_32x32b_x16(uint32_t taddr, const uint32_t (&r)[16]) {
    asm volatile(
        "tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], "
        "{%1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, %16};" ::"r"(taddr),
        "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]),
        "r"(r[8]), "r"(r[9]), "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15])
        : "memory");
}
__device__ __forceinline__ void tmem_st_32x32b_x32(uint32_t taddr, const uint32_t (&r)[32]) {
    asm volatile(
        "tcgen05.st.sync.aligned.32x32b.x32.b32 [%0], "
        "{%1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, %16, "
        "%17, %18, %19, %20, %21, %22, %23, %24, %25, %26, %27, %28, %29, %30, %31, %32};" ::"r"(taddr),
        "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]),
        "r"(r[8]), "r"(r[9]), "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15]),
        "r"(r[16]), "r"(r[17]), "r"(r[18]), "r"(r[19]), "r"(r[20]), "r"(r[21]), "r"(r[22]), "r"(r[23]),
        "r"(r[24]), "r"(r[25]), "r"(r[26]), "r"(r[27]), "r"(r[28]), "r"(r[29]), "r"(r[30]), "r"(r[31])
        : "memory");
}
__device__ __forceinline__ void tmem_st_wait() {
    asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory");
}

// ---------------------------------------------------------------------------
// The attention
// ---------------------------------------------------------------------------
// A unit of work as every warp reads it.
struct Unit {
    Item item;
    int head, first, steps, part;  // steps < 0: no more units
};

// Values that are not finite, in steps that some of the item's queries see in part: the first
// position of each dimension with NaN, +infinity and -infinity.  They enter the products as
// zeros, so that queries before them are left alone.
template <int DP>
struct Odd {
    int any;
    int first[3][DP];
};

template <int DP>
struct Rest {
    uint64_t unit_full[2], unit_free[2], unit_wanted, q_full, q_free;
    uint64_t kv_full[kSlots], kv_free[kSlots], looked[kSlots];
    uint64_t s_full[2], p_full[2][2], o_full[2], other_full, other_free, done;
    uint32_t tmem;
    uint32_t valid[4][4];  // of a step, a bit a position (step / 4 a word)
    Unit unit[2];
    float2 other[kQueryTile];  // maxima and sums of the second group's steps of the first tile
    Odd<DP> odd[kUnits];
};

// (With DP = 256 a softmax thread spills 4 bytes, of 20 that it loads again.)
template <typename T, int DP>
__global__ void __launch_bounds__(kThreads, 1)
    chunk_kernel(const __grid_constant__ CUtensorMap q_map, const __grid_constant__ CUtensorMap k_map,
                 const __grid_constant__ CUtensorMap v_map, const __grid_constant__ ChunkArgs a) {
    using S = Shape<DP>;
    static_assert(sizeof(Rest<DP>) <= 16384, "the rest of shared memory");
    constexpr bool kHalf = std::is_same<T, __half>::value;
    // Weights are held times 2^headroom: FP16 has nothing below 2^-24, and many small weights
    // beside a large one would vanish.  A new maximum is let be up to 2^slack above the old.
    constexpr float kHeadroom = kHalf ? 12.f : 0.f, kSlack = kHalf ? 3.f : 8.f;
    extern __shared__ uint8_t smem_raw[];
    const uint32_t base = (smem_u32(smem_raw) + 1023u) & ~1023u;
    uint8_t* smem = smem_raw + (base - smem_u32(smem_raw));
    Rest<DP>& rest = *reinterpret_cast<Rest<DP>*>(smem + S::kOffRest);
    // (by a shuffle, so that a warp is known to take one way together: its addresses and loop counts
    // stay in uniform registers, which the MMAs want; without it 1 row of 2048 after 129023 takes
    // 2.80 ms for 2.56)
    const int warp = __shfl_sync(~0u, threadIdx.x / 32, 0), lane = threadIdx.x % 32;
    const auto bar = [&](const uint64_t& b) { return smem_u32(&b); };

    if (threadIdx.x == 0) {
        for (int i = 0; i < 2; ++i) {
            mbar_init(bar(rest.unit_full[i]), 1);
            mbar_init(bar(rest.unit_free[i]), 4 * S::kTiles + kCopyWarps + 1 + kLookWarps);
            mbar_init(bar(rest.s_full[i]), 2);
            mbar_init(bar(rest.p_full[i][0]), 4);
            mbar_init(bar(rest.p_full[i][1]), 4);
            mbar_init(bar(rest.o_full[i]), 2);
        }
        mbar_init(bar(rest.unit_wanted), 1);
        mbar_init(bar(rest.q_full), 33 * kCopyWarps);
        mbar_init(bar(rest.q_free), 1);
        for (int i = 0; i < kSlots; ++i) {
            // every copying thread's copies, and an arrival of each warp for its boxes and its writes
            mbar_init(bar(rest.kv_full[i]), 33 * kCopyWarps);
            mbar_init(bar(rest.kv_free[i]), i % 2 ? 1 + kLookWarps : 1);  // values: also the lookers'
            mbar_init(bar(rest.looked[i]), kLookWarps);
        }
        mbar_init(bar(rest.other_full), 4);
        mbar_init(bar(rest.other_free), 4);
        mbar_init(bar(rest.done), 1);
        fence_barrier_init();
    }
    if (warp == kMmaWarp) {
        tmem_alloc(smem_u32(&rest.tmem), 512);
        tmem_relinquish();
    }
    tc_fence_before_sync();
    __syncthreads();
    tc_fence_after_sync();
    // All 512 columns are this block's, so that they begin at address 0, a constant in what follows.
    constexpr uint32_t tmem = 0;
    const bool fits = *reinterpret_cast<volatile uint32_t*>(&rest.tmem) == tmem;
    grid_dependency_wait();
    grid_launch_dependents();
    const int group = a.group.value;

    // Waits for unit number n and reads it; false where there is none, or the wait gave up.
    const auto next_unit = [&](uint32_t n, Unit& u) {
        const bool ok = warp_wait(bar(rest.unit_full[n % 2]), n / 2, a.timeout_ns, a.status);
        u.steps = -1;
        if (ok) u = rest.unit[n % 2];
        u.steps = __shfl_sync(~0u, u.steps, 0), u.first = __shfl_sync(~0u, u.first, 0);
        u.item.lin0 = __shfl_sync(~0u, u.item.lin0, 0), u.item.lins = __shfl_sync(~0u, u.item.lins, 0);
        u.item.position0 = __shfl_sync(~0u, u.item.position0, 0), u.head = __shfl_sync(~0u, u.head, 0);
        __syncwarp();
        if (ok && lane == 0) mbar_arrive(bar(rest.unit_free[n % 2]));
        return u.steps > 0;
    };
    // Steps that tile q of a unit takes part in.
    const auto steps_of = [&](const Unit& u, int q) {
        const int end = min(u.item.lins, (q + 1) * a.tile_rows);
        if (end <= q * a.tile_rows) return 0;
        const int64_t seen = (int64_t)u.item.position0 + a.group.quotient(u.item.lin0 + end - 1) + 1;
        const int64_t steps = seen > 0 ? (seen + S::kStep - 1) / S::kStep : 0;
        return (int)min(max(steps - u.first, (int64_t)0), (int64_t)u.steps);
    };
    // Whether the two softmax groups share the one tile of a unit.
    const auto one_tile = [&](const Unit& u) { return S::kTiles == 2 && u.item.lins <= a.tile_rows; };
    // The first step of a unit that some of its queries do not see whole.
    const auto part_seen_from = [&](const Unit& u) {
        const int64_t all = max((int64_t)u.item.position0 + a.group.quotient(u.item.lin0) + 1, (int64_t)0);
        return (int)min(max(all / S::kStep - u.first, (int64_t)0), (int64_t)u.steps);
    };

    if (!fits) {
        if (threadIdx.x == 0) atomicOr(a.status, kDevBadLaunch);
    } else if (warp >= kMmaWarp) {
        registers_down();
        if (warp == kUnitWarp) {
            // ============================== units ===============================
            const unsigned whole = (unsigned)a.plan->whole, parts = (unsigned)a.plan->parts;
            const unsigned heads = (unsigned)a.c.kv_heads;
            for (uint32_t n = 0;; ++n) {
                unsigned i = blockIdx.x;
                if (n) {
                    // (not before the last unit's end is near: blocks that took theirs two ahead were
                    // as good as dealt out from the start)
                    if (!warp_wait(bar(rest.unit_wanted), n - 1, a.timeout_ns, a.status)) break;
                    if (lane == 0) i = gridDim.x + atomicAdd(&a.plan->next, 1u);
                    i = __shfl_sync(~0u, i, 0);
                }
                Unit u = {};
                u.steps = -1;
                if (i < (whole + parts) * heads) {
                    const bool part = i >= whole * heads;
                    const unsigned j = part ? i - whole * heads : i;
                    u.head = (int)(j % heads);
                    const Entry entry = a.entries[(part ? a.slot_count : 0) + j / heads];
                    u.item = entry.item;
                    u.first = entry.first;
                    u.steps = entry.steps;
                    u.part = entry.part;
                }
                if (n >= 2 && !warp_wait(bar(rest.unit_free[n % 2]), n / 2 - 1, a.timeout_ns, a.status))
                    break;
                Odd<DP>& odd = rest.odd[n % kUnits];
                for (int x = lane; x < 3 * DP; x += 32) (&odd.first[0][0])[x] = INT32_MAX;
                if (lane == 0) {
                    odd.any = 0;
                    rest.unit[n % 2] = u;
                }
                __syncwarp();
                if (lane == 0) mbar_arrive(bar(rest.unit_full[n % 2]));
                if (u.steps < 0) break;
            }
        } else if (warp == kMmaWarp) {
            // =============================== MMAs ===============================
            constexpr uint32_t kType = kHalf ? 0u : (1u << 7) | (1u << 10);
            const uint32_t scores = umma_idesc_f16_f32(kQueryTile, S::kStep) | kType |
                                    (a.negative ? 1u << 13 : 0u);  // (minus the queries)
            const uint32_t values = umma_idesc_f16_f32(kQueryTile, DP) | kType | (1u << 16);  // V: MN-major
            const uint32_t q_desc = desc_k_major(base), k_desc = desc_k_major(base + S::kOffRing);
            const uint32_t v_desc = desc_mn_major(base + S::kOffRing, S::kStep * 128);
            uint32_t step = 0;         // the unit's first of the block, for the ring's slots
            uint32_t taken = 0;        // steps of each tile, modulo 2: a bit each
            uint32_t looks = 0;        // looks at each slot of values, modulo 2
            Unit u;
            bool ok = true;
            const auto wait = [&](uint64_t& b, uint32_t phase) {
                if (ok) ok = warp_wait(bar(b), phase, a.timeout_ns, a.status);
            };
            // The values of step i, as each tile's weights come, then the keys of the next step of that
            // tile.  (One loop for all of it: this code, unrolled over starts and ends too, was a
            // third of the kernel's.)
            for (uint32_t n = 0; ok && next_unit(n, u); ++n) {
                const bool shared = one_tile(u);
                const int ahead = shared ? 2 : 1;
                const int steps0 = steps_of(u, 0);
                const int steps1 = shared ? steps0 : S::kTiles == 2 ? steps_of(u, 1) : 0;
                const int looked_from = part_seen_from(u);
                wait(rest.q_full, n);
#pragma unroll 1
                for (int i = -ahead; ok && i < u.steps; ++i) {
                    const int next = i + ahead;
                    const uint32_t v = 2 * (step + i) + 1, k = 2 * (step + next);
                    if (i >= looked_from) {
                        wait(rest.looked[v % kSlots], looks >> (v % kSlots / 2));
                        looks ^= 1u << (v % kSlots / 2);
                    } else if (i >= 0) {
                        wait(rest.kv_full[v % kSlots], v / kSlots);
                    }
                    if (next < u.steps) wait(rest.kv_full[k % kSlots], k / kSlots);
                    fence_proxy_async_smem();
#pragma unroll 1
                    for (int q = 0; q < S::kTiles; ++q) {
                        const int steps = q ? steps1 : steps0;
                        if (i >= steps || (shared && (i & 1) != q)) continue;
                        if (i >= 0) {
                            // the first half of the weights, while the second is still made
#pragma unroll
                            for (int half = 0; half < 2; ++half) {
                                wait(rest.p_full[q][half], taken >> q);
                                if (!ok) break;
                                tc_fence_after_sync();
                                const uint32_t va = v_desc + v % kSlots * (S::kSlotBytes >> 4) +
                                                    half * (S::kStep / 2 * 128 >> 4);
                                const uint32_t pa = tmem + q * 128 + half * (S::kStep / 4);
#pragma unroll
                                for (int j = 0; j < S::kStep / 64; ++j)
                                    mma_ts_32(tmem + S::kOutColumn + q * DP, pa + 16 * j, va + j * (4096 >> 4),
                                              values, i >= ahead || (half | j) != 0);
                            }
                            if (!ok) break;
                            taken ^= 1u << q;
                        }
                        const bool more = next < steps;
                        if (more) {
                            const uint32_t qa = q_desc + (shared ? 0 : q * (S::kTileBytes >> 4));
                            const uint32_t ka = k_desc + k % kSlots * (S::kSlotBytes >> 4);
#pragma unroll
                            for (int j = 0; j < DP / 64; ++j)
                                mma_ss_64(tmem + q * 128, qa + j * (kQueryTile * 8), ka + j * (S::kStep * 8),
                                          scores, j != 0);
                        }
                        if (more || i >= 0) {
                            // reports the MMAs issued so far, and passes on (by an arrival of this
                            // thread) what the copying warps wrote
                            const uint32_t to = more ? bar(rest.s_full[q]) : bar(rest.o_full[q]);
                            mma_commit(to);
                            if (lane == 0) mbar_arrive(to);
                        }
                    }
                    if (!ok) break;
                    if (i >= 0) mma_commit(bar(rest.kv_free[v % kSlots]));
                    if (next < u.steps) mma_commit(bar(rest.kv_free[k % kSlots]));
                    if (next + 1 == u.steps) mma_commit(bar(rest.q_free));
                }
                step += u.steps;
            }
            // nothing in flight when the block ends
            mma_commit(bar(rest.done));
            warp_wait(bar(rest.done), 0, drain_bound(a.timeout_ns), a.status);
        } else {
            // ============================== looking =============================
            constexpr uint32_t kExponent = kHalf ? 0x7C00u : 0x7F80u;
            uint32_t step = 0;
            Unit u;
            bool ok = true;
            for (uint32_t n = 0; ok && next_unit(n, u); ++n) {
                Odd<DP>& odd = rest.odd[n % kUnits];
                const int looked_from = part_seen_from(u);
                for (int i = 0; i < u.steps; ++i, ++step) {
                    // (every step's, so that the barriers' phases are followed one by one)
                    const uint32_t v = 2 * step + 1, slot = v % kSlots;
                    ok = warp_wait(bar(rest.kv_full[slot]), v / kSlots, a.timeout_ns, a.status);
                    if (!ok) break;
                    if (i < looked_from) {
                        if (lane == 0) mbar_arrive(bar(rest.kv_free[slot]));
                        continue;
                    }
                    const uint32_t from = base + S::kOffRing + slot * S::kSlotBytes;
                    // Eight pieces at a time, by the largest of the magnitudes' bits; any one that
                    // is not finite is then looked for.
                    constexpr int kAhead = 8, kEach = S::kSlotBytes / 16 / (32 * kLookWarps);
#pragma unroll 1
                    for (int first = 0; first < kEach; first += kAhead) {
                        const uint32_t x0 = ((warp - kLookWarp) * kEach + first) * 32 + lane;
                        uint4 piece[kAhead];
#pragma unroll
                        for (int y = 0; y < kAhead; ++y) piece[y] = lds128(from + 16 * (x0 + 32 * y));
                        uint32_t most = 0;
#pragma unroll
                        for (int y = 0; y < kAhead; ++y) {
                            most = __vmaxu2(most, piece[y].x & 0x7FFF7FFFu);
                            most = __vmaxu2(most, piece[y].y & 0x7FFF7FFFu);
                            most = __vmaxu2(most, piece[y].z & 0x7FFF7FFFu);
                            most = __vmaxu2(most, piece[y].w & 0x7FFF7FFFu);
                        }
                        if ((most & 0xFFFFu) < kExponent && most >> 16 < kExponent) continue;
#pragma unroll 1
                        for (int y = 0; y < 8 * kAhead; ++y) {
                            const uint32_t x = x0 + 32 * (y / 8);
                            // value y % 8 of piece x: its row, and its dimension behind the swizzle
                            const uint32_t where = from + 16 * x + 2 * (y % 8);
                            const int row = x / 8 % S::kStep;
                            const int dim = (x / 8 / S::kStep * 8 + (x % 8 ^ row % 8)) * 8 + y % 8;
                            uint16_t one;
                            asm volatile("ld.shared.u16 %0, [%1];" : "=h"(one) : "r"(where) : "memory");
                            if ((one & kExponent) != kExponent) continue;
                            const int kind = (one & (kExponent ^ 0x7FFFu)) ? 0 : one >> 15 ? 2 : 1;
                            atomicMin(&odd.first[kind][dim], (u.first + i) * S::kStep + row);
                            odd.any = 1;
                            asm volatile("st.shared.u16 [%0], %1;" ::"r"(where), "h"((uint16_t)0) : "memory");
                        }
                    }
                    fence_proxy_async_smem();
                    __syncwarp();
                    if (lane == 0) {
                        mbar_arrive(bar(rest.looked[slot]));
                        mbar_arrive(bar(rest.kv_free[slot]));
                    }
                }
            }
        }
    } else if (warp >= kSoftmaxWarps) {
        // =============================== copies ===============================
        registers_down();
        constexpr int kPieces = DP / 8;              // of a row, 16 bytes each
        constexpr int kRowsPass = kPieces < 32 ? 32 / kPieces : 1;
        static_assert(kPieces <= 32, "a pass of a warp is whole rows");
        constexpr int kRowsWarp = S::kStep / kCopyWarps;
        const int w = warp - kSoftmaxWarps, piece = lane % kPieces, row0 = lane / kPieces;
        const bool in_dim = piece * 8 < a.c.head_dim;
        // a piece's place in a tile of `rows` rows: blocks of 64 dimensions, swizzled by the row
        const auto at = [&](int row, int rows) {
            return (uint32_t)(piece / 8 * rows * 128 + row * 128 + ((piece % 8 ^ row % 8) << 4));
        };
        uint32_t step = 0;
        Unit u;
        bool ok = true;
        const auto wait = [&](uint64_t& b, uint32_t phase) {
            ok = warp_wait(bar(b), phase, a.timeout_ns, a.status);
        };
        for (uint32_t n = 0; ok && next_unit(n, u); ++n) {
            const int64_t head = (int64_t)u.head * a.c.head_stride;
            const int32_t* table = a.tables + u.item.row * a.c.table_stride;
            // this lane's position in step i, and its page
            const auto position_of = [&](int i) {
                return (int64_t)(u.first + i) * S::kStep + w * kRowsWarp + lane % kRowsWarp;
            };
            const auto page_of = [&](int i) {
                const int64_t p = position_of(i);
                return p < u.item.length ? table[a.c.page_size.quotient((int)p)] : -1;
            };
            // Keys and values in turn; where two groups share a tile, the keys a step further ahead.
            const int lag = one_tile(u) ? 1 : 0;
            int next = page_of(0), behind = -1;  // pages of the step to come, and of the one before
            for (int i = 0; i < u.steps + lag; ++i) {
                const int now = next;
                if (i + 1 < u.steps) next = page_of(i + 1);
                if (w == 0 && lane == 0 && i == max(u.steps - kWanted, 0)) mbar_arrive(bar(rest.unit_wanted));
#pragma unroll 1
                for (int value = 0; value < 2; ++value) {
                    const int of = value ? i - lag : i;  // the step
                    if (of < 0 || of >= u.steps) continue;
                    const int page = value && lag ? behind : now;
                    const int in_page = a.c.page_size.remainder((int)position_of(of));
                    const bool there = (uint32_t)page < (uint32_t)a.c.pages;
                    const uint32_t all = __ballot_sync(~0u, there);
                    const uint32_t g = 2 * (step + of) + value, slot = g % kSlots;
                    if (g >= kSlots) wait(rest.kv_free[slot], g / kSlots - 1);
                    if (!ok) break;
                    if (!value && lane == 0)
                        rest.valid[(step + of) % 4][w] =
                            kRowsWarp == 32 ? all : all & ((1u << kRowsWarp % 32) - 1);
                    const uint32_t to = base + S::kOffRing + slot * S::kSlotBytes;
                    const uint32_t full = bar(rest.kv_full[slot]);
                    if (a.box_rows && all == ~0u) {
                        if (lane == 0) mbar_arrive_expect_tx(full, kRowsWarp * DP * 2);
                        __syncwarp();
                        fence_proxy_async_smem();  // (rows of the slot that were written one by one)
                        for (int r = 0; r < kRowsWarp; r += a.box_rows) {
                            const int in_box = __shfl_sync(~0u, in_page, r), box = __shfl_sync(~0u, page, r);
#pragma unroll
                            for (int x = 0; x < DP / 64; ++x)
                                box_load_4d(to + x * S::kStep * 128 + (w * kRowsWarp + r) * 128,
                                            value ? &v_map : &k_map, 64 * x, in_box, u.head, box, full);
                        }
                    } else {
                        const uint16_t* pool = (value ? a.v_pool : a.k_pool) + 8 * piece;
                        const int64_t place =
                            there ? page * a.c.page_stride + in_page * a.c.slot_stride + head : -1;
#pragma unroll 4
                        for (int r = 0; r < kRowsWarp; r += kRowsPass) {
                            const int64_t o = __shfl_sync(~0u, place, r + row0);
                            const bool in = o >= 0 && in_dim;
                            copy16(to + at(w * kRowsWarp + r + row0, S::kStep), in ? pool + o : a.k_pool,
                                   in);
                        }
                        if (lane == 0) mbar_arrive(full);
                    }
                    copy_arrive(full);
                    if (value || i) continue;
                    // the queries, behind the first keys: theirs is the longer wait
                    if (n > 0) wait(rest.q_free, n - 1);
                    if (!ok) break;
                    const uint32_t queries = bar(rest.q_full);
                    if (a.q_map) {
                        const int tiles = u.item.lins > a.tile_rows ? 2 : 1;
                        if (lane == 0) {
                            if (w)
                                mbar_arrive(queries);
                            else
                                mbar_arrive_expect_tx(queries, tiles * a.tile_rows * DP * 2);
                        }
                        __syncwarp();
                        const int token = (int)(int64_t)u.item.token0 + a.group.quotient(u.item.lin0);
                        const int tokens = a.group.quotient(a.tile_rows);
                        for (int q = 0; w == 0 && q < tiles; ++q)
#pragma unroll
                            for (int x = 0; x < DP / 64; ++x)
                                box_load_3d(base + q * S::kTileBytes + x * (kQueryTile * 128), &q_map, 64 * x,
                                            u.head * group, token + q * tokens, queries);
                    } else {
                        const uint16_t* q0 = a.q + (int64_t)u.item.token0 * a.q_row + (int64_t)u.head * group * a.q_head;
#pragma unroll 1
                        for (int r = w * (S::kRows / kCopyWarps) + row0; r < (w + 1) * (S::kRows / kCopyWarps);
                             r += kRowsPass) {
                            const int row = r % kQueryTile, lin = r / kQueryTile * a.tile_rows + row;
                            const bool in = row < a.tile_rows && lin < u.item.lins && in_dim;
                            const int token = a.group.quotient(u.item.lin0 + lin);
                            const int h = u.item.lin0 + lin - token * group;
                            copy16(base + r / kQueryTile * S::kTileBytes + at(row, kQueryTile),
                                   in ? q0 + token * a.q_row + h * a.q_head + 8 * piece : a.q, in);
                        }
                        if (lane == 0) mbar_arrive(queries);
                    }
                    copy_arrive(queries);
                }
                if (!ok) break;
                behind = now;
            }
            step += u.steps;
        }
        copy_commit();
        copy_wait<0>();
        if (!ok) {  // a wait gave up: boxes on their way land before the block ends
            const uint64_t since = global_timer_ns();
            while (global_timer_ns() - since < kDrainFloorNs) {}
        }
    } else if (warp < 4 * S::kTiles) {
        // ============================== softmax ===============================
        registers_up();
        const int q = warp / 4, r = warp % 4 * 32 + lane;
        const uint32_t lanes = (uint32_t)(warp % 4 * 32) << 16;
        const uint32_t t_scores = tmem + lanes + q * 128;
        const uint32_t t_out = tmem + lanes + S::kOutColumn + q * DP;
        // What no unit writes, dealt out over all blocks; of a row, a slot's tokens at a time.  (Rows
        // left to a block each, a thread a head, took 3.0 ms for 8192 tokens without a position beside
        // 64 after 636, and the block's other warps waited through all of it; this takes 61 us, of
        // which the 64 MB of zeros are 16.)
        const int pieces = a.c.head_dim / 8;
        const auto zero = [&](int64_t t, int h, int piece) {
            *reinterpret_cast<uint4*>(a.out + t * a.out_row + h * a.out_head + 8 * piece) =
                make_uint4(0, 0, 0, 0);
            if (a.lse && piece == 0) a.lse[t * a.q_heads + h] = -INFINITY;
        };
        // queries of positions below 0
#pragma unroll 1
        for (int64_t s0 = blockIdx.x; s0 < a.slot_count; s0 += 32 * (int64_t)gridDim.x) {
            const int64_t s = s0 + (int64_t)lane * gridDim.x;
            bool some = false;
            if (s < a.slot_count) {
                const Item& item = a.slots[s].item;
                some = item.lins > 0 && item.position0 + a.group.quotient(item.lin0) < 0;
            }
            uint32_t all = __ballot_sync(~0u, some);
#pragma unroll 1
            for (; all; all &= all - 1) {
                const Item item = a.slots[s0 + (int64_t)(__ffs(all) - 1) * gridDim.x].item;
                const int below = (int)min((int64_t)item.lins, -(int64_t)item.position0 * group - item.lin0);
#pragma unroll 1
                for (int i = threadIdx.x; i < below * a.c.kv_heads * pieces; i += 128 * S::kTiles) {
                    const int query = i / pieces, lin = item.lin0 + query / a.c.kv_heads;
                    const int token = a.group.quotient(lin);
                    zero((int64_t)item.token0 + token, query % a.c.kv_heads * group + lin - token * group,
                         i % pieces);
                }
            }
        }
        // tokens before the first row and behind the last
        {
            const int64_t from = a.offset(0), to = a.offset(a.c.batch);
            const int64_t held = max(to - from, (int64_t)0);
#pragma unroll 1
            for (int64_t i = blockIdx.x; i < a.tokens - held; i += gridDim.x)
#pragma unroll 1
                for (int x = threadIdx.x; x < a.q_heads * pieces; x += 128 * S::kTiles)
                    zero(i < from ? i : i + to - from, x / pieces, x % pieces);
        }
        // steps and units of this group, joined units, steps of the block
        uint32_t taken = 0, units = 0, joins = 0, step0 = 0;
        bool ok = true;
        const float2 scale2 = make_float2(a.scale_log2, a.scale_log2);
        for (uint32_t n = 0;; ++n) {
            ok = warp_wait(bar(rest.unit_full[n % 2]), n / 2, a.timeout_ns, a.status);
            // (stays where it is until the unit is done: the scores take most registers)
            const Unit& u = rest.unit[n % 2];
            if (!ok || u.steps < 0) break;
            // steps first, first + stride, ... of the unit are this group's
            const bool shared = one_tile(u);
            const int tile = shared ? 0 : q, stride = shared ? 2 : 1;
            int steps = __shfl_sync(~0u, steps_of(u, tile), 0);
            const bool joined = shared && steps > 1;
            if (shared) steps = (steps + 1 - q) / 2;
            const int lin = u.item.lin0 + tile * a.tile_rows + r;
            const bool in = r < a.tile_rows && tile * a.tile_rows + r < u.item.lins;
            const int token = a.group.quotient(lin), h = u.head * group + lin - token * group;
            // positions that the query sees; all, for a row that is not there
            const int limit = in ? max(u.item.position0 + token + 1, 0) : INT32_MAX;
            const int least = __reduce_min_sync(~0u, limit);
            const int first = u.first + (shared ? q : 0);
            float top = -INFINITY;
            float2 sum2 = make_float2(0.f, 0.f), more2 = sum2;
#pragma unroll 1
            for (int i = 0; i < steps; ++i) {
                ok = warp_wait(bar(rest.s_full[q]), taken, a.timeout_ns, a.status);
                if (!ok) break;
                ++taken;
                tc_fence_after_sync();
                const int position = (first + i * stride) * S::kStep;
                uint32_t part[S::kStep / 64][64];
#pragma unroll
                for (int k = 0; k < S::kStep / 64; ++k) tmem_load(t_scores + 64 * k, part[k]);
                tmem_ld_wait();
#pragma unroll
                for (int k = 0; k < S::kStep / 64; ++k) tmem_loaded(part[k]);
                const auto s = [&](int j) { return __uint_as_float(part[j / 64][j % 64]); };
                const uint32_t* v = rest.valid[(step0 + (shared ? q : 0) + i * stride) % 4];
                bool whole = least - position >= S::kStep;
#pragma unroll
                for (int k = 0; k < 4; ++k)
                    whole = whole && v[k] == (S::kStep == 128 ? ~0u : 0xFFFFu);
                if (!whole) {  // scores that do not count become -infinity
                    const int left = min(max(limit - position, 0), S::kStep);
#pragma unroll
                    for (int k = 0; k < S::kStep / 32; ++k) {
                        uint32_t bits = S::kStep == 128 ? v[k] : v[2 * k] | v[2 * k + 1] << 16;
                        bits &= left >= 32 * k + 32 ? ~0u
                                : left <= 32 * k    ? 0u
                                                    : (1u << (left - 32 * k)) - 1;
#pragma unroll
                        for (int j = 0; j < 32; ++j) {
                            uint32_t& x = part[k / 2][k % 2 * 32 + j];
                            x = bits >> j & 1 ? x : 0xFF800000u;
                        }
                    }
                }
                float high[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
#pragma unroll
                for (int j = 0; j < S::kStep; j += 8)
#pragma unroll
                    for (int x = 0; x < 4; ++x)
                        high[x] = max3(high[x], s(j + 2 * x), s(j + 2 * x + 1));
                float highest = fmaxf(max3(high[0], high[1], high[2]), high[3]);
                highest = highest == -INFINITY ? highest : highest * a.scale_log2;
                if (__any_sync(~0u, highest > top + kSlack)) {
                    // (each query by its own: what the others see makes no difference to it)
                    const float higher = highest > top + kSlack ? highest : top;
                    const float keep = higher == top ? 1.f : exp2_fast(top - higher);
                    top = higher;
                    sum2.x *= keep, sum2.y *= keep, more2.x *= keep, more2.y *= keep;
                    if (i > 0) {
                        // (the scores are there, so the MMAs before them are done)
#pragma unroll 1
                        for (int c = 0; c < DP; c += 32) {
                            uint32_t o[32];
                            tmem_load(t_out + c, o);
                            tmem_ld_wait();
                            tmem_loaded(o);
#pragma unroll
                            for (int j = 0; j < 32; ++j) o[j] = __float_as_uint(__uint_as_float(o[j]) * keep);
                            tmem_st_32x32b_x32(t_out + c, o);
                        }
                    }
                }
                const float down = kHeadroom - (top == -INFINITY ? 0.f : top);
                const float2 down2 = make_float2(down, down);
#pragma unroll
                for (int k = 0; k < S::kStep / 32; ++k) {
                    uint32_t p[16];
#pragma unroll
                    for (int j = 0; j < 32; j += 2) {
                        const float2 x =
                            __ffma2_rn(make_float2(s(32 * k + j), s(32 * k + j + 1)), scale2, down2);
                        const float2 e = make_float2(exp2_fast(x.x), exp2_fast(x.y));
                        float2& to = j % 4 ? more2 : sum2;
                        to = __fadd2_rn(to, e);
                        p[j / 2] = pack2<T>(e.x, e.y);
                    }
                    tmem_st_32x32b_x16(t_scores + 16 * k, p);
                    if (k % (S::kStep / 64) == S::kStep / 64 - 1) {  // half of them
                        tmem_st_wait();
                        tc_fence_before_sync();
                        __syncwarp();
                        if (lane == 0) mbar_arrive(bar(rest.p_full[q][k / (S::kStep / 64)]));
                    }
                }
            }
            if (!ok) break;
            float sum = (sum2.x + sum2.y) + (more2.x + more2.y);
            const bool whole = u.part < 0;
            const int64_t part = whole ? 0 : (int64_t)u.part * a.c.kv_heads + u.head;
            if (steps > 0) {
                ok = warp_wait(bar(rest.o_full[q]), units, a.timeout_ns, a.status);
                if (!ok) break;
                ++units;
                tc_fence_after_sync();
            }
            if (shared && q == 1) {
                // The second group's part is the first's to write; its output must stay until then.
                if (joined) {
                    rest.other[r] = make_float2(top, sum);
                    tc_fence_before_sync();
                    __syncwarp();
                    if (lane == 0) mbar_arrive(bar(rest.other_full));
                    ok = warp_wait(bar(rest.other_free), joins, a.timeout_ns, a.status);
                    if (!ok) break;
                    ++joins;
                }
            } else if (steps > 0) {
                float keep = 1.f, add = 0.f;  // of this group's part, of the other's
                if (joined) {
                    ok = warp_wait(bar(rest.other_full), joins, a.timeout_ns, a.status);
                    if (!ok) break;
                    ++joins;
                    tc_fence_after_sync();
                    const float2 other = rest.other[r];
                    const float higher = fmaxf(top, other.x), base_exp = higher == -INFINITY ? 0.f : higher;
                    keep = exp2_fast(top - base_exp);
                    add = exp2_fast(other.x - base_exp);
                    sum = keep * sum + add * other.y;
                    top = higher;
                }
                const float inv = whole ? (sum == 0.f ? 0.f : 1.f / sum) : 1.f;
                const int64_t t = (int64_t)u.item.token0 + token;
                // (a query that sees nothing has its zeros already)
                uint16_t* mine = in && limit > 0 ? a.out + t * a.out_row + h * a.out_head : nullptr;
                float* part_to = a.partial + ((part * S::kTiles + tile) * (DP / 4) * kQueryTile + r) * 4;
                uint16_t* there[4];  // of the four neighbours' queries
#pragma unroll
                for (int j = 0; j < 4; ++j)
                    there[j] = reinterpret_cast<uint16_t*>(
                        __shfl_sync(~0u, reinterpret_cast<uint64_t>(mine), lane / 4 * 4 + j));
#pragma unroll 1
                for (int c = 0; c < DP; c += 32) {
                    uint32_t o[32];
                    __syncwarp();
                    tmem_load(t_out + c, o);
                    if (joined) {
                        uint32_t other[32];
                        tmem_load(t_out + DP + c, other);
                        tmem_ld_wait();
                        tmem_loaded(o);
                        tmem_loaded(other);
#pragma unroll
                        for (int j = 0; j < 32; ++j)
                            o[j] = __float_as_uint(keep * __uint_as_float(o[j]) +
                                                   add * __uint_as_float(other[j]));
                    }
                    tmem_ld_wait();
                    tmem_loaded(o);
                    if (whole) {
                        // Four neighbours turn their four pieces of 16 bytes each around, so that
                        // every store has 64 bytes of a query in a row: half the sectors.
                        uint4 v[4];
#pragma unroll
                        for (int j = 0; j < 4; ++j) {
                            const auto two = [&](int x) {
                                return pack2<T>(__uint_as_float(o[8 * j + x]) * inv,
                                                __uint_as_float(o[8 * j + x + 1]) * inv);
                            };
                            v[j] = make_uint4(two(0), two(2), two(4), two(6));
                        }
                        turn4(v, lane);
                        const int x = c + lane % 4 * 8;
#pragma unroll
                        for (int j = 0; j < 4; ++j)
                            if (there[j] && x < a.c.head_dim) *reinterpret_cast<uint4*>(there[j] + x) = v[j];
                    } else if (in) {
                        float* to = part_to + (int64_t)c * kQueryTile;
#pragma unroll
                        for (int j = 0; j < 32; j += 4)
                            *reinterpret_cast<uint4*>(to + j * kQueryTile) =
                                make_uint4(o[j], o[j + 1], o[j + 2], o[j + 3]);
                    }
                }
                if (joined) {
                    tc_fence_before_sync();
                    __syncwarp();
                    if (lane == 0) mbar_arrive(bar(rest.other_free));
                }
            }
            const bool writes = !(shared && q == 1);
            if (steps > 0 && writes && *reinterpret_cast<const volatile int*>(&rest.odd[n % kUnits].any) != 0) {
                // What was not finite is added to what was written, in the dimensions it is in.
                __syncwarp();
                const Odd<DP>& odd = rest.odd[n % kUnits];
                for (int d = 0; in && limit > 0 && d < a.c.head_dim; ++d) {
                    float x = 0.f;
                    if (odd.first[1][d] < limit) x += INFINITY;
                    if (odd.first[2][d] < limit) x -= INFINITY;
                    if (odd.first[0][d] < limit) x += NAN;
                    if (x == 0.f) continue;
                    if (whole) {
                        T* o = reinterpret_cast<T*>(a.out) + ((int64_t)u.item.token0 + token) * a.out_row +
                               h * a.out_head + d;
                        *o = (T)((float)*o + x);
                    } else {
                        a.partial[((part * S::kTiles + tile) * (DP / 4) + d / 4) * (4 * kQueryTile) + 4 * r +
                                  d % 4] += x;
                    }
                }
            }
            if (in && writes && whole && limit > 0 && a.lse)
                a.lse[((int64_t)u.item.token0 + token) * a.q_heads + h] =
                    sum == 0.f ? -INFINITY : (top - kHeadroom + log2f(sum)) * kLn2;
            if (in && writes && !whole)
                a.partial_ml[part * S::kRows + tile * kQueryTile + r] = make_float2(top - kHeadroom, sum);
            step0 += u.steps;
            __syncwarp();
            if (lane == 0) mbar_arrive(bar(rest.unit_free[n % 2]));
        }
    }
    tc_fence_before_sync();
    __syncthreads();
    tc_fence_after_sync();
    if (warp == kMmaWarp) tmem_dealloc(*reinterpret_cast<volatile uint32_t*>(&rest.tmem), 512);
}

// ---------------------------------------------------------------------------
// The join
// ---------------------------------------------------------------------------
// Adds up items' parts; a block takes eight dimensions of a tile's 128 queries at a time.
template <typename T, int DP>
__global__ void __launch_bounds__(kJoinThreads) join_kernel(ChunkArgs a) {
    using S = Shape<DP>;
    grid_dependency_wait();
    grid_launch_dependents();
    const int pieces = a.c.head_dim / 8, r = threadIdx.x;
    const int work = a.plan->joints * a.c.kv_heads * S::kTiles * pieces;
    for (int i = blockIdx.x; i < work; i += gridDim.x) {
        const int piece = i % pieces, tile = i / pieces, q = tile % S::kTiles, item = tile / S::kTiles;
        const int which = item / a.c.kv_heads, head = item - which * a.c.kv_heads;
        const Joint joint = a.joints[which];
        const int of_item = q * a.tile_rows + r;
        if (r >= a.tile_rows || of_item >= joint.item.lins) continue;
        const int lin = joint.item.lin0 + of_item;
        const int token = a.group.quotient(lin), h = head * a.group.value + lin - token * a.group.value;
        if (joint.item.position0 + token < 0) continue;  // zeros already
        float top = -INFINITY, sum = 0.f, v[8] = {};
#pragma unroll 1
        for (int first = 0; first < joint.count; first += kJoinAhead) {
            float2 ml[kJoinAhead];
            float4 x[kJoinAhead], y[kJoinAhead];
            float higher = top;
#pragma unroll
            for (int n = 0; n < kJoinAhead; ++n) {
                ml[n] = make_float2(-INFINITY, 0.f);
                if (first + n >= joint.count) continue;
                const int64_t part = (int64_t)(joint.part + first + n) * a.c.kv_heads + head;
                const float* from =
                    a.partial + (((part * S::kTiles + q) * (DP / 4) + 2 * piece) * kQueryTile + r) * 4;
                ml[n] = a.partial_ml[part * S::kRows + q * kQueryTile + r];
                x[n] = *reinterpret_cast<const float4*>(from);
                y[n] = *reinterpret_cast<const float4*>(from + 4 * kQueryTile);
                higher = fmaxf(higher, ml[n].x);
            }
            const float base = higher == -INFINITY ? 0.f : higher, keep = exp2_fast(top - base);
            top = higher;
            sum *= keep;
#pragma unroll
            for (int k = 0; k < 8; ++k) v[k] *= keep;
#pragma unroll
            for (int n = 0; n < kJoinAhead; ++n) {
                if (ml[n].y == 0.f) continue;  // no step, or nothing seen: what lies there is no output
                const float e = exp2_fast(ml[n].x - base);
                sum += e * ml[n].y;
                v[0] += e * x[n].x, v[1] += e * x[n].y, v[2] += e * x[n].z, v[3] += e * x[n].w;
                v[4] += e * y[n].x, v[5] += e * y[n].y, v[6] += e * y[n].z, v[7] += e * y[n].w;
            }
        }
        const float inv = sum == 0.f ? 0.f : 1.f / sum;
        const int64_t t = joint.item.token0 + token;
        *reinterpret_cast<uint4*>(a.out + t * a.out_row + h * a.out_head + 8 * piece) =
            make_uint4(pack2<T>(v[0] * inv, v[1] * inv), pack2<T>(v[2] * inv, v[3] * inv),
                       pack2<T>(v[4] * inv, v[5] * inv), pack2<T>(v[6] * inv, v[7] * inv));
        if (a.lse && piece == 0)
            a.lse[t * a.q_heads + h] = sum == 0.f ? -INFINITY : (top + log2f(sum)) * kLn2;
    }
}

// ---------------------------------------------------------------------------
// Launches
// ---------------------------------------------------------------------------
int padded_dim(int64_t dim) { return dim <= 64 ? 64 : dim <= 128 ? 128 : 256; }

struct Workspace {
    int64_t slot_count, most_parts;
    int64_t entries, joints, slots, partial, ml, bytes;
};
Workspace plan_workspace(const w4a16_cache_shape& c, int64_t q_heads, int64_t tokens,
                         const DeviceCtx& ctx) {
    const int64_t group = q_heads / c.kv_heads, dim = padded_dim(c.head_dim);
    const int64_t rows = tiles_of(c.head_dim) * kQueryTile;
    Workspace w;
    w.slot_count = tokens * group / (tiles_of(c.head_dim) * tile_rows_of(group)) + c.batch;
    // parts of all heads; items are at most slots, and a part has two steps or more
    const int64_t steps = (c.table_width * c.page_size + step_of(c.head_dim) - 1) / step_of(c.head_dim);
    w.most_parts = steps < 2 ? 0
                             : std::min((int64_t)kPartsPerSm * ctx.num_sms,
                                        w.slot_count * c.kv_heads * steps);
    const int64_t parts = w.most_parts / c.kv_heads;  // of one head
    w.entries = 256;
    w.joints = w.entries + (w.slot_count + parts) * (int64_t)sizeof(Entry);
    w.slots = w.joints + (parts + 1) * (int64_t)sizeof(Joint);
    w.ml = w.slots + w.slot_count * (int64_t)sizeof(Slot);
    w.partial = (w.ml + w.most_parts * rows * 8 + 255) / 256 * 256;
    w.bytes = w.partial + w.most_parts * rows * dim * 4;
    return w;
}

// Tensor maps of 128-byte rows, swizzled: sizes and byte strides from the second dimension on (a
// dimension of size 1 gets a stride that will do).  False where the strides cannot be had.
bool encode(CUtensorMap* map, bool half, const void* data, int rank, const int64_t* sizes,
            const int64_t* strides, const uint32_t* box) {
    const auto encoder = tensor_map_encoder();
    if (!encoder) return false;
    cuuint64_t dims[4], bytes[3];
    cuuint32_t boxes[4], ones[4] = {1, 1, 1, 1};
    for (int i = 0; i < rank; ++i) {
        dims[i] = (cuuint64_t)sizes[i];
        boxes[i] = box[i];
        if (i) bytes[i - 1] = (cuuint64_t)(sizes[i] == 1 ? 16 : 2 * strides[i]);
        if (i && (bytes[i - 1] == 0 || bytes[i - 1] >= (cuuint64_t)1 << 40)) return false;
    }
    return encoder(map, half ? CU_TENSOR_MAP_DATA_TYPE_FLOAT16 : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16,
                   (cuuint32_t)rank, const_cast<void*>(data), dims, bytes, boxes, ones,
                   CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
                   CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                   CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

template <typename T, int DP>
cudaError_t attend(ChunkArgs a, const w4a16_cache_shape& cache, cudaStream_t stream,
                   const DeviceCtx& ctx) {
    using S = Shape<DP>;
    static std::once_flag once[64];
    static cudaError_t set[64];
    int device = 0;
    cudaError_t e = cudaGetDevice(&device);
    if (e != cudaSuccess) return e;
    std::call_once(once[device], [&]() {
        set[device] = cudaFuncSetAttribute(chunk_kernel<T, DP>,
                                           cudaFuncAttributeMaxDynamicSharedMemorySize, S::kSmem);
    });
    if (set[device] != cudaSuccess) return set[device];
    constexpr bool kHalf = std::is_same<T, __half>::value;
    alignas(64) CUtensorMap maps[3] = {};
    if (a.group.value <= kQueryTile) {
        const int64_t sizes[3] = {a.c.head_dim, a.q_heads, a.tokens}, strides[3] = {1, a.q_head, a.q_row};
        const uint32_t box[3] = {64, (uint32_t)a.group.value, (uint32_t)(a.tile_rows / a.group.value)};
        a.q_map = encode(&maps[0], kHalf, a.q, 3, sizes, strides, box);
    }
    // boxes of 8 to 32 (16) rows: whole swizzled groups of eight, within a page and a warp's rows
    uint32_t box_rows = S::kStep / kCopyWarps;
    while (cache.page_size % box_rows) box_rows /= 2;
    if (box_rows >= 8) {
        const int64_t sizes[4] = {a.c.head_dim, cache.page_size, a.c.kv_heads, a.c.pages};
        const int64_t strides[4] = {1, a.c.slot_stride, a.c.head_stride, a.c.page_stride};
        const uint32_t box[4] = {64, box_rows, 1, 1};
        if (encode(&maps[1], kHalf, a.k_pool, 4, sizes, strides, box) &&
            encode(&maps[2], kHalf, a.v_pool, 4, sizes, strides, box))
            a.box_rows = (int)box_rows;
    }
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cudaLaunchConfig_t cfg = {};
    cfg.stream = stream;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    cfg.gridDim = dim3(1);
    cfg.blockDim = dim3(kPlanThreads);
    if ((e = cudaLaunchKernelEx(&cfg, plan_kernel, a, Divisor(S::kTiles * a.tile_rows),
                                S::kStep == 128 ? 7 : 6)) != cudaSuccess) return e;
    cfg.gridDim = dim3((unsigned)ctx.num_sms);
    cfg.blockDim = dim3(kThreads);
    cfg.dynamicSmemBytes = S::kSmem;
    if ((e = cudaLaunchKernelEx(&cfg, chunk_kernel<T, DP>, maps[0], maps[1], maps[2], a)) != cudaSuccess)
        return e;
    if (a.most_parts == 0) return cudaSuccess;
    cfg.gridDim = dim3((unsigned)(16 * ctx.num_sms));
    cfg.blockDim = dim3(kJoinThreads);
    cfg.dynamicSmemBytes = 0;
    return cudaLaunchKernelEx(&cfg, join_kernel<T, DP>, a);
}

template <typename T>
cudaError_t attend(const ChunkArgs& a, const w4a16_cache_shape& cache, cudaStream_t stream,
                   const DeviceCtx& ctx) {
    switch (padded_dim(a.c.head_dim)) {
        case 64: return attend<T, 64>(a, cache, stream, ctx);
        case 128: return attend<T, 128>(a, cache, stream, ctx);
        default: return attend<T, 256>(a, cache, stream, ctx);
    }
}

}  // namespace

int64_t paged_chunk_workspace(const w4a16_cache_shape& cache, int64_t q_heads, int64_t tokens,
                              const DeviceCtx& ctx) {
    return plan_workspace(cache, q_heads, tokens, ctx).bytes;
}

cudaError_t launch_paged_chunk_attention(const void* q, const void* k_pool, const void* v_pool,
                                         const int32_t* tables, const int32_t* lengths,
                                         const int32_t* offsets, void* out, float* lse,
                                         void* workspace, const w4a16_cache_shape& cache,
                                         const w4a16_query_shape& query, int64_t tokens,
                                         cudaStream_t stream, const DeviceCtx& ctx) {
    ChunkArgs a;
    a.q = static_cast<const uint16_t*>(q);
    a.k_pool = static_cast<const uint16_t*>(k_pool);
    a.v_pool = static_cast<const uint16_t*>(v_pool);
    a.tables = tables;
    a.lengths = lengths;
    a.offsets = offsets;
    a.out = static_cast<uint16_t*>(out);
    a.lse = lse;
    const Workspace w = plan_workspace(cache, query.q_heads, tokens, ctx);
    char* base = static_cast<char*>(workspace);
    a.plan = reinterpret_cast<Plan*>(base);
    a.entries = reinterpret_cast<Entry*>(base + w.entries);
    a.joints = reinterpret_cast<Joint*>(base + w.joints);
    a.slots = reinterpret_cast<Slot*>(base + w.slots);
    a.partial = reinterpret_cast<float*>(base + w.partial);
    a.partial_ml = reinterpret_cast<float2*>(base + w.ml);
    a.slot_count = w.slot_count;
    a.most_parts = w.most_parts;
    a.tokens = tokens;
    a.q_row = query.q_row_stride;
    a.q_head = query.q_head_stride;
    a.out_row = query.out_row_stride;
    a.out_head = query.out_head_stride;
    a.q_heads = (int)query.q_heads;
    a.sms = ctx.num_sms;
    // (not 0, which would make NaN of the -infinity of a position that does not count)
    a.scale_log2 = std::max((float)(std::abs(query.scale) * 1.4426950408889634), 0x1p-126f);
    a.negative = query.scale < 0;
    a.status = ctx.status;
    a.timeout_ns = ctx.timeout_ns;
    a.c = cache_of(cache);
    a.group = Divisor(query.q_heads / cache.kv_heads);
    a.tile_rows = tile_rows_of(a.group.value);
    a.q_map = a.box_rows = 0;
    return cache.type == W4A16_BF16 ? attend<__nv_bfloat16>(a, cache, stream, ctx)
                                    : attend<__half>(a, cache, stream, ctx);
}

}  // namespace w4a16
