// pages.cu -- the books of a paged cache: freeing, extending, forking and
// compacting rows, and the page copies these need.
//
// The books are small (a few int32 per page and per row) and every decision
// in them is a prefix sum: the k-th free page in ascending order, the pages
// wanted before request i.  One thread-block cluster does them: its barrier is
// cheaper than a second launch, and its shared memory carries the sums.  What
// moves whole pages runs over all SMs in a second launch that reads the list
// of copies from the workspace, so nothing waits for the host.  Page copies are
// bound by HBM: on one GB300 (6790 GB/s copied) 473 pages of 64 planes of 32 KB
// move in 294 us (6740 GB/s), 250 are copied for branches, with the books and
// the freeing of as many rows, in 152 us (6900 GB/s); four branches take 9.8 us,
// the compaction of 64 pages 11.5, of which their 16 and 54 MB are 2.5 and 8.
// With the books in place both have a plan in a launch of its own: 13.1 us, and
// 11.8 for the compaction of a pool in L2 (8.3 apart).  A fork in place goes
// through the pieces of children that copy nothing as well: 256 children of a
// parent that ends on a page's edge take 37 us.  Making 16 rows longer takes 6.4
// us in 640 pages and 9.7 in 40000, 1024 rows 11.5; copying 250 listed pages of
// 64 planes of 32 KB 156 us (6710 GB/s).
#include <algorithm>

#include "common.cuh"
#include "kernels.h"

namespace w4a16 {
namespace {

constexpr int kBookThreads = 1024;
constexpr int kBookWarps = kBookThreads / 32;
constexpr int kPagesPerLane = 16;                          // pages a lane looks at per sweep
constexpr int kPagesPerWarp = 32 * kPagesPerLane;          // consecutive ones of a warp

__device__ __forceinline__ uint32_t cluster_size() {
    uint32_t n;
    asm volatile("mov.u32 %0, %%cluster_nctaid.x;" : "=r"(n));
    return n;
}

__device__ __forceinline__ int ld_cluster_s32(uint32_t addr) {
    int v;
    asm volatile("ld.shared::cluster.s32 %0, [%1];" : "=r"(v) : "r"(addr) : "memory");
    return v;
}

// Every thread of the cluster; orders global and shared memory within it.
__device__ __forceinline__ void books_sync(uint32_t ctas) {
    if (ctas == 1)
        __syncthreads();
    else
        cluster_sync_all();
}

struct ScanShared {
    int warp_total[kBookWarps];
    int cta_total;
};

// Sum of `count` (the same in all lanes of a warp) over the warps before this
// one, in the order of (CTA rank, warp); *total: over all warps of the cluster.
__device__ int scan_warps(int count, ScanShared& sh, uint32_t rank, uint32_t ctas, int* total) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    if (lane == 0) sh.warp_total[warp] = count;
    __syncthreads();
    int v = sh.warp_total[lane];
#pragma unroll
    for (int d = 1; d < 32; d *= 2) {
        const int o = __shfl_up_sync(~0u, v, d);
        if (lane >= d) v += o;
    }
    int before = __shfl_sync(~0u, v, warp) - count;
    int sum = __shfl_sync(~0u, v, 31);
    if (ctas > 1) {
        if (threadIdx.x == 0) sh.cta_total = sum;
        cluster_sync_all();
        int t = lane < (int)ctas ? ld_cluster_s32(map_to_cta(smem_u32(&sh.cta_total), lane)) : 0;
        int lower = lane < (int)rank ? t : 0;
#pragma unroll
        for (int d = 16; d > 0; d /= 2) {
            t += __shfl_xor_sync(~0u, t, d);
            lower += __shfl_xor_sync(~0u, lower, d);
        }
        before += lower;
        sum = t;
    }
    books_sync(ctas);  // the totals may be overwritten by the next scan
    *total = sum;
    return before;
}

// Calls visit(page, ordinal, is_member) for every page in [0, pages), ordinal
// being the number of members (pages with in(refs[page])) before it; returns
// the number of members.  Called by all threads of the cluster.
template <typename In, typename Visit>
__device__ int sweep_pages(const int32_t* refs, int64_t pages, ScanShared& sh, uint32_t rank,
                           uint32_t ctas, In in, Visit visit) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int64_t sweep = (int64_t)ctas * kBookWarps * kPagesPerWarp;
    int carry = 0;
    for (int64_t base = 0; base < pages; base += sweep) {
        const int64_t first = base + ((int64_t)rank * kBookWarps + warp) * kPagesPerWarp;
        uint32_t mask[kPagesPerLane];
        int count = 0;
#pragma unroll
        for (int k = 0; k < kPagesPerLane; ++k) {
            const int64_t p = first + 32 * k + lane;
            mask[k] = __ballot_sync(~0u, p < pages && in(refs[p < pages ? p : 0]));
            count += __popc(mask[k]);
        }
        int total;
        int at = carry + scan_warps(count, sh, rank, ctas, &total);
        carry += total;
#pragma unroll
        for (int k = 0; k < kPagesPerLane; ++k) {
            const int64_t p = first + 32 * k + lane;
            const int mine = at + __popc(mask[k] & ((1u << lane) - 1));
            if (p < pages) visit(p, mine, (mask[k] >> lane) & 1u);
            at += __popc(mask[k]);
        }
    }
    return carry;
}

struct Books {
    const int32_t *refs_in, *tables_in, *lengths_in;
    int32_t *refs_out, *tables_out, *lengths_out;
    int64_t pages, rows, width, in_stride, out_stride, page_size;
};

// The `in` books into the `out` ones where these are other tensors.
__device__ void copy_books(const Books& b, int64_t thread, int64_t threads) {
    if (b.refs_in != b.refs_out)
        for (int64_t p = thread; p < b.pages; p += threads) b.refs_out[p] = b.refs_in[p];
    if (b.lengths_in != b.lengths_out)
        for (int64_t r = thread; r < b.rows; r += threads) b.lengths_out[r] = b.lengths_in[r];
    if (b.tables_in != b.tables_out)
        for (int64_t r = thread / 32; r < b.rows; r += threads / 32)
            for (int64_t j = thread % 32; j < b.width; j += 32)
                b.tables_out[r * b.out_stride + j] = b.tables_in[r * b.in_stride + j];
}

__global__ void __launch_bounds__(kBookThreads) free_kernel(Books b, const int32_t* listed,
                                                            int64_t count) {
    const uint32_t ctas = cluster_size();
    const int64_t threads = (int64_t)ctas * kBookThreads;
    const int64_t thread = (int64_t)cluster_cta_rank() * kBookThreads + threadIdx.x;
    grid_dependency_wait();
    grid_launch_dependents();
    copy_books(b, thread, threads);
    books_sync(ctas);
    for (int64_t i = thread / 32; i < count; i += threads / 32) {
        const int64_t r = listed[i];
        if (r < 0 || r >= b.rows) continue;
        int32_t* row = b.tables_out + r * b.out_stride;
        for (int64_t j = thread % 32; j < b.width; j += 32) {
            if (row[j] == -1) continue;
            // the exchange gives each page back once, however often its row is listed
            const int32_t p = atomicExch(&row[j], -1);
            if (p >= 0 && p < b.pages) atomicSub(&b.refs_out[p], 1);
        }
        if (thread % 32 == 0) b.lengths_out[r] = 0;
    }
}

// Workspace of extend, fork and compact: one int32 array after another.
struct Space {
    int32_t* claim;  // [rows]    first request that names the row
    int32_t* order;  // [count]   first of the request's pages in `free`, -1: refused
    int32_t* from;   // [count]   fork: page to copy, -1: none
    int32_t* to;     // [count]
    int32_t* length; // [count]   fork: the child's length
    int32_t* free;   // [pages]   free pages, ascending; compact: holes
    int32_t* high;   // [pages]   compact: held pages from the top
    int32_t* place;  // [pages]   compact: place of a page in `high`
    int32_t* copies; // [1]       page copies listed
    unsigned long long* next;  // [1]  the piece to copy next
};

Space split_space(void* workspace, int64_t rows, int64_t pages, int64_t count) {
    Space s;
    int32_t* w = static_cast<int32_t*>(workspace);
    s.copies = w;
    s.next = reinterpret_cast<unsigned long long*>(w + 2);
    w += 4;
    s.claim = w, w += rows;
    s.order = w, w += count;
    s.from = w, w += count;
    s.to = w, w += count;
    s.length = w, w += count;
    s.free = w, w += pages;
    s.high = w, w += pages;
    s.place = w;
    return s;
}

// Gives every in-range row of the list its first request's number.  `claim` has
// a place a row: s.claim, or shared memory where one CTA works on few rows (a
// round trip to L2 less for each of the steps that depend on one another).
constexpr int kSharedRows = 4096;
__device__ void claim_rows(int32_t* claim, const int32_t* listed, int64_t count, int64_t rows,
                           uint32_t ctas, int64_t thread, int64_t threads) {
    for (int64_t r = thread; r < rows; r += threads) claim[r] = 0x7FFFFFFF;
    books_sync(ctas);
    for (int64_t i = thread; i < count; i += threads) {
        const int32_t r = listed[i];
        if (r >= 0 && r < rows) atomicMin(&claim[r], (int)i);
    }
}

// One CTA: runs want(i) -> pages wanted (-1: refused) over the list in order and
// calls grant(i, first, wanted): first of the pages in the free list, or -1.
template <typename Want, typename Grant>
__device__ void serve_in_order(int64_t count, int64_t n_free, Want want, Grant grant) {
    __shared__ int64_t warp_total[kBookWarps];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    int64_t carry = 0;
    for (int64_t base = 0; base < count; base += kBookThreads) {
        const int64_t i = base + threadIdx.x;
        const int64_t w = i < count ? want(i) : -1;
        int64_t v = w > 0 ? w : 0;
#pragma unroll
        for (int d = 1; d < 32; d *= 2) {
            const int64_t o = __shfl_up_sync(~0u, v, d);
            if (lane >= d) v += o;
        }
        if (lane == 31) warp_total[warp] = v;
        __syncthreads();
        int64_t t = warp_total[lane];
#pragma unroll
        for (int d = 1; d < 32; d *= 2) {
            const int64_t o = __shfl_up_sync(~0u, t, d);
            if (lane >= d) t += o;
        }
        const int64_t own = __shfl_sync(~0u, t, warp) - __shfl_sync(~0u, v, 31);
        const int64_t upto = carry + own + v;
        if (i < count) grant(i, w >= 0 && upto <= n_free ? upto - w : -1, w);
        carry += __shfl_sync(~0u, t, 31);
        __syncthreads();
    }
}

__device__ __forceinline__ int64_t pages_of(int64_t length, int64_t page_size) {
    return (length + page_size - 1) / page_size;
}

__global__ void __launch_bounds__(kBookThreads)
    extend_kernel(Books b, const int32_t* listed, const int32_t* counts, int64_t count,
                  int32_t* done, Space s) {
    __shared__ ScanShared sh;
    __shared__ int32_t shared_claim[kSharedRows];
    const uint32_t ctas = cluster_size(), rank = cluster_cta_rank();
    const int64_t threads = (int64_t)ctas * kBookThreads;
    const int64_t thread = (int64_t)rank * kBookThreads + threadIdx.x;
    int32_t* const claim = ctas == 1 && b.rows <= kSharedRows ? shared_claim : s.claim;
    grid_dependency_wait();
    grid_launch_dependents();
    const int64_t n_free = sweep_pages(
        b.refs_in, b.pages, sh, rank, ctas, [](int32_t r) { return r <= 0; },
        [&](int64_t p, int k, bool member) {
            if (member) s.free[k] = (int32_t)p;
        });
    copy_books(b, thread, threads);
    claim_rows(claim, listed, count, b.rows, ctas, thread, threads);
    books_sync(ctas);
    if (rank == 0)
        serve_in_order(
            count, n_free,
            [&](int64_t i) -> int64_t {
                const int64_t r = listed[i], more = counts[i];
                if (r < 0 || r >= b.rows || claim[r] != i || more < 0) return -1;
                const int64_t n = max(b.lengths_out[r], 0);
                if (n + more > b.width * b.page_size) return -1;
                return pages_of(n + more, b.page_size) - pages_of(n, b.page_size);
            },
            [&](int64_t i, int64_t first, int64_t) {
                s.order[i] = (int32_t)first;
                done[i] = first >= 0;
                if (first >= 0)
                    b.lengths_out[listed[i]] = max(b.lengths_out[listed[i]], 0) + counts[i];
            });
    books_sync(ctas);
    for (int64_t i = thread / 32; i < count; i += threads / 32) {
        const int64_t first = s.order[i];
        if (first < 0) continue;
        const int64_t r = listed[i], n = b.lengths_out[r];
        const int64_t had = pages_of(n - counts[i], b.page_size), has = pages_of(n, b.page_size);
        for (int64_t j = had + thread % 32; j < has; j += 32) {
            const int32_t p = s.free[first + j - had];
            b.tables_out[r * b.out_stride + j] = p;
            b.refs_out[p] = 1;
        }
    }
}

// What request i of a fork reads of the books.
struct ForkRequest {
    int64_t from = -1, to = -1;
    int32_t length = 0, child_length = -1, last = -1;  // last: the parent's partly filled page

    __device__ void read(const Books& b, const int32_t* parents, const int32_t* children, int64_t i) {
        from = parents[i], to = children[i];
        if (from < 0 || from >= b.rows || to < 0 || to >= b.rows) return;
        child_length = b.lengths_in[to];
        length = (int32_t)min((int64_t)max(b.lengths_in[from], 0), b.width * b.page_size);
        if (length % b.page_size)
            last = b.tables_in[from * b.in_stride + length / b.page_size];
    }
};

// What forking decides; the tables and the pages follow in fork_apply_kernel.
__global__ void __launch_bounds__(kBookThreads)
    fork_plan_kernel(Books b, const int32_t* parents, const int32_t* children, int64_t count,
                     int32_t* done, Space s) {
    __shared__ ScanShared sh;
    __shared__ int32_t shared_claim[kSharedRows];
    const uint32_t ctas = cluster_size(), rank = cluster_cta_rank();
    const int64_t threads = (int64_t)ctas * kBookThreads;
    const int64_t thread = (int64_t)rank * kBookThreads + threadIdx.x;
    int32_t* const claim = ctas == 1 && b.rows <= kSharedRows ? shared_claim : s.claim;
    grid_dependency_wait();
    grid_launch_dependents();
    ForkRequest early;  // of request threadIdx.x: three reads in a row, on their way with the sweep's
    if (rank == 0 && threadIdx.x < count) early.read(b, parents, children, threadIdx.x);
    const int64_t n_free = sweep_pages(
        b.refs_in, b.pages, sh, rank, ctas, [](int32_t r) { return r <= 0; },
        [&](int64_t p, int k, bool member) {
            if (member && k < count) s.free[k] = (int32_t)p;  // one page a child at most
            if (b.refs_in != b.refs_out) b.refs_out[p] = b.refs_in[p];
        });
    claim_rows(claim, children, count, b.rows, ctas, thread, threads);
    books_sync(ctas);
    if (rank == 0)
        serve_in_order(
            count, n_free,
            [&](int64_t i) -> int64_t {
                ForkRequest q;  // a new one: reading leaves what it does not find as it was
                if (i < kBookThreads)
                    q = early;
                else
                    q.read(b, parents, children, i);
                s.from[i] = s.to[i] = -1;
                s.length[i] = q.length;
                if (q.child_length != 0 || claim[q.to] != i) return -1;
                if (q.length % b.page_size == 0) return 0;
                if (q.last < 0 || q.last >= b.pages) return -1;
                s.from[i] = q.last;
                return 1;
            },
            [&](int64_t i, int64_t first, int64_t wanted) {
                s.order[i] = (int32_t)first;
                done[i] = first >= 0;
                if (first >= 0 && wanted > 0) {
                    s.to[i] = s.free[first];
                    b.refs_out[s.free[first]] = 1;
                }
            });
    if (rank == 0 && threadIdx.x == 0) *s.next = 0;
    if (claim != s.claim)
        for (int64_t r = thread; r < b.rows; r += threads) s.claim[r] = claim[r];
}

// Page copies, in pieces of 16 KB.  Pieces are handed out as blocks become
// free: shared out beforehand, the blocks that sit further from their pages'
// memory end last (992 MB in and out: 321 us, handed out 292 us, 6.8 TB/s).
constexpr int kCopyThreads = 256;
constexpr int kCopyUnroll = 4;
constexpr int kCopyBlocksPerSm = 6;
constexpr int64_t kPiece = (int64_t)kCopyThreads * kCopyUnroll * 16;

struct Pool {
    char* base;
    int64_t planes, plane_stride, page_stride, page_bytes, pages;

    __device__ int64_t pieces() const { return (page_bytes + kPiece - 1) / kPiece; }
};

// Piece `unit` of the copies from(i) -> to(i).
template <typename From, typename To>
__device__ __forceinline__ void copy_piece(const Pool& pool, int64_t unit, From from, To to) {
    const int64_t pieces = pool.pieces();
    const int64_t piece = unit % pieces, plane = unit / pieces % pool.planes;
    const int64_t i = unit / pieces / pool.planes;
    const int64_t src = from(i), dst = to(i);
    if (src < 0 || src >= pool.pages || dst < 0 || dst >= pool.pages) return;
    const char* a = pool.base + plane * pool.plane_stride + src * pool.page_stride;
    char* z = pool.base + plane * pool.plane_stride + dst * pool.page_stride;
    uint4 v[kCopyUnroll];
#pragma unroll
    for (int k = 0; k < kCopyUnroll; ++k) {
        const int64_t at = piece * kPiece + (k * kCopyThreads + threadIdx.x) * 16;
        if (at < pool.page_bytes) v[k] = *reinterpret_cast<const uint4*>(a + at);
    }
#pragma unroll
    for (int k = 0; k < kCopyUnroll; ++k) {
        const int64_t at = piece * kPiece + (k * kCopyThreads + threadIdx.x) * 16;
        if (at < pool.page_bytes) *reinterpret_cast<uint4*>(z + at) = v[k];
    }
}

// All pieces of `copies` copies; *next is 0 at first.
template <typename From, typename To>
__device__ void copy_pages(const Pool& pool, int64_t copies, unsigned long long* next, From from,
                           To to) {
    __shared__ unsigned long long turn[2];  // this piece, and the one asked for while it is copied
    const unsigned long long units = copies * pool.planes * pool.pieces();
    if (threadIdx.x == 0) turn[0] = units ? atomicAdd(next, 1ull) : 0;
    __syncthreads();
    int which = 0;
    for (unsigned long long u = turn[0]; u < units; u = turn[which]) {
        which ^= 1;
        if (threadIdx.x == 0) turn[which] = atomicAdd(next, 1ull);
        copy_piece(pool, (int64_t)u, from, to);
        __syncthreads();
    }
}

__global__ void __launch_bounds__(kCopyThreads)
    fork_apply_kernel(Books b, const int32_t* parents, const int32_t* children, int64_t count,
                      Space s, Pool pool) {
    grid_dependency_wait();
    const int64_t thread = (int64_t)blockIdx.x * kCopyThreads + threadIdx.x;
    const int64_t threads = (int64_t)gridDim.x * kCopyThreads;
    const int lane = threadIdx.x & 31;
    for (int64_t r = thread / 32; r < b.rows; r += threads / 32) {
        const int32_t i = s.claim[r];
        const bool forked = i < count && s.order[i] >= 0;
        const int64_t from = forked ? parents[i] : r;
        if (!forked && b.tables_in == b.tables_out && b.lengths_in == b.lengths_out) continue;
        const int32_t* in = b.tables_in + from * b.in_stride;
        int32_t* out = b.tables_out + r * b.out_stride;
        if (!forked) {
            if (in != out)
                for (int64_t j = lane; j < b.width; j += 32) out[j] = in[j];
            if (lane == 0) b.lengths_out[r] = b.lengths_in[r];
            continue;
        }
        // not from the books: where `out` is `in`, the parent may be a child written just now
        // (it was empty then, so none of its page numbers are read here)
        const int64_t n = s.length[i];
        const int64_t full = n / b.page_size;
        const int32_t last = s.to[i];
        for (int64_t j = lane; j < b.width; j += 32) {
            int32_t p = -1;
            if (j < full) {
                p = in[j];
                if (p >= 0 && p < b.pages) atomicAdd(&b.refs_out[p], 1);
            } else if (j == full) {
                p = last;
            }
            out[j] = p;
        }
        if (lane == 0) b.lengths_out[r] = (int32_t)n;
    }
    copy_pages(pool, count, s.next, [&](int64_t i) { return s.from[i]; },
               [&](int64_t i) { return s.to[i]; });
}

// The holes below the number of held pages, ascending, and the held pages from the top.
__global__ void __launch_bounds__(kBookThreads)
    compact_plan_kernel(Books b, int32_t* used, Space s) {
    __shared__ ScanShared sh;
    const uint32_t ctas = cluster_size(), rank = cluster_cta_rank();
    const auto held = [](int32_t r) { return r > 0; };
    grid_dependency_wait();
    grid_launch_dependents();
    int n = 0, unused;
    {
        const int64_t threads = (int64_t)ctas * kBookThreads;
        for (int64_t p = (int64_t)rank * kBookThreads + threadIdx.x; p < b.pages; p += threads)
            n += held(b.refs_in[p]);
#pragma unroll
        for (int d = 16; d > 0; d /= 2) n += __shfl_xor_sync(~0u, n, d);
        (void)scan_warps(n, sh, rank, ctas, &unused);
        n = unused;
    }
    // page p is the k-th held one: the k before it leave p - k holes below it, n - 1 - k come after
    sweep_pages(b.refs_in, b.pages, sh, rank, ctas, held, [&](int64_t p, int k, bool member) {
        if (p < n && !member) s.free[p - k] = (int32_t)p;
        if (p >= n && member) {
            s.high[n - 1 - k] = (int32_t)p;
            s.place[p] = n - 1 - k;
        }
        if (p == n - 1) *s.copies = (int32_t)(p + 1 - k - (member ? 1 : 0));
    });
    if (rank == 0 && threadIdx.x == 0) {
        used[0] = n;
        *s.next = 0;
        if (n == 0) *s.copies = 0;
    }
}

// The books of a compaction: pair i moves page high(copies - 1 - i) to page hole(i); place(p) is
// the place of a moving page p in `high`, anything for another page.
template <typename High, typename Hole, typename Place>
__device__ void compact_books(const Books& b, int64_t n, int64_t copies, High high, Hole hole,
                              Place place) {
    const int64_t thread = (int64_t)blockIdx.x * kCopyThreads + threadIdx.x;
    const int64_t threads = (int64_t)gridDim.x * kCopyThreads;
    // a pair's two counts belong to one thread, so `out` may be `in`
    for (int64_t i = thread; i < copies; i += threads) {
        const int32_t src = high(copies - 1 - i), dst = hole(i);
        const int32_t held = b.refs_in[src];
        b.refs_out[dst] = held;
        b.refs_out[src] = 0;
    }
    if (b.refs_in != b.refs_out)
        for (int64_t p = thread; p < b.pages; p += threads)
            if ((b.refs_in[p] > 0) == (p < n)) b.refs_out[p] = b.refs_in[p];
    for (int64_t r = thread / 32; r < b.rows; r += threads / 32)
        for (int64_t j = thread % 32; j < b.width; j += 32) {
            int32_t p = b.tables_in[r * b.in_stride + j];
            // a number n or above that no count holds is left as it is
            if (p >= n && p < b.pages) {
                const int32_t k = place(p);
                if (k >= 0 && k < copies && high(k) == p) p = hole(copies - 1 - k);
            }
            b.tables_out[r * b.out_stride + j] = p;
        }
}

__global__ void __launch_bounds__(kCopyThreads)
    compact_apply_kernel(Books b, const int32_t* used, Space s, Pool pool) {
    grid_dependency_wait();
    const int64_t copies = *s.copies;
    compact_books(b, used[0], copies, [&](int64_t k) { return s.high[k]; },
                  [&](int64_t i) { return s.free[i]; }, [&](int64_t p) { return s.place[p]; });
    copy_pages(pool, copies, s.next, [&](int64_t i) { return s.high[copies - 1 - i]; },
               [&](int64_t i) { return s.free[i]; });
}

// ---------------------------------------------------------------------------
// One launch for small pools.  Every block reads the counts of all pages and
// comes to the same lists, in shared memory; so nothing has to wait for a plan,
// and there is no workspace.  Only where the books are written apart from the
// ones read (another block may still be reading), and where the copies are few
// enough to be shared out beforehand.
// ---------------------------------------------------------------------------
constexpr int kAloneWarps = kCopyThreads / 32;
constexpr int kAlonePages = kAloneWarps * kPagesPerWarp;  // a sweep of one block
constexpr int kAloneRows = 16384, kAloneCount = kCopyThreads;
constexpr int64_t kAloneBytes = (int64_t)128 << 20;  // of copies

// sweep_pages by one block on its own, for up to kAlonePages pages.
template <typename In, typename Visit>
__device__ __forceinline__ int sweep_alone(const int32_t* refs, int64_t pages, int (&total)[kAloneWarps],
                                           In in, Visit visit) {
    const int lane = threadIdx.x % 32, warp = threadIdx.x / 32;
    uint32_t mask[kPagesPerLane];
    int count = 0;
#pragma unroll
    for (int k = 0; k < kPagesPerLane; ++k) {
        const int p = warp * kPagesPerWarp + 32 * k + lane;
        mask[k] = __ballot_sync(~0u, p < pages && in(refs[p < pages ? p : 0]));
        count += __popc(mask[k]);
    }
    if (lane == 0) total[warp] = count;
    __syncthreads();
    int at = 0, sum = 0;
#pragma unroll
    for (int w = 0; w < kAloneWarps; ++w) {
        if (w < warp) at += total[w];
        sum += total[w];
    }
#pragma unroll
    for (int k = 0; k < kPagesPerLane; ++k) {
        const int p = warp * kPagesPerWarp + 32 * k + lane;
        if (p < pages) visit(p, at + __popc(mask[k] & ((1u << lane) - 1)), (mask[k] >> lane) & 1u, sum);
        at += __popc(mask[k]);
    }
    return sum;
}

__global__ void __launch_bounds__(kCopyThreads)
    compact_alone_kernel(Books b, int32_t* used, Pool pool) {
    __shared__ uint16_t hole[kAlonePages / 2], high[kAlonePages / 2], place[kAlonePages];
    __shared__ int total[kAloneWarps], moves;
    if (threadIdx.x == 0) moves = 0;
    grid_dependency_wait();
    grid_launch_dependents();
    const int n = sweep_alone(
        b.refs_in, b.pages, total, [](int32_t r) { return r > 0; },
        [&](int p, int k, bool member, int n) {
            if (p < n && !member) hole[p - k] = (uint16_t)p;
            if (p >= n && member) {
                high[n - 1 - k] = (uint16_t)p;
                place[p] = (uint16_t)(n - 1 - k);
            }
            if (p == n - 1) moves = p + 1 - k - (member ? 1 : 0);
        });
    __syncthreads();
    const int copies = moves;
    if (blockIdx.x == 0 && threadIdx.x == 0) used[0] = n;
    compact_books(b, n, copies, [&](int64_t k) { return (int32_t)high[k]; },
                  [&](int64_t i) { return (int32_t)hole[i]; },
                  [&](int64_t p) { return (int32_t)place[p]; });
    const int64_t units = copies * pool.planes * pool.pieces();
    for (int64_t u = blockIdx.x; u < units; u += gridDim.x)
        copy_piece(pool, u, [&](int64_t i) { return (int64_t)high[copies - 1 - i]; },
                   [&](int64_t i) { return (int64_t)hole[i]; });
}

__global__ void __launch_bounds__(kCopyThreads)
    fork_alone_kernel(Books b, const int32_t* parents, const int32_t* children, int64_t count,
                      int32_t* done, Pool pool) {
    __shared__ int total[kAloneWarps], wanted_total[kAloneWarps];
    __shared__ uint16_t free[kAloneCount];
    __shared__ int32_t child[kAloneCount], parent[kAloneCount], length[kAloneCount];
    __shared__ int32_t from[kAloneCount], to[kAloneCount];
    __shared__ uint32_t forked[kAloneRows / 32];  // a bit a row
    const int tid = threadIdx.x, lane = tid % 32, warp = tid / 32;
    for (int i = tid; i < kAloneRows / 32; i += kCopyThreads) forked[i] = 0;
    grid_dependency_wait();
    grid_launch_dependents();
    ForkRequest q;  // of request tid
    if (tid < count) q.read(b, parents, children, tid);
    child[tid] = q.to >= 0 && q.to < b.rows ? (int32_t)q.to : -1;
    const int n_free = sweep_alone(
        b.refs_in, b.pages, total, [](int32_t r) { return r <= 0; },
        [&](int p, int k, bool member, int) {
            if (member && k < kAloneCount) free[k] = (uint16_t)p;
        });
    int want = -1;
    if (q.child_length == 0) {
        want = q.length % b.page_size == 0 ? 0 : q.last >= 0 && q.last < b.pages ? 1 : -1;
        for (int j = 0; j < tid; ++j)
            if (child[j] == child[tid]) want = -1;  // listed before
    }
    const uint32_t mask = __ballot_sync(~0u, want > 0);
    if (lane == 0) wanted_total[warp] = __popc(mask);
    __syncthreads();
    int upto = __popc(mask & ((2u << lane) - 1));  // pages wanted up to this request
#pragma unroll
    for (int w = 0; w < kAloneWarps; ++w)
        if (w < warp) upto += wanted_total[w];
    const bool granted = want >= 0 && upto <= n_free;
    from[tid] = granted && want > 0 ? q.last : -1;
    to[tid] = granted && want > 0 ? free[upto - 1] : -1;
    parent[tid] = granted ? (int32_t)q.from : -1;
    length[tid] = q.length;
    if (granted) atomicOr(&forked[q.to / 32], 1u << (q.to % 32));
    if (blockIdx.x == 0 && tid < count) done[tid] = granted;
    __syncthreads();

    // the first block has the counts; the rows go round
    if (blockIdx.x == 0) {
        for (int p = tid; p < b.pages; p += kCopyThreads) b.refs_out[p] = b.refs_in[p];
        __syncthreads();
        if (to[tid] >= 0) b.refs_out[to[tid]] = 1;
    }
    const int warps = gridDim.x * kAloneWarps, my_warp = blockIdx.x * kAloneWarps + warp;
    for (int r = my_warp; r < b.rows; r += warps) {
        if (forked[r / 32] >> (r % 32) & 1) continue;
        for (int64_t j = lane; j < b.width; j += 32)
            b.tables_out[r * b.out_stride + j] = b.tables_in[r * b.in_stride + j];
        if (lane == 0) b.lengths_out[r] = b.lengths_in[r];
    }
    const int first = blockIdx.x == 0 ? warp : my_warp, stride = blockIdx.x == 0 ? kAloneWarps : warps;
    for (int i = first; i < count; i += stride) {
        if (parent[i] < 0) continue;
        const int64_t full = length[i] / b.page_size;
        const bool mine = i % warps == my_warp;
        for (int64_t j = lane; j < b.width; j += 32) {
            const int32_t p = j < full    ? b.tables_in[parent[i] * b.in_stride + j]
                              : j == full ? to[i]
                                          : -1;
            if (blockIdx.x == 0 && j < full && p >= 0 && p < b.pages) atomicAdd(&b.refs_out[p], 1);
            if (mine) b.tables_out[child[i] * b.out_stride + j] = p;
        }
        if (mine && lane == 0) b.lengths_out[child[i]] = length[i];
    }
    const int64_t units = count * pool.planes * pool.pieces();
    for (int64_t u = blockIdx.x; u < units; u += gridDim.x)
        copy_piece(pool, u, [&](int64_t i) { return (int64_t)from[i]; },
                   [&](int64_t i) { return (int64_t)to[i]; });
}

__global__ void __launch_bounds__(kCopyThreads)
    copy_kernel(Pool pool, const int32_t* from, const int32_t* to, int64_t units) {
    grid_dependency_wait();
    grid_launch_dependents();
    for (int64_t u = blockIdx.x; u < units; u += gridDim.x)
        copy_piece(pool, u, [&](int64_t i) { return from[i]; }, [&](int64_t i) { return to[i]; });
}

// The listed rows' page numbers and lengths; those of a row out of range are none and 0.
constexpr int kRowPiece = 4 * kCopyThreads;
__global__ void __launch_bounds__(kCopyThreads)
    rows_kernel(Books b, const int32_t* listed, int64_t count) {
    grid_dependency_wait();
    grid_launch_dependents();
    const int64_t pieces = (b.width + kRowPiece - 1) / kRowPiece;
    for (int64_t u = blockIdx.x; u < count * pieces; u += gridDim.x) {
        const int64_t i = u / pieces, first = u % pieces * kRowPiece, r = listed[i];
        const bool there = r >= 0 && r < b.rows;
        for (int64_t j = first + threadIdx.x; j < min(first + kRowPiece, b.width); j += kCopyThreads)
            b.tables_out[i * b.width + j] = there ? b.tables_in[r * b.in_stride + j] : -1;
        if (first == 0 && threadIdx.x == 0 && b.lengths_out)
            b.lengths_out[i] = there ? b.lengths_in[r] : 0;
    }
}

// The cluster of a books kernel: one CTA for up to a sweep of pages and as many
// page numbers in rows to read or copy, else eight.
template <typename... P, typename... A>
cudaError_t launch_books(void (*kernel)(P...), int64_t numbers, cudaStream_t stream, A... args) {
    const unsigned ctas = numbers <= kBookWarps * kPagesPerWarp ? 1 : 8;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(ctas);
    cfg.blockDim = dim3(kBookThreads);
    cfg.stream = stream;
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.x = ctas;
    attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 2;
    return cudaLaunchKernelEx(&cfg, kernel, P(args)...);
}

template <typename... P, typename... A>
cudaError_t launch_apply(void (*kernel)(P...), unsigned ctas, cudaStream_t stream, A... args) {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(ctas);
    cfg.blockDim = dim3(kCopyThreads);
    cfg.stream = stream;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, kernel, P(args)...);
}

Books books_of(const PageBooks& b) {
    return {b.refs_in,     b.tables_in,  b.lengths_in, b.refs_out,        b.tables_out,
            b.lengths_out, b.shape.pages, b.shape.rows, b.shape.width,     b.shape.in_stride,
            b.shape.out_stride, b.shape.page_size};
}

// Page numbers that a books kernel copies from one table to another.
int64_t copied(const PageBooks& b) {
    return b.tables_in == b.tables_out ? 0 : b.shape.rows * b.shape.width;
}

Pool pool_of(void* pool, const w4a16_pool_shape& s, int64_t pages) {
    return {static_cast<char*>(pool), s.planes, s.plane_stride, s.page_stride, s.page_bytes, pages};
}

unsigned copy_ctas(const DeviceCtx& ctx) { return (unsigned)(kCopyBlocksPerSm * ctx.num_sms); }

// Whether a fork or compaction of at most `copies` pages goes in one launch.
bool alone(const w4a16_books_shape& b, const w4a16_pool_shape& pool, int64_t copies, bool apart) {
    return apart && b.pages <= kAlonePages && b.rows <= kAloneRows && b.rows * b.width <= 1 << 20 &&
           copies * pool.planes <= kAloneBytes / pool.page_bytes;
}
bool fork_alone(const w4a16_books_shape& b, const w4a16_pool_shape& pool, int64_t count, bool apart) {
    return count <= kAloneCount && count * b.width <= 1 << 14 && alone(b, pool, count, apart);
}
bool compact_alone(const w4a16_books_shape& b, const w4a16_pool_shape& pool, bool apart) {
    return alone(b, pool, b.pages / 2, apart);
}

// Blocks for at most `copies` copies to share out.
unsigned alone_ctas(const w4a16_pool_shape& pool, int64_t copies, const DeviceCtx& ctx) {
    const int64_t units = copies * pool.planes * ((pool.page_bytes + kPiece - 1) / kPiece);
    return (unsigned)std::max<int64_t>(1, std::min<int64_t>(units, copy_ctas(ctx)));
}

}  // namespace

int64_t pages_fork_workspace(const w4a16_books_shape& b, const w4a16_pool_shape& pool,
                             int64_t count, bool apart) {
    return fork_alone(b, pool, count, apart) ? 0 : pages_workspace(b, count);
}

int64_t pages_compact_workspace(const w4a16_books_shape& b, const w4a16_pool_shape& pool,
                                bool apart) {
    return compact_alone(b, pool, apart) ? 0 : pages_workspace(b, 0);
}

int64_t pages_workspace(const w4a16_books_shape& b, int64_t count) {
    return 4 * (4 + b.rows + 4 * count + 3 * b.pages);
}

cudaError_t launch_pages_rows(const PageBooks& b, const int32_t* listed, int64_t count,
                              cudaStream_t stream) {
    if (count == 0) return cudaSuccess;
    const int64_t units = count * ((b.shape.width + kRowPiece - 1) / kRowPiece);
    return launch_apply(rows_kernel, (unsigned)std::min<int64_t>(units, 1 << 20), stream, books_of(b),
                        listed, count);
}

cudaError_t launch_pages_free(const PageBooks& b, const int32_t* listed, int64_t count,
                              cudaStream_t stream) {
    // a warp goes through a listed row, three round trips to L2 each: eight CTAs from a few rows on
    const int64_t rows = count <= 2 * kBookWarps ? 0 : (int64_t)1 << 40;
    return launch_books(free_kernel, std::max({b.shape.pages, copied(b), rows}), stream, books_of(b),
                        listed, count);
}

cudaError_t launch_pages_extend(const PageBooks& b, const int32_t* listed, const int32_t* counts,
                                int64_t count, int32_t* done, void* workspace,
                                cudaStream_t stream) {
    return launch_books(extend_kernel, std::max(b.shape.pages, copied(b)), stream, books_of(b),
                        listed, counts, count, done,
                        split_space(workspace, b.shape.rows, b.shape.pages, count));
}

cudaError_t launch_pages_fork(void* pool, const PageBooks& b, const int32_t* parents,
                              const int32_t* children, int64_t count, int32_t* done,
                              void* workspace, const w4a16_pool_shape& shape, cudaStream_t stream,
                              const DeviceCtx& ctx) {
    if (fork_alone(b.shape, shape, count,
                   b.refs_in != b.refs_out && b.tables_in != b.tables_out &&
                       b.lengths_in != b.lengths_out))
        return launch_apply(fork_alone_kernel, alone_ctas(shape, count, ctx), stream, books_of(b),
                            parents, children, count, done, pool_of(pool, shape, b.shape.pages));
    const Space s = split_space(workspace, b.shape.rows, b.shape.pages, count);
    cudaError_t e = launch_books(fork_plan_kernel, b.shape.pages, stream, books_of(b), parents,
                                 children, count, done, s);
    if (e != cudaSuccess) return e;
    return launch_apply(fork_apply_kernel, copy_ctas(ctx), stream, books_of(b), parents, children,
                        count, s, pool_of(pool, shape, b.shape.pages));
}

cudaError_t launch_pages_compact(void* pool, const PageBooks& b, int32_t* used, void* workspace,
                                 const w4a16_pool_shape& shape, cudaStream_t stream,
                                 const DeviceCtx& ctx) {
    if (compact_alone(b.shape, shape, b.refs_in != b.refs_out && b.tables_in != b.tables_out))
        return launch_apply(compact_alone_kernel, alone_ctas(shape, b.shape.pages / 2, ctx), stream,
                            books_of(b), used, pool_of(pool, shape, b.shape.pages));
    const Space s = split_space(workspace, b.shape.rows, b.shape.pages, 0);
    cudaError_t e = launch_books(compact_plan_kernel, b.shape.pages, stream, books_of(b), used, s);
    if (e != cudaSuccess) return e;
    return launch_apply(compact_apply_kernel, copy_ctas(ctx), stream, books_of(b),
                        (const int32_t*)used, s, pool_of(pool, shape, b.shape.pages));
}

cudaError_t launch_pages_copy(void* pool, const int32_t* from, const int32_t* to, int64_t count,
                              int64_t pages, const w4a16_pool_shape& shape,
                              cudaStream_t stream) {
    if (count == 0) return cudaSuccess;
    // a piece a block: the scheduler hands them out
    const int64_t units = count * shape.planes * ((shape.page_bytes + kPiece - 1) / kPiece);
    return launch_apply(copy_kernel, (unsigned)std::min<int64_t>(units, 1 << 30), stream,
                        pool_of(pool, shape, pages), from, to, units);
}

}  // namespace w4a16
