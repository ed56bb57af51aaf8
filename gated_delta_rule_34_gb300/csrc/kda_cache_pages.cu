// kda_cache_pages.cu -- pages of the 8-bit cache changing hands: copied, given to rows of the block table and taken
// back, shared by rows that fork, moved to the front of the pool.
//
// refs[p] counts the entries of block tables that hold page p; a page with none is free.  What is taken is always the
// lowest free page, in the order of what asks for it, so that the same call gives the same table:
//
//   the k-th entry that lacks a page gets the k-th page with refs == 0
//
// which is a prefix sum over the entries and one over the pages.  A call's work is small (a table of 400 rows x 1,024
// entries and the counts of 262,144 pages are 2.7 MB) and its steps follow one another, so what bounds it is the time
// that memory takes to answer, some times over.  One cluster of CTAs does all steps in one launch, its CTAs' sums handed over
// through distributed shared memory between hardware barriers (one CTA where there is little to look through).  Where
// the rows have many entries, these are walked by kernels of their own over the whole GPU and the cluster does the sums
// between them.
#include <climits>
#include <cstdint>

#include <cooperative_groups.h>

#include "kda_cache_internal.h"
#include "kda_chained.cuh"

namespace kda {
namespace {

namespace cg = cooperative_groups;

constexpr int kThreads = 1024;
constexpr int kWarps = kThreads / 32;
constexpr int kCluster = 8;
constexpr int kUnits = 8192;               // units of a CTA at most: their counts are in shared memory
constexpr int kEach = 8;                   // loads of a lane at once
constexpr int kSegment = 32 * kEach;       // entries of a unit, at least
constexpr int kBlock = 1024;               // pages whose marks a warp holds, 32 a lane
constexpr int kListed = 1024;              // rows up to which a CTA looks through a call's list in shared memory
constexpr int kRowThreads = 256;           // of the kernels that walk rows over the whole GPU

struct Shared {
    int warp_sum[kWarps];
    int slot[8];                           // of sums that the cluster's CTAs tell one another
    int units[kUnits];
    int32_t list[2][kListed];
};

// Counts and entries that other CTAs of the cluster have written: from L2.
__device__ __forceinline__ int read(const int32_t* p) { return __ldcg(p); }

struct Cluster {
    Shared& s;
    cg::cluster_group group = cg::this_cluster();
    int used = 0;

    __device__ __forceinline__ int rank() const { return (int)group.block_rank(); }
    __device__ __forceinline__ int size() const { return (int)group.num_blocks(); }
    // What was written before is seen after, by all threads of the cluster.
    __device__ __forceinline__ void meet() { group.sync(); }

    // Sum of all CTAs' values, and of those of lower rank (the same value in all threads of a CTA).
    __device__ __forceinline__ int2 sum(int value) {
        int* slot = &s.slot[used++];
        if (threadIdx.x == 0) *slot = value;
        meet();
        int before = 0, total = 0;
        for (int r = 0; r < size(); ++r) {
            const int v = *group.map_shared_rank(slot, r);
            before += r < rank() ? v : 0;
            total += v;
        }
        return make_int2(before, total);
    }

    // Of one value a warp: the sum over the warps before this one, and of all.
    __device__ __forceinline__ int2 scan_warps(int value) {
        const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
        __syncthreads();
        if (lane == 0) s.warp_sum[warp] = value;
        __syncthreads();
        int up = s.warp_sum[lane];
#pragma unroll
        for (int w = 1; w < 32; w <<= 1) {
            const int x = __shfl_up_sync(0xffffffffu, up, w);
            if (lane >= w) up += x;
        }
        return make_int2(__shfl_sync(0xffffffffu, up, warp) - value, __shfl_sync(0xffffffffu, up, 31));
    }
    // Of one value a thread: the sum over the threads before this one, and of all.
    __device__ __forceinline__ int2 scan(int value) {
        const int lane = threadIdx.x & 31;
        int up = value;
#pragma unroll
        for (int w = 1; w < 32; w <<= 1) {
            const int x = __shfl_up_sync(0xffffffffu, up, w);
            if (lane >= w) up += x;
        }
        const int2 warps = scan_warps(__shfl_sync(0xffffffffu, up, 31));
        return make_int2(warps.x + up - value, warps.y);
    }
};

// [0, n) in equal parts of whole multiples of `unit`, in order.
__device__ __forceinline__ int64_t part(int64_t n, int size, int rank, int unit = 1) {
    const int64_t each = ((n + size - 1) / size + unit - 1) / unit * unit, at = each * rank;
    return at < n ? at : n;
}

// A warp's pages [from, to), 1024 at a time: which of them have no holder, lane i the marks of 32 i .. 32 i + 31 (none past
// the end), eight loads at once.
__device__ __forceinline__ uint32_t free_marks(const int32_t* refs, int64_t from, int64_t to) {
    const int lane = threadIdx.x & 31;
    uint32_t marks = 0;
#pragma unroll 1
    for (int g = 0; g < 32; g += kEach) {
        int count[kEach];
#pragma unroll
        for (int x = 0; x < kEach; ++x) {
            const int64_t p = from + (g + x) * 32 + lane;
            count[x] = p < to ? read(refs + p) : 1;
        }
#pragma unroll
        for (int x = 0; x < kEach; ++x) {
            const uint32_t m = __ballot_sync(0xffffffffu, count[x] <= 0);
            if (lane == g + x) marks = m;
        }
    }
    return marks;
}
// Those of marks that lie before page `end`, the first of them being page `from`.
__device__ __forceinline__ uint32_t marks_before(uint32_t marks, int64_t from, int64_t end) {
    const int64_t left = end - (from + 32 * (threadIdx.x & 31));
    return left <= 0 ? 0u : left >= 32 ? marks : marks & ((1u << left) - 1u);
}
__device__ __forceinline__ int count_marks(uint32_t marks) { return __reduce_add_sync(0xffffffffu, __popc(marks)); }

// A warp's share of all pages.
struct Range {
    int64_t from, to;
};
__device__ __forceinline__ Range pages_of_warp(const Cluster& c, int64_t n_pages) {
    const int64_t p0 = part(n_pages, c.size(), c.rank(), 32 * kWarps), p1 = part(n_pages, c.size(), c.rank() + 1, 32 * kWarps);
    const int warp = threadIdx.x >> 5;
    return {p0 + part(p1 - p0, kWarps, warp, 32), p0 + part(p1 - p0, kWarps, warp + 1, 32)};
}

// The lowest `wanted` free pages, in order, to `list`; returns how many pages are free.  All threads of the cluster call
// it, after what changes refs, and meet before they read the list.
__device__ __forceinline__ int list_free(Cluster& c, const int32_t* refs, int64_t n_pages, int wanted, int32_t* list) {
    const int lane = threadIdx.x & 31;
    const Range r = pages_of_warp(c, n_pages);
    int mine = 0;
    uint32_t marks = 0;
    for (int64_t at = r.from; at < r.to; at += kBlock) {
        marks = free_marks(refs, at, r.to);
        mine += count_marks(marks);
    }
    const int2 of_cta = c.scan_warps(mine);
    const int2 all = c.sum(of_cta.y);
    int rank = all.x + of_cta.x;
    for (int64_t at = r.from; at < r.to && rank < wanted; at += kBlock) {
        if (r.to - r.from > kBlock) marks = free_marks(refs, at, r.to);   // (one block's are still there)
#pragma unroll 1
        for (int i = 0; i < 32; ++i) {
            const uint32_t m = __shfl_sync(0xffffffffu, marks, i);
            const int mark_rank = rank + __popc(m & ((1u << lane) - 1u));
            if ((m >> lane & 1u) && mark_rank < wanted) list[mark_rank] = (int32_t)(at + 32 * i + lane);
            rank += __popc(m);
            if (rank >= wanted) break;
        }
    }
    return all.y;
}

struct Pages {
    int32_t* refs;
    int32_t* table;
    int64_t n_pages;
    int n_rows, wide;
    int page_shift;
    int n;                                 // rows, or pairs of rows, that the call names
    int segment, segments;                 // a row's entries in units of that many
    int32_t* missing;                      // nullable
    int32_t* list;                         // the workspace: [n_pages],
    int32_t* first;                        // for long lists [n_rows],
    int32_t* units;                        // and, where rows are walked by kernels of their own, [kCluster kUnits], and
    int32_t* sums;                         // how many entries lack a page, and how many pages are free

    __device__ __forceinline__ bool held(int32_t e) const { return e >= 0 && e < n_pages; }
    __device__ __forceinline__ bool is_row(int r) const { return r >= 0 && r < n_rows; }
};

// Which of a call's rows count: the first of those that name the same one, and none that `bars` names.  Short lists are looked
// through in shared memory, a warp an entry; long ones leave their least index at the row, in the workspace.
struct Listed {
    const Pages& a;
    int32_t (*list)[kListed];
    const int32_t* rows;
    const int32_t* bars;                   // nullable

    // The threads of a CTA call it, and meet.
    __device__ __forceinline__ void to_shared() {
        if (a.n > kListed) return;
        for (int i = threadIdx.x; i < a.n; i += blockDim.x) {
            list[0][i] = rows[i];
            if (bars) list[1][i] = bars[i];
        }
    }
    // Long lists: t of `step` threads, first the one, then, when all have done so, the other.
    __device__ __forceinline__ void clear(int64_t t, int64_t step) {
        for (int64_t i = t; i < a.n; i += step) {
            if (a.is_row(rows[i])) a.first[rows[i]] = INT_MAX;
            if (bars && a.is_row(bars[i])) a.first[bars[i]] = INT_MAX;
        }
    }
    __device__ __forceinline__ void claim(int64_t t, int64_t step) {
        for (int64_t i = t; i < a.n; i += step) {
            if (a.is_row(rows[i])) atomicMin(a.first + rows[i], (int)i);
            if (bars && a.is_row(bars[i])) atomicMin(a.first + bars[i], -1);
        }
    }
    __device__ __forceinline__ void begin(Cluster& c) {
        const int64_t step = (int64_t)c.size() * kThreads, t = (int64_t)c.rank() * kThreads + threadIdx.x;
        to_shared();
        __syncthreads();
        if (a.n <= kListed) return;
        clear(t, step);
        c.meet();
        claim(t, step);
        c.meet();
    }
    // Whole warps; row = rows[i].
    __device__ __forceinline__ bool counts(int i, int row) const {
        if (!a.is_row(row)) return false;
        if (a.n > kListed) return read(a.first + row) == i;
        bool other = false;
        for (int j = threadIdx.x & 31; j < i; j += 32) other |= list[0][j] == row;
        if (bars)
            for (int j = threadIdx.x & 31; j < a.n; j += 32) other |= list[1][j] == row;
        return !__any_sync(0xffffffffu, other);
    }
};

// For lists that the kernels over the whole GPU cannot look through: the two halves of Listed::begin.
__global__ void __launch_bounds__(kRowThreads) clear_kernel(const Pages a, const int32_t* rows, const int32_t* bars) {
    after_the_kernel_before();
    Listed{a, nullptr, rows, bars}.clear((int64_t)blockIdx.x * kRowThreads + threadIdx.x, (int64_t)gridDim.x * kRowThreads);
}
__global__ void __launch_bounds__(kRowThreads) claim_kernel(const Pages a, const int32_t* rows, const int32_t* bars) {
    after_the_kernel_before();
    Listed{a, nullptr, rows, bars}.claim((int64_t)blockIdx.x * kRowThreads + threadIdx.x, (int64_t)gridDim.x * kRowThreads);
}

__device__ __forceinline__ int pages_for(int tokens, const Pages& a) {
    const int n = tokens > 0 ? ((tokens - 1) >> a.page_shift) + 1 : 0;
    return n < a.wide ? n : a.wide;
}

// Eight of a row's entries a lane: entries j + 32 x, -1 past j1.
__device__ __forceinline__ void load_entries(const int32_t* entries, int j, int j1, int32_t (&e)[kEach]) {
#pragma unroll
    for (int x = 0; x < kEach; ++x) e[x] = j + 32 * x < j1 ? entries[j + 32 * x] : -1;
}

// A unit of a row that counts: entries past its need go back; returns how many others lack a page.
__device__ __forceinline__ int release_unit(const Pages& a, int row, int need, int j0) {
    const int lane = threadIdx.x & 31, j1 = j0 + a.segment < a.wide ? j0 + a.segment : a.wide;
    int32_t* entries = a.table + (int64_t)row * a.wide;
    int lacks = 0;
    for (int j = j0 + lane; j < j1 + lane; j += kSegment) {
        int32_t e[kEach];
        load_entries(entries, j, j1, e);
        int before[kEach];
#pragma unroll
        for (int x = 0; x < kEach; ++x) {
            const int at = j + 32 * x;
            const bool gone = at < j1 && at >= need;
            // One holder less.  (A count that says none is left alone: the table did not match it.)
            before[x] = gone && a.held(e[x]) ? atomicSub(a.refs + e[x], 1) : 1;
            if (gone && e[x] != -1) entries[at] = -1;
            lacks += at < j1 && at < need && !a.held(e[x]);
        }
#pragma unroll
        for (int x = 0; x < kEach; ++x)
            if (before[x] <= 0) atomicAdd(a.refs + e[x], 1);
    }
    return __reduce_add_sync(0xffffffffu, lacks);
}
// Its entries that lack one get pages rank, rank + 1, ... of the free ones.
__device__ __forceinline__ void fill_unit(const Pages& a, int row, int need, int j0, int rank, int free) {
    const int lane = threadIdx.x & 31, j1 = j0 + a.segment < need ? j0 + a.segment : need;
    int32_t* entries = a.table + (int64_t)row * a.wide;
    for (int j = j0 + lane; j < j1 + lane; j += kSegment) {
        int32_t e[kEach], page[kEach];
        load_entries(entries, j, j1, e);
#pragma unroll
        for (int x = 0; x < kEach; ++x) {
            const bool lacks = j + 32 * x < j1 && !a.held(e[x]);
            const uint32_t lacking = __ballot_sync(0xffffffffu, lacks);
            const int k = rank + __popc(lacking & ((1u << lane) - 1u));
            page[x] = !lacks ? -2 : k < free ? read(a.list + k) : -1;
            rank += __popc(lacking);
        }
#pragma unroll
        for (int x = 0; x < kEach; ++x) {
            if (page[x] != -2) entries[j + 32 * x] = page[x];
            if (page[x] >= 0) a.refs[page[x]] = 1;
        }
    }
}
// The places of a CTA's units that lack pages among all such entries: what they count becomes how many before them, -1 where
// they lack none; returns the sum of those of CTAs before, and of all.
__device__ __forceinline__ int2 place_units(Cluster& c, int32_t* units, int mine) {
    int of_cta = 0;
    for (int u = 0; u < mine; u += kThreads) {
        const int at = u + threadIdx.x, n = at < mine ? units[at] : 0;
        const int2 order = c.scan(n);
        if (at < mine) units[at] = n > 0 ? of_cta + order.x : -1;
        of_cta += order.y;
    }
    return c.sum(of_cta);
}

__global__ void __launch_bounds__(kThreads, 1) resize_kernel(const Pages a, const int32_t* rows, const int32_t* tokens) {
    __shared__ Shared s;
    after_the_kernel_before();
    Cluster c{s};
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int64_t units = (int64_t)a.n * a.segments;
    const int64_t u0 = part(units, c.size(), c.rank()), u1 = part(units, c.size(), c.rank() + 1);
    const int mine = (int)(u1 - u0);
    Listed listed{a, s.list, rows, nullptr};
    listed.begin(c);
    for (int u = warp; u < mine; u += kWarps) {
        const int i = (int)((u0 + u) / a.segments), j0 = (int)((u0 + u) % a.segments) * a.segment;
        const int row = rows[i], need = pages_for(tokens[i], a);
        const int lacks = listed.counts(i, row) ? release_unit(a, row, need, j0) : 0;
        if (lane == 0) s.units[u] = lacks;
    }
    __syncthreads();
    const int2 all = place_units(c, s.units, mine);        // (and all that goes back has gone)
    int free = 0;
    if (all.y > 0) {
        free = list_free(c, a.refs, a.n_pages, all.y, a.list);
        c.meet();
        for (int u = warp; u < mine; u += kWarps) {
            if (s.units[u] < 0) continue;
            const int i = (int)((u0 + u) / a.segments), j0 = (int)((u0 + u) % a.segments) * a.segment;
            fill_unit(a, rows[i], pages_for(tokens[i], a), j0, all.x + s.units[u], free);
        }
    }
    if (a.missing && c.rank() == 0 && threadIdx.x == 0) *a.missing = all.y > free ? all.y - free : 0;
    c.meet();                                              // no CTA's sums go while others read them
}

// The same in three kernels: a warp a unit, the sums, a warp a unit.
__global__ void __launch_bounds__(kRowThreads) release_kernel(const Pages a, const int32_t* rows, const int32_t* tokens) {
    __shared__ int32_t list[2][kListed];
    after_the_kernel_before();
    Listed listed{a, list, rows, nullptr};
    listed.to_shared();
    __syncthreads();
    const int64_t u = (int64_t)blockIdx.x * (kRowThreads / 32) + (threadIdx.x >> 5);
    if (u >= (int64_t)a.n * a.segments) return;
    const int i = (int)(u / a.segments), j0 = (int)(u % a.segments) * a.segment;
    const int row = rows[i], need = pages_for(tokens[i], a);
    const int lacks = listed.counts(i, row) ? release_unit(a, row, need, j0) : 0;
    if ((threadIdx.x & 31) == 0) a.units[u] = lacks;
}
__global__ void __launch_bounds__(kThreads, 1) place_kernel(const Pages a) {
    __shared__ Shared s;
    after_the_kernel_before();
    Cluster c{s};
    const int64_t units = (int64_t)a.n * a.segments;
    const int64_t u0 = part(units, c.size(), c.rank()), u1 = part(units, c.size(), c.rank() + 1);
    const int2 all = place_units(c, a.units + u0, (int)(u1 - u0));
    for (int64_t u = u0 + threadIdx.x; u < u1; u += kThreads)
        if (a.units[u] >= 0) a.units[u] += all.x;          // (each thread's own)
    const int free = all.y > 0 ? list_free(c, a.refs, a.n_pages, all.y, a.list) : 0;
    if (c.rank() == 0 && threadIdx.x == 0) {
        a.sums[0] = all.y;
        a.sums[1] = free;
        if (a.missing) *a.missing = all.y > free ? all.y - free : 0;
    }
    c.meet();
}
__global__ void __launch_bounds__(kRowThreads) fill_kernel(const Pages a, const int32_t* rows, const int32_t* tokens) {
    after_the_kernel_before();
    const int64_t u = (int64_t)blockIdx.x * (kRowThreads / 32) + (threadIdx.x >> 5);
    if (u >= (int64_t)a.n * a.segments || a.units[u] < 0) return;
    const int i = (int)(u / a.segments), j0 = (int)(u % a.segments) * a.segment;
    fill_unit(a, rows[i], pages_for(tokens[i], a), j0, a.units[u], a.sums[1]);
}

__device__ __forceinline__ int tokens_of(const Pages& a, const int32_t* lengths, int row) {
    const int most = a.wide << a.page_shift, n = lengths[row];
    return n < 0 ? 0 : n < most ? n : most;
}
// A unit of a pair that counts: the full pages' entries to the target, with one holder more each; nothing behind them.
__device__ __forceinline__ void share_unit(const Pages& a, int source, int row, int full, int j0) {
    const int lane = threadIdx.x & 31, j1 = j0 + a.segment < a.wide ? j0 + a.segment : a.wide;
    const int32_t* theirs = a.table + (int64_t)source * a.wide;
    int32_t* entries = a.table + (int64_t)row * a.wide;
    for (int j = j0 + lane; j < j1 + lane; j += kSegment) {
        int32_t e[kEach];
        load_entries(theirs, j, full < j1 ? full : j1, e);
#pragma unroll
        for (int x = 0; x < kEach; ++x) {
            if (a.held(e[x])) atomicAdd(a.refs + e[x], 1);
            if (j + 32 * x < j1) entries[j + 32 * x] = a.held(e[x]) ? e[x] : -1;
        }
    }
}
__global__ void __launch_bounds__(kRowThreads)
    share_kernel(const Pages a, const int32_t* lengths, const int32_t* src, const int32_t* dst) {
    __shared__ int32_t list[2][kListed];
    after_the_kernel_before();
    Listed listed{a, list, dst, src};
    listed.to_shared();
    __syncthreads();
    const int64_t u = (int64_t)blockIdx.x * (kRowThreads / 32) + (threadIdx.x >> 5);
    if (u >= (int64_t)a.n * a.segments) return;
    const int i = (int)(u / a.segments), j0 = (int)(u % a.segments) * a.segment, row = dst[i], source = src[i];
    if (a.is_row(source) && listed.counts(i, row)) share_unit(a, source, row, tokens_of(a, lengths, source) >> a.page_shift, j0);
}

// SHARE: with the rows' full pages, else share_kernel has been before.
template <bool SHARE>
__global__ void __launch_bounds__(kThreads, 1)
    fork_kernel(const Pages a, int32_t* lengths, const int32_t* src, const int32_t* dst, int32_t* from, int32_t* to) {
    __shared__ Shared s;
    after_the_kernel_before();
    Cluster c{s};
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    // A pair counts if its target is the target of no pair before and the source of none.
    Listed listed{a, s.list, dst, src};
    const bool one_each = SHARE && a.segments == 1;        // a unit is a pair
    if (SHARE) {
        listed.begin(c);
        const int64_t units = (int64_t)a.n * a.segments;
        const int64_t u0 = part(units, c.size(), c.rank()), u1 = part(units, c.size(), c.rank() + 1);
        for (int64_t u = u0 + warp; u < u1; u += kWarps) {
            const int i = (int)(u / a.segments), j0 = (int)(u % a.segments) * a.segment;
            const int row = dst[i], source = src[i];
            int mark = -1;
            if (a.is_row(source) && listed.counts(i, row)) {
                const int n = tokens_of(a, lengths, source), full = n >> a.page_shift;
                const bool more = one_each && (n & ((1 << a.page_shift) - 1));
                const int32_t last = more ? a.table[(int64_t)source * a.wide + full] : -1;   // (beside the others' loads)
                share_unit(a, source, row, full, j0);
                mark = a.held(last);
            }
            if (one_each && lane == 0) s.units[u - u0] = mark;
        }
    } else {
        listed.to_shared();                                // (what long lists leave in the workspace is still there)
        __syncthreads();
    }
    // Pairs whose last page is partly filled, which want one of their own: in `units` first that, then their place.  (Where a unit
    // is a pair it has been seen there: 12.4 to 11.9 us for 8 rows of 64 entries.)
    const int64_t i0 = part(a.n, c.size(), c.rank()), i1 = part(a.n, c.size(), c.rank() + 1);
    const int mine = (int)(i1 - i0);
    for (int x = warp; x < mine && !one_each; x += kWarps) {
        const int i = (int)i0 + x, source = src[i];
        int mark = -1;
        if (a.is_row(source) && listed.counts(i, dst[i])) {
            const int n = tokens_of(a, lengths, source), full = n >> a.page_shift;
            mark = (n & ((1 << a.page_shift) - 1)) && a.held(a.table[(int64_t)source * a.wide + full]);
        }
        if (lane == 0) s.units[x] = mark;
    }
    __syncthreads();
    int of_cta = 0;
    for (int x = 0; x < mine; x += kThreads) {
        const int at = x + threadIdx.x, mark = at < mine ? s.units[at] : -1;
        const int2 order = c.scan(mark > 0);
        // -1: does not count; else twice its place, and one where it wants a page
        if (at < mine) s.units[at] = mark < 0 ? -1 : 2 * (of_cta + order.x) + mark;
        of_cta += order.y;
    }
    __syncthreads();
    const int2 all = c.sum(of_cta);
    int free = 0;
    if (all.y > 0) {
        free = list_free(c, a.refs, a.n_pages, all.y, a.list);
        c.meet();
    }
    for (int x = threadIdx.x; x < mine; x += kThreads) {
        const int i = (int)i0 + x, mark = s.units[x];
        int32_t page = -1, old = -1;
        if (mark >= 0) {
            const int n = tokens_of(a, lengths, src[i]), full = n >> a.page_shift;
            if (mark & 1) {
                const int k = all.x + (mark >> 1);
                if (k < free) {
                    page = read(a.list + k);
                    old = a.table[(int64_t)src[i] * a.wide + full];
                    a.refs[page] = 1;
                    a.table[(int64_t)dst[i] * a.wide + full] = page;
                }
            }
            lengths[dst[i]] = n;
        }
        from[i] = old;
        to[i] = page;
    }
    if (a.missing && c.rank() == 0 && threadIdx.x == 0) *a.missing = all.y > free ? all.y - free : 0;
    c.meet();
}

// Pages [0, H) are to be the held ones, H their number: the k-th held page from H on goes to the k-th free one below.
__global__ void __launch_bounds__(kThreads, 1)
    compact_kernel(const int32_t* refs, int32_t* refs_out, int64_t n_pages, int32_t* map, int32_t* from, int32_t* to,
                   int32_t* held) {
    __shared__ Shared s;
    after_the_kernel_before();
    Cluster c{s};
    const int lane = threadIdx.x & 31;
    const Range r = pages_of_warp(c, n_pages);
    const int warp_pages = (int)(r.to - r.from);
    uint32_t marks = 0;
    int mine = 0;                                          // held
    for (int64_t at = r.from; at < r.to; at += kBlock) {
        marks = free_marks(refs, at, r.to);
        mine -= count_marks(marks);
    }
    mine += warp_pages;
    const int2 of_cta = c.scan_warps(mine);
    const int2 all = c.sum(of_cta.y);
    const int64_t H = all.y;
    int holes = 0;
    for (int64_t at = r.from; at < r.to && at < H; at += kBlock) {
        if (warp_pages > kBlock) marks = free_marks(refs, at, r.to);
        holes += count_marks(marks_before(marks, at, H));
    }
    const int moves = c.sum(c.scan_warps(holes).y).y;
    int before = all.x + of_cta.x;                         // held pages before the next 32
    for (int64_t at = r.from; at < r.to; at += kBlock) {
        if (warp_pages > kBlock) marks = free_marks(refs, at, r.to);
#pragma unroll 1
        for (int g = 0; g < 32 && at + 32 * g < r.to; g += kEach) {
            int count[kEach];
#pragma unroll
            for (int x = 0; x < kEach; ++x) {
                const int64_t p = at + 32 * (g + x) + lane;
                count[x] = refs_out != refs && p < r.to ? read(refs + p) : 0;
            }
#pragma unroll
            for (int x = 0; x < kEach; ++x) {
                const int64_t p = at + 32 * (g + x) + lane;
                const uint32_t m = __shfl_sync(0xffffffffu, marks, g + x);   // the free ones
                const bool real = p < r.to, is_held = real && !(m >> lane & 1u);
                const uint32_t holders = __ballot_sync(0xffffffffu, is_held);
                const int rank = before + __popc(holders & ((1u << lane) - 1u));
                before += __popc(holders);
                if (!real) continue;
                const int page = (int)p;
                if (p < H) {
                    if (!is_held) to[page - rank] = page;
                    else if (refs_out != refs) refs_out[page] = count[x];
                    map[page] = is_held ? page : -1;
                } else if (is_held) {
                    from[rank - (int)(H - moves)] = page;
                } else {
                    refs_out[page] = 0;
                    map[page] = -1;
                }
            }
        }
    }
    c.meet();
    const int64_t most = n_pages / 2;
    for (int64_t k = (int64_t)c.rank() * kThreads + threadIdx.x; k < most; k += (int64_t)c.size() * kThreads) {
        if (k < moves) {
            const int32_t a = read(from + k), b = read(to + k);
            const int32_t count = read(refs + a);
            refs_out[b] = count;
            refs_out[a] = 0;
            map[a] = b;
        } else {
            from[k] = to[k] = -1;
        }
    }
    if (c.rank() == 0 && threadIdx.x == 0) *held = (int32_t)H;
    c.meet();
}

constexpr int kRemapThreads = 256;

__global__ void __launch_bounds__(kRemapThreads)
    remap_kernel(const int32_t* table, int32_t* table_out, int64_t entries, const int32_t* map, int64_t n_pages) {
    after_the_kernel_before();
    const int64_t i = (int64_t)blockIdx.x * kRemapThreads + threadIdx.x;
    if (i >= entries) return;
    const int32_t e = table[i];
    table_out[i] = e >= 0 && e < n_pages ? map[e] : -1;
}

// Pages copied: a page's codes of all heads are one run of bytes, a pair of them for keys and for values.  16 bytes a load,
// eight of a thread's in flight.  A CTA takes every so many-th 32 KB of the list, so that its empty places cost a glance
// each: with a CTA for each, 3,620 moves in a list of 8,192 took 191 us, of which 50 were empty CTAs.  16 times as many CTAs
// as the GPU holds: 8,192 pages of 128 KB 318 us (6.8 TB/s), 328 with four times, 352 with no more than it holds.
constexpr int kCopyThreads = 256;
constexpr int kCopyLoads = 8;
constexpr int kCopyVectors = kCopyThreads * kCopyLoads;
constexpr int kCopyCtas = 4, kCopyWaves = 16;   // CTAs a SM holds, and of all

struct PageCopy {
    uint8_t* codes[2];
    float* scale[2];
    const int32_t* src;
    const int32_t* dst;
    int64_t n_pages;
    unsigned works;
    int n;
    int heads;
    int vectors;                           // of 16 bytes in a page's keys, or values
    int parts;                             // CTAs' works that a page pair makes, or
    int together;                          // pairs that a work takes (one of the two is 1)
};

// Works of one large page pair's parts: the next work's pages are read while this one's are copied.
__global__ void __launch_bounds__(kCopyThreads, kCopyCtas) copy_parts_kernel(const PageCopy a) {
    after_the_kernel_before();
    const int both = 2 * a.vectors;
    unsigned work = blockIdx.x;
    auto read_pair = [&](unsigned w, int& pair, int& part, int32_t& from, int32_t& to) {
        pair = (int)(w / (unsigned)a.parts);
        part = (int)(w - (unsigned)pair * a.parts);
        from = w < a.works ? a.src[pair] : -1;
        to = w < a.works ? a.dst[pair] : -1;
    };
    int pair, part;
    int32_t from, to;
    read_pair(work, pair, part, from, to);
    while (work < a.works) {
        const unsigned next = work + gridDim.x;
        int next_pair, next_part;
        int32_t next_from, next_to;
        read_pair(next, next_pair, next_part, next_from, next_to);
        if (from >= 0 && from < a.n_pages && to >= 0 && to < a.n_pages) {
            const int begin = part * kCopyVectors + threadIdx.x;
            uint4 x[kCopyLoads];
#pragma unroll
            for (int k = 0; k < kCopyLoads; ++k) {
                const int at = begin + k * kCopyThreads, kv = at >= a.vectors;
                if (at < both)
                    x[k] = __ldcs(reinterpret_cast<const uint4*>(kv ? a.codes[1] : a.codes[0]) + (int64_t)from * a.vectors + at -
                                  kv * a.vectors);
            }
#pragma unroll
            for (int k = 0; k < kCopyLoads; ++k) {
                const int at = begin + k * kCopyThreads, kv = at >= a.vectors;
                if (at < both)
                    __stcs(reinterpret_cast<uint4*>(kv ? a.codes[1] : a.codes[0]) + (int64_t)to * a.vectors + at - kv * a.vectors, x[k]);
            }
            if (part == 0)
                for (int h = threadIdx.x; h < 2 * a.heads; h += kCopyThreads) {
                    float* scale = h < a.heads ? a.scale[0] + h : a.scale[1] + h - a.heads;
                    scale[(int64_t)to * a.heads] = scale[(int64_t)from * a.heads];
                }
        }
        work = next;
        pair = next_pair, part = next_part, from = next_from, to = next_to;
    }
}

// Several small page pairs a CTA.
__global__ void __launch_bounds__(kCopyThreads, kCopyCtas) copy_pairs_kernel(const PageCopy a) {
    after_the_kernel_before();
    auto held = [&](int32_t p) { return p >= 0 && p < a.n_pages; };
    const int both = 2 * a.vectors, first = (int)(blockIdx.x * (unsigned)a.together);
    uint4 x[kCopyLoads];
    uint4* out[kCopyLoads];
#pragma unroll
    for (int k = 0; k < kCopyLoads; ++k) {
        const int at = k * kCopyThreads + threadIdx.x;
        out[k] = nullptr;
        if (at >= a.together * both) continue;
        const int pair = at / both, in = at - pair * both;
        if (first + pair >= a.n) continue;
        const int32_t from = a.src[first + pair], to = a.dst[first + pair];
        if (!held(from) || !held(to)) continue;
        const int kv = in >= a.vectors, v = in - kv * a.vectors;
        uint4* codes = reinterpret_cast<uint4*>(kv ? a.codes[1] : a.codes[0]);
        x[k] = __ldcs(codes + (int64_t)from * a.vectors + v);
        out[k] = codes + (int64_t)to * a.vectors + v;
    }
#pragma unroll
    for (int k = 0; k < kCopyLoads; ++k)
        if (out[k]) __stcs(out[k], x[k]);
    const int scales = 2 * a.heads;
    for (int at = threadIdx.x; at < a.together * scales; at += kCopyThreads) {
        const int pair = at / scales, in = at - pair * scales;
        if (first + pair >= a.n) continue;
        const int32_t from = a.src[first + pair], to = a.dst[first + pair];
        if (!held(from) || !held(to)) continue;
        const int kv = in >= a.heads, h = in - kv * a.heads;
        float* scale = kv ? a.scale[1] : a.scale[0];
        scale[(int64_t)to * a.heads + h] = scale[(int64_t)from * a.heads + h];
    }
}

// One cluster, or one CTA where `work` (entries and counts to look through) is some rounds of its threads.  Resize and fork, us, one
// CTA and a cluster of eight: of 2,560 7.9 and 8.5; 16,896 7.8 and 8.4, 12.4 and 13.4; 24,576 9.2 and 9.0, 13.7 and 13.4; 32,768
// 11.8 and 9.0, 16.6 and 13.5.
template <typename... P>
cudaError_t launch_cluster(void (*kernel)(P...), int64_t work, cudaStream_t stream, typename as_given<P>::type... args) {
    const unsigned ctas = work <= 20 * kThreads ? 1 : kCluster;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(ctas);
    cfg.blockDim = dim3(kThreads);
    cfg.stream = stream;
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.x = ctas;
    attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 2;
    return cudaLaunchKernelEx(&cfg, kernel, args...);
}

Pages pages_of(const CachePages& p, void* workspace) {
    Pages a = {};
    a.list = static_cast<int32_t*>(workspace);
    a.first = a.list + p.n_pages;
    a.units = a.first + p.n_rows;
    a.sums = a.units + (int64_t)kCluster * kUnits;
    a.refs = p.refs;
    a.table = p.table;
    a.n_pages = p.n_pages;
    a.n_rows = p.n_rows;
    a.wide = p.table_pages;
    a.page_shift = p.page_shift;
    a.n = p.n;
    a.missing = p.missing;
    a.segment = kSegment;
    // (whatever the launch's CTAs: no CTA of one has more units than its shared memory counts)
    for (;;) {
        a.segments = (a.wide + a.segment - 1) / a.segment;
        if ((int64_t)a.n * a.segments <= (int64_t)kCluster * kUnits || a.segments <= 1) break;
        a.segment *= 2;
    }
    return a;
}
// (More rows or units than a CTA's shared memory counts are a cluster's, whatever there is to look through.)
int64_t looked_through(const CachePages& p, const Pages& a) {
    const bool many = a.n > kUnits || (int64_t)a.n * a.segments > kUnits;
    return many ? INT64_MAX : (int64_t)p.n * p.table_pages + p.n_pages;
}

}  // namespace

// Rows that one call takes: a CTA of the cluster counts for kUnits of them.
int cache_pages_most_rows() { return kCluster * kUnits; }

size_t cache_pages_workspace_bytes(int64_t n_pages, int n_rows) {
    return ((size_t)(n_pages + n_rows + (int64_t)kCluster * kUnits + 2) * sizeof(int32_t) + 255) / 256 * 256;
}

// Entries up to which one cluster walks the rows too.  A resize that takes a page a row, us in the cluster and over the whole GPU:
// 8 rows x 64 entries 8.4 and 10.6, 128 x 256 9.3 and 10.6, 64 x 1,024 9.9 and 11.0, 400 x 1,024 25.8 and 12.4; a fork of as many
// rows: 13.4 and 14.3, 13.9 and 15.2, 14.6 and 15.4, 22.4 and 16.7.
constexpr int64_t kWide = 65536;

template <typename... P>
cudaError_t launch_rows(void (*kernel)(P...), const Pages& a, cudaStream_t stream, typename as_given<P>::type... args) {
    const int64_t units = (int64_t)a.n * a.segments;
    return launch_chained(kernel, (unsigned)((units + kRowThreads / 32 - 1) / (kRowThreads / 32)), kRowThreads, 0, stream, args...);
}
cudaError_t claim_rows(const Pages& a, const int32_t* rows, const int32_t* bars, cudaStream_t stream) {
    if (a.n <= kListed) return cudaSuccess;
    const unsigned ctas = (unsigned)((a.n + kRowThreads - 1) / kRowThreads);
    const cudaError_t e = launch_chained(clear_kernel, ctas, kRowThreads, 0, stream, a, rows, bars);
    return e != cudaSuccess ? e : launch_chained(claim_kernel, ctas, kRowThreads, 0, stream, a, rows, bars);
}

cudaError_t run_cache_resize(const CachePages& p, const int32_t* rows, const int32_t* tokens, void* workspace,
                             cudaStream_t stream) {
    const Pages a = pages_of(p, workspace);
    if ((int64_t)p.n * p.table_pages <= kWide) return launch_cluster(resize_kernel, looked_through(p, a), stream, a, rows, tokens);
    cudaError_t e = claim_rows(a, rows, nullptr, stream);
    if (e == cudaSuccess) e = launch_rows(release_kernel, a, stream, a, rows, tokens);
    if (e == cudaSuccess) e = launch_cluster(place_kernel, looked_through(p, a), stream, a);
    return e != cudaSuccess ? e : launch_rows(fill_kernel, a, stream, a, rows, tokens);
}

cudaError_t run_cache_fork(const CachePages& p, int32_t* lengths, const int32_t* src, const int32_t* dst, int32_t* from,
                           int32_t* to, void* workspace, cudaStream_t stream) {
    const Pages a = pages_of(p, workspace);
    if ((int64_t)p.n * p.table_pages <= kWide)
        return launch_cluster(fork_kernel<true>, looked_through(p, a), stream, a, lengths, src, dst, from, to);
    cudaError_t e = claim_rows(a, dst, src, stream);
    if (e == cudaSuccess) e = launch_rows(share_kernel, a, stream, a, lengths, src, dst);
    return e != cudaSuccess ? e : launch_cluster(fork_kernel<false>, looked_through(p, a), stream, a, lengths, src, dst, from, to);
}

cudaError_t run_cache_compact(const int32_t* refs, int32_t* refs_out, int64_t n_pages, const int32_t* table,
                              int32_t* table_out, int64_t entries, int32_t* map, int32_t* from, int32_t* to, int32_t* held,
                              cudaStream_t stream) {
    // (the counts are looked through three times)
    cudaError_t e = launch_cluster(compact_kernel, 3 * n_pages, stream, refs, refs_out, n_pages, map, from, to, held);
    if (e != cudaSuccess || entries == 0) return e;
    return launch_chained(remap_kernel, (unsigned)((entries + kRemapThreads - 1) / kRemapThreads), kRemapThreads, 0, stream,
                          table, table_out, entries, map, n_pages);
}

cudaError_t run_cache_copy(void* k_codes, void* v_codes, float* k_scale, float* v_scale, const int32_t* src,
                           const int32_t* dst, int n, int heads, int d, int64_t n_pages, int page, cudaStream_t stream,
                           int num_sms) {
    PageCopy a = {};
    a.codes[0] = static_cast<uint8_t*>(k_codes);
    a.codes[1] = static_cast<uint8_t*>(v_codes);
    a.scale[0] = k_scale;
    a.scale[1] = v_scale;
    a.src = src;
    a.dst = dst;
    a.n_pages = n_pages;
    a.n = n;
    a.heads = heads;
    a.vectors = heads * (page * d / 16);
    const int both = 2 * a.vectors;
    a.parts = (both + kCopyVectors - 1) / kCopyVectors;
    a.together = a.parts > 1 ? 1 : kCopyVectors / both;
    if (a.parts == 1) return launch_chained(copy_pairs_kernel, (unsigned)((n + a.together - 1) / a.together), kCopyThreads, 0, stream, a);
    a.works = (unsigned)n * (unsigned)a.parts;
    const unsigned most = (unsigned)(num_sms * kCopyCtas * kCopyWaves);
    return launch_chained(copy_parts_kernel, a.works < most ? a.works : most, kCopyThreads, 0, stream, a);
}

}  // namespace kda
