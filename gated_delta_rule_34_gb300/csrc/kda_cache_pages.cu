// kda_cache_pages.cu -- pages of the 8-bit cache changing hands: copied, given to rows of the block table and taken
// back, shared by rows that fork, moved to the front of the pool.
//
// refs[p] counts the entries of block tables that hold page p; a page with none is free.  What is taken is always the
// lowest free page, in the order of what asks for it, so that the same call gives the same table:
//
//   the k-th entry that lacks a page gets the k-th page with refs == 0
//
// which is a prefix sum over the entries and one over the pages.  A call's work is small (a table of 400 rows x 1,024
// entries and the counts of 262,144 pages are 2.7 MB) and its steps follow one another, so what bounds it is their
// number: one cluster of CTAs does all of them in one launch, its CTAs' sums handed over through distributed shared memory
// between hardware barriers.  One CTA where there is little to look through.
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
constexpr int kSegment = 256;              // entries of a unit, at least

struct Shared {
    int warp_sum[kWarps];
    int slot[8];                           // of sums that the cluster's CTAs tell one another
    int units[kUnits];
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

    // Sum over the CTA's threads before this one, and of all.
    __device__ __forceinline__ int2 scan(int value) {
        const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
        int up = value;
#pragma unroll
        for (int w = 1; w < 32; w <<= 1) {
            const int x = __shfl_up_sync(0xffffffffu, up, w);
            if (lane >= w) up += x;
        }
        __syncthreads();
        if (lane == 31) s.warp_sum[warp] = up;
        __syncthreads();
        int of_warps = s.warp_sum[lane];
#pragma unroll
        for (int w = 1; w < 32; w <<= 1) {
            const int x = __shfl_up_sync(0xffffffffu, of_warps, w);
            if (lane >= w) of_warps += x;
        }
        const int before = __shfl_sync(0xffffffffu, of_warps, warp > 0 ? warp - 1 : 0);
        return make_int2((warp > 0 ? before : 0) + up - value, __shfl_sync(0xffffffffu, of_warps, 31));
    }
};

// [0, n) in equal parts, one a CTA, in order.
__device__ __forceinline__ int64_t part(int64_t n, int size, int rank) {
    const int64_t each = (n + size - 1) / size, at = each * rank;
    return at < n ? at : n;
}

// Calls f(page, count, 0 to 3) for the CTA's pages [from, to), four neighbours a thread; rounds in order.  f may meet the
// CTA's other threads; pages past the end come with count 1.
template <typename F>
__device__ __forceinline__ void for_pages(const int32_t* refs, int64_t from, int64_t to, F f) {
    for (int64_t p0 = from; p0 < to; p0 += 4 * kThreads) {
        const int64_t p = p0 + 4 * threadIdx.x;
        int count[4];
#pragma unroll
        for (int k = 0; k < 4; ++k) count[k] = p + k < to ? read(refs + p + k) : 1;
        if (!f(p, count)) return;
    }
}

// The lowest `wanted` free pages, in order, to `list`; returns how many pages are free.  All threads of the cluster call
// it, after what changes refs, and meet before they read the list.
__device__ __forceinline__ int list_free(Cluster& c, const int32_t* refs, int64_t n_pages, int wanted, int32_t* list) {
    const int64_t from = part(n_pages, c.size(), c.rank()), to = part(n_pages, c.size(), c.rank() + 1);
    int mine = 0;
    for_pages(refs, from, to, [&](int64_t, const int (&count)[4]) {
#pragma unroll
        for (int k = 0; k < 4; ++k) mine += count[k] <= 0;
        return true;
    });
    const int2 all = c.sum(c.scan(mine).y);
    int at = all.x;
    for_pages(refs, from, to, [&](int64_t p, const int (&count)[4]) {
        if (at >= wanted) return false;
        int n = 0;
#pragma unroll
        for (int k = 0; k < 4; ++k) n += count[k] <= 0;
        const int2 order = c.scan(n);
        int rank = at + order.x;
#pragma unroll
        for (int k = 0; k < 4; ++k)
            if (count[k] <= 0) {
                if (rank < wanted) list[rank] = (int32_t)(p + k);
                ++rank;
            }
        at += order.y;
        return true;
    });
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
    int32_t* list;                         // the workspace: [n_pages]

    __device__ __forceinline__ bool held(int32_t e) const { return e >= 0 && e < n_pages; }
    __device__ __forceinline__ bool is_row(int r) const { return r >= 0 && r < n_rows; }
};

// Whether x stands among list[0 .. n): a warp looks.
__device__ __forceinline__ bool among(const int32_t* list, int n, int x) {
    bool found = false;
    for (int j = threadIdx.x & 31; j < n; j += 32) found |= list[j] == x;
    return __any_sync(0xffffffffu, found);
}

// One holder less.  (A count that says none is left alone: the table did not match it.)
__device__ __forceinline__ void give_back(int32_t* refs, int32_t page) {
    if (atomicSub(refs + page, 1) <= 0) atomicAdd(refs + page, 1);
}

__device__ __forceinline__ int pages_for(int tokens, const Pages& a) {
    const int n = tokens > 0 ? ((tokens - 1) >> a.page_shift) + 1 : 0;
    return n < a.wide ? n : a.wide;
}

__global__ void __launch_bounds__(kThreads, 1) resize_kernel(const Pages a, const int32_t* rows, const int32_t* tokens) {
    __shared__ Shared s;
    after_the_kernel_before();
    Cluster c{s};
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int64_t units = (int64_t)a.n * a.segments;
    const int64_t u0 = part(units, c.size(), c.rank()), u1 = part(units, c.size(), c.rank() + 1);
    const int mine = (int)(u1 - u0);
    // What rows do not need goes back; what they lack is counted.
    for (int u = warp; u < mine; u += kWarps) {
        const int i = (int)((u0 + u) / a.segments), j0 = (int)((u0 + u) % a.segments) * a.segment;
        const int row = rows[i];
        int lacks = 0;
        if (a.is_row(row) && !among(rows, i, row)) {
            const int need = pages_for(tokens[i], a), j1 = j0 + a.segment < a.wide ? j0 + a.segment : a.wide;
            int32_t* entries = a.table + (int64_t)row * a.wide;
            for (int j = j0 + lane; j < j1; j += 32) {
                const int32_t e = entries[j];
                if (j >= need) {
                    if (a.held(e)) give_back(a.refs, e);
                    if (e != -1) entries[j] = -1;
                } else {
                    lacks += !a.held(e);
                }
            }
            lacks = __reduce_add_sync(0xffffffffu, lacks);
        }
        if (lane == 0) s.units[u] = lacks;
    }
    __syncthreads();
    // Their places among all that lack.
    int of_cta = 0;
    for (int u = 0; u < mine; u += kThreads) {
        const int at = u + threadIdx.x, n = at < mine ? s.units[at] : 0;
        const int2 order = c.scan(n);
        if (at < mine) s.units[at] = n > 0 ? of_cta + order.x : -1;
        of_cta += order.y;
    }
    const int2 all = c.sum(of_cta);                        // (and all that goes back has gone)
    int free = 0;
    if (all.y > 0) {
        free = list_free(c, a.refs, a.n_pages, all.y, a.list);
        c.meet();
        for (int u = warp; u < mine; u += kWarps) {
            if (s.units[u] < 0) continue;
            const int i = (int)((u0 + u) / a.segments), j0 = (int)((u0 + u) % a.segments) * a.segment;
            const int need = pages_for(tokens[i], a), j1 = j0 + a.segment < need ? j0 + a.segment : need;
            int32_t* entries = a.table + (int64_t)rows[i] * a.wide;
            int rank = all.x + s.units[u];
            for (int j = j0; j < j1; j += 32) {
                const bool lacks = j + lane < j1 && !a.held(entries[j + lane]);
                const uint32_t lacking = __ballot_sync(0xffffffffu, lacks);
                const int k = rank + __popc(lacking & ((1u << lane) - 1));
                if (lacks) {
                    const int32_t page = k < free ? read(a.list + k) : -1;
                    entries[j + lane] = page;
                    if (page >= 0) a.refs[page] = 1;
                }
                rank += __popc(lacking);
            }
        }
    }
    if (a.missing && c.rank() == 0 && threadIdx.x == 0) *a.missing = all.y > free ? all.y - free : 0;
    c.meet();                                              // no CTA's sums go while others read them
}

__global__ void __launch_bounds__(kThreads, 1)
    fork_kernel(const Pages a, int32_t* lengths, const int32_t* src, const int32_t* dst, int32_t* from, int32_t* to) {
    __shared__ Shared s;
    after_the_kernel_before();
    Cluster c{s};
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    auto tokens_of = [&](int row) {
        const int most = a.wide << a.page_shift, n = lengths[row];
        return n < 0 ? 0 : n < most ? n : most;
    };
    // A pair counts if its target is the target of no pair before and the source of none.
    auto counts = [&](int i) {
        return a.is_row(src[i]) && a.is_row(dst[i]) && !among(dst, i, dst[i]) && !among(src, a.n, dst[i]);
    };
    const int64_t units = (int64_t)a.n * a.segments;
    const int64_t u0 = part(units, c.size(), c.rank()), u1 = part(units, c.size(), c.rank() + 1);
    for (int64_t u = u0 + warp; u < u1; u += kWarps) {
        const int i = (int)(u / a.segments), j0 = (int)(u % a.segments) * a.segment;
        if (!counts(i)) continue;
        const int full = tokens_of(src[i]) >> a.page_shift, j1 = j0 + a.segment < a.wide ? j0 + a.segment : a.wide;
        const int32_t* theirs = a.table + (int64_t)src[i] * a.wide;
        int32_t* entries = a.table + (int64_t)dst[i] * a.wide;
        for (int j = j0 + lane; j < j1; j += 32) {
            const int32_t e = j < full ? theirs[j] : -1;
            if (a.held(e)) atomicAdd(a.refs + e, 1);
            entries[j] = a.held(e) ? e : -1;
        }
    }
    // Pairs whose last page is partly filled, which want one of their own: one bit of `units` a pair, its place in the rest.
    const int64_t i0 = part(a.n, c.size(), c.rank()), i1 = part(a.n, c.size(), c.rank() + 1);
    const int mine = (int)(i1 - i0);
    for (int x = warp; x < mine; x += kWarps) {
        const int i = (int)i0 + x;
        bool wants = false;
        if (counts(i)) {
            const int n = tokens_of(src[i]), full = n >> a.page_shift;
            wants = (n & ((1 << a.page_shift) - 1)) && a.held(a.table[(int64_t)src[i] * a.wide + full]);
            if (lane == 0) s.units[x] = wants ? 1 : 0;
        } else if (lane == 0) {
            s.units[x] = -1;
        }
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
            const int n = tokens_of(src[i]), full = n >> a.page_shift;
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
    const int64_t p0 = part(n_pages, c.size(), c.rank()), p1 = part(n_pages, c.size(), c.rank() + 1);
    int mine = 0;
    for_pages(refs, p0, p1, [&](int64_t p, const int (&count)[4]) {
#pragma unroll
        for (int k = 0; k < 4; ++k) mine += p + k < p1 && count[k] > 0;
        return true;
    });
    const int2 all = c.sum(c.scan(mine).y);
    const int64_t H = all.y;
    mine = 0;
    for_pages(refs, p0, H < p1 ? H : p1, [&](int64_t p, const int (&count)[4]) {
#pragma unroll
        for (int k = 0; k < 4; ++k) mine += count[k] <= 0;
        return true;
    });
    const int2 holes = c.sum(c.scan(mine).y);
    const int moves = holes.y;
    int at = all.x;                                        // held pages before the round
    for_pages(refs, p0, p1, [&](int64_t p, const int (&count)[4]) {
        int n = 0;
#pragma unroll
        for (int k = 0; k < 4; ++k) n += p + k < p1 && count[k] > 0;
        const int2 order = c.scan(n);
        int before = at + order.x;
#pragma unroll
        for (int k = 0; k < 4; ++k) {
            if (p + k >= p1) break;
            const bool is_held = count[k] > 0;
            const int page = (int)(p + k);
            if (page < H) {
                if (!is_held) to[page - before] = page;
                else refs_out[page] = count[k];
                map[page] = is_held ? page : -1;
            } else {
                if (is_held) from[before - (int)(H - moves)] = page;
                else {
                    refs_out[page] = 0;
                    map[page] = -1;
                }
            }
            before += is_held;
        }
        at += order.y;
        return true;
    });
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
// eight of a thread's in flight.
constexpr int kCopyThreads = 256;
constexpr int kCopyLoads = 8;
constexpr int kCopyVectors = kCopyThreads * kCopyLoads;

struct PageCopy {
    uint8_t* codes[2];
    float* scale[2];
    const int32_t* src;
    const int32_t* dst;
    int64_t n_pages;
    int n;
    int heads;
    int vectors;                           // of 16 bytes in a page's keys, or values
    int parts;                             // CTAs of a page pair, or
    int together;                          // pairs of a CTA (one of the two is 1)
};

__global__ void __launch_bounds__(kCopyThreads) copy_kernel(const PageCopy a) {
    after_the_kernel_before();
    const int64_t first = a.parts > 1 ? blockIdx.x / a.parts : (int64_t)blockIdx.x * a.together;
    const int both = 2 * a.vectors;
    const int begin = a.parts > 1 ? (int)(blockIdx.x % a.parts) * kCopyVectors : 0;
    const int end = a.parts > 1 ? (begin + kCopyVectors < both ? begin + kCopyVectors : both) : a.together * both;
    auto held = [&](int32_t p) { return p >= 0 && p < a.n_pages; };
    uint4 x[kCopyLoads];
    uint4* out[kCopyLoads];
#pragma unroll
    for (int k = 0; k < kCopyLoads; ++k) {
        const int at = begin + k * kCopyThreads + threadIdx.x;
        out[k] = nullptr;
        if (at >= end) continue;
        const int pair = a.parts > 1 ? 0 : at / both, in = a.parts > 1 ? at : at - pair * both;
        const int64_t i = first + pair;
        if (i >= a.n) continue;
        const int32_t from = a.src[i], to = a.dst[i];
        if (!held(from) || !held(to)) continue;
        const int kv = in >= a.vectors, v = in - kv * a.vectors;
        uint4* codes = reinterpret_cast<uint4*>(kv ? a.codes[1] : a.codes[0]);
        x[k] = __ldcs(codes + (int64_t)from * a.vectors + v);
        out[k] = codes + (int64_t)to * a.vectors + v;
    }
#pragma unroll
    for (int k = 0; k < kCopyLoads; ++k)
        if (out[k]) __stcs(out[k], x[k]);
    if (begin > 0) return;
    const int scales = 2 * a.heads;
    for (int at = threadIdx.x; at < a.together * scales; at += kCopyThreads) {
        const int pair = at / scales, in = at - pair * scales;
        const int64_t i = first + pair;
        if (i >= a.n) continue;
        const int32_t from = a.src[i], to = a.dst[i];
        if (!held(from) || !held(to)) continue;
        const int kv = in >= a.heads, h = in - kv * a.heads;
        float* scale = kv ? a.scale[1] : a.scale[0];
        scale[(int64_t)to * a.heads + h] = scale[(int64_t)from * a.heads + h];
    }
}

// One cluster, or one CTA where `work` (entries and counts to look through) is a few rounds of its threads.
template <typename... P>
cudaError_t launch_cluster(void (*kernel)(P...), int64_t work, cudaStream_t stream, typename as_given<P>::type... args) {
    const unsigned ctas = work <= 8 * kThreads ? 1 : kCluster;
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

Pages pages_of(const CachePages& p, int32_t* list) {
    Pages a = {};
    a.refs = p.refs;
    a.table = p.table;
    a.n_pages = p.n_pages;
    a.n_rows = p.n_rows;
    a.wide = p.table_pages;
    a.page_shift = p.page_shift;
    a.n = p.n;
    a.missing = p.missing;
    a.list = list;
    a.segment = kSegment;
    // (whatever the launch's CTAs: no CTA of one has more units than its shared memory counts)
    for (;;) {
        a.segments = (a.wide + a.segment - 1) / a.segment;
        if ((int64_t)a.n * a.segments <= (int64_t)kCluster * kUnits || a.segments <= 1) break;
        a.segment *= 2;
    }
    return a;
}
int64_t looked_through(const CachePages& p) { return (int64_t)p.n * p.table_pages + p.n_pages; }

}  // namespace

// Rows that one call takes: a CTA of the cluster counts for kUnits of them.
int cache_pages_most_rows() { return kCluster * kUnits; }

size_t cache_pages_workspace_bytes(int64_t n_pages) { return ((size_t)n_pages * sizeof(int32_t) + 255) / 256 * 256; }

cudaError_t run_cache_resize(const CachePages& p, const int32_t* rows, const int32_t* tokens, void* workspace,
                             cudaStream_t stream) {
    return launch_cluster(resize_kernel, looked_through(p), stream, pages_of(p, static_cast<int32_t*>(workspace)), rows,
                          tokens);
}

cudaError_t run_cache_fork(const CachePages& p, int32_t* lengths, const int32_t* src, const int32_t* dst, int32_t* from,
                           int32_t* to, void* workspace, cudaStream_t stream) {
    return launch_cluster(fork_kernel, looked_through(p), stream, pages_of(p, static_cast<int32_t*>(workspace)), lengths,
                          src, dst, from, to);
}

cudaError_t run_cache_compact(const int32_t* refs, int32_t* refs_out, int64_t n_pages, const int32_t* table,
                              int32_t* table_out, int64_t entries, int32_t* map, int32_t* from, int32_t* to, int32_t* held,
                              cudaStream_t stream) {
    cudaError_t e = launch_cluster(compact_kernel, n_pages, stream, refs, refs_out, n_pages, map, from, to, held);
    if (e != cudaSuccess || entries == 0) return e;
    return launch_chained(remap_kernel, (unsigned)((entries + kRemapThreads - 1) / kRemapThreads), kRemapThreads, 0, stream,
                          table, table_out, entries, map, n_pages);
}

cudaError_t run_cache_copy(void* k_codes, void* v_codes, float* k_scale, float* v_scale, const int32_t* src,
                           const int32_t* dst, int n, int heads, int d, int64_t n_pages, int page, cudaStream_t stream) {
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
    const int64_t ctas = a.parts > 1 ? (int64_t)n * a.parts : (n + a.together - 1) / a.together;
    return launch_chained(copy_kernel, (unsigned)ctas, kCopyThreads, 0, stream, a);
}

}  // namespace kda
