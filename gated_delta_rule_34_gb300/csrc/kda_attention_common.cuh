// kda_attention_common.cuh -- what the attention kernels over the paged 8-bit cache share: the
// list of an item's steps, its sharing out over CTAs, and how a finished row is written.
#pragma once

#include <climits>

#include "kda_cache.cuh"
#include "kda_cache_internal.h"
#include "kda_chained.cuh"
#include "tc_util.cuh"

namespace kda {
namespace attn {

// What a launch attends over: a sequence's whole cache; the prefix that a group of sequences shares, all their rows as one
// item's, whose sums are carried on; the rest of a sequence, joined with what its rows carry.
enum Part { kAll, kPrefix, kRest };

constexpr int kStep = 16;             // tokens of a step; a page holds whole steps
constexpr int kMinShare = 16;         // steps below which no item is cut further
constexpr int kJoinThreads = 256;
constexpr int kJoinFew = 32;          // pieces up to which a warp joins a row
constexpr int kAtOnce = 4;            // pieces that a warp loads at once
constexpr int kMaxScan = 8192;        // (sequence, row tile) pairs that every CTA sums up
constexpr float kWeightBits = 12.0f;  // log2 of what the largest weight is brought to
constexpr float kSlack = 2.0f;        // log2 of how far scores may pass the reference
constexpr float kLowest = -3.402823466e38f;   // the reference before any score

// Where the many-row kernel's loaders and products stop (a self-test's; else never), and the limit of its waits.
struct Stall {
    int loads = INT_MAX;     // tiles that a CTA's loaders load
    int tiles = INT_MAX;     // tiles of which a CTA's products are issued
    int wait_us = 2000000;
};

struct Plan {
    int group;          // query heads of a head of keys
    int rows;           // T_q * group
    int tile_rows;      // rows of a tile
    int row_tiles;
    int pairs;          // kPrefix: (group, row tile) places, as groups_tile deals them out
    int stored;         // rows of a tile that exist
    int item_cost;      // what an item's start and end cost, in steps
    int cut;            // items are cut at multiples of this many steps
    float* sums;        // [grid][2][stored][D]
    float4* stats;      // [grid][2][stored]: m, dm, l
    int4* joins;        // [grid]: pair (sequence, row tile), head, last CTA, slot; pair < 0: none
    Stall stall;
};

// What a row tile of a sequence sees, in steps.
struct Tile {
    int p0, p1;         // positions of its first and last row
    int end;            // tokens [0, end) at most
    int first_step;     // of the window (or 0), after sink_steps steps from 0
    int sink_steps;
    int steps;          // at least 1, so that a row that sees nothing is written too (kPrefix: 0 where there are no rows)
    bool carried;       // kRest: rows go on from what they carry
    __device__ __forceinline__ int token(int s) const {
        return (s < sink_steps ? s : first_step + s - sink_steps) * kStep;
    }
};

// Sequences of group g, and the tokens that they share: whole pages, and none for fewer than two sequences.
__device__ __forceinline__ int2 group_range(const CacheAttention& a, int g, int n_seqs) {
    int lo = a.cu_groups[g], hi = a.cu_groups[g + 1];
    lo = lo < 0 ? 0 : lo > n_seqs ? n_seqs : lo;
    hi = hi < lo ? lo : hi > n_seqs ? n_seqs : hi;
    return make_int2(lo, hi);
}
__device__ __forceinline__ int shared_tokens(const CacheAttention& a, int g, int2 range) {
    const int cap = a.prefix_pages << a.page_shift, n = a.prefix_len[g];
    if (range.y - range.x < 2 || n <= 0) return 0;
    return (n < cap ? n : cap) >> a.page_shift << a.page_shift;
}
// kRest: how many of sequence b's tokens its rows carry the sums of.  All of them must see all of the prefix; a
// sequence whose rows do not attends over all of its own table.
__device__ __forceinline__ int carried_tokens(const CacheAttention& a, int b, int len) {
    if (a.prefix_pages == 0) return 0;
    int g = 0, end = a.n_groups;                           // the last group that starts at b or before
    while (end - g > 1) {
        const int mid = (g + end) >> 1;
        if (a.cu_groups[mid] <= b) g = mid;
        else end = mid;
    }
    const int2 range = group_range(a, g, a.B);
    if (b < range.x || b >= range.y) return 0;
    const int n = shared_tokens(a, g, range);
    return len - a.T_q + 1 >= n ? n : 0;
}

// kPrefix: place `pair` of plan.pairs is row tile .y of group .x.  Group g's start at floor(rows before it / tile_rows) + g, which
// leaves each room enough wherever its rows begin.  (a.B: sequences, as everywhere.)
__device__ __forceinline__ int groups_first(const CacheAttention& a, const Plan& plan, int g) {
    int lo = a.cu_groups[g];
    lo = lo < 0 ? 0 : lo > a.B ? a.B : lo;
    return (int)((int64_t)lo * plan.group * a.T_q / plan.tile_rows) + g;
}
__device__ __forceinline__ int2 groups_tile(const CacheAttention& a, const Plan& plan, int pair) {
    int g = 0, end = a.n_groups;
    while (end - g > 1) {
        const int mid = (g + end) >> 1;
        if (groups_first(a, plan, mid) <= pair) g = mid;
        else end = mid;
    }
    return make_int2(g, pair - groups_first(a, plan, g));
}

// (sequence or group, row tile) of a pair.
template <Part P>
__device__ __forceinline__ int2 split_pair(const CacheAttention& a, const Plan& plan, int pair) {
    if constexpr (P == kPrefix) return groups_tile(a, plan, pair);
    else return make_int2(pair / plan.row_tiles, pair % plan.row_tiles);
}
// The first query token of sequence or group b, and its rows.
template <Part P>
__device__ __forceinline__ int64_t first_query(const CacheAttention& a, int b) {
    if constexpr (P == kPrefix) return (int64_t)group_range(a, b, a.B).x * a.T_q;
    else return (int64_t)b * a.T_q;
}
template <Part P>
__device__ __forceinline__ int item_rows(const CacheAttention& a, const Plan& plan, int b) {
    if constexpr (P == kPrefix) {
        const int2 range = group_range(a, b, a.B);
        return (range.y - range.x) * a.T_q * plan.group;
    } else {
        return plan.rows;
    }
}

__device__ __forceinline__ Tile make_tile(const CacheAttention& a, const Plan& plan, int len, int rt, int carried = 0) {
    Tile t;
    if (plan.row_tiles == 1) {                             // no division on the way to a decode step's first loads
        t.p0 = len - a.T_q;
        t.p1 = len - 1;
    } else {
        const int r0 = rt * plan.tile_rows;
        const int r1 = (plan.rows < r0 + plan.tile_rows ? plan.rows : r0 + plan.tile_rows) - 1;
        t.p0 = len - a.T_q + r0 / plan.group;
        t.p1 = len - a.T_q + r1 / plan.group;
    }
    t.end = t.p1 + 1 > 0 ? t.p1 + 1 : 0;
    int lo = carried, sink_end = 0;
    t.carried = carried > 0;
    if (a.window > 0) {
        const int64_t l = (int64_t)t.p0 - a.window + 1;
        lo = l > 0 ? (int)l : 0;
        sink_end = a.sinks < lo ? a.sinks : lo;
    }
    t.first_step = lo / kStep;
    t.sink_steps = (sink_end + kStep - 1) / kStep;
    if (t.sink_steps > t.first_step) t.sink_steps = t.first_step;
    const int n = t.sink_steps + (t.end + kStep - 1) / kStep - t.first_step;
    t.steps = n > 1 ? n : 1;
    return t;
}

__device__ __forceinline__ int length_of(const CacheAttention& a, int b) {
    const int cap = a.table_pages << a.page_shift;
    const int len = a.lengths[b];
    return len < 0 ? 0 : (len > cap ? cap : len);
}

__device__ __forceinline__ float ex2(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}
// The tile of pair (sequence, row tile).
template <Part P = kAll>
__device__ __forceinline__ Tile tile_of(const CacheAttention& a, const Plan& plan, int pair) {
    if constexpr (P == kPrefix) {                          // every row sees all of the prefix
        const int2 at = groups_tile(a, plan, pair);
        const int2 range = group_range(a, at.x, a.B);
        const int64_t rows = (int64_t)(range.y - range.x) * a.T_q * plan.group;
        Tile t;
        t.end = at.y >= 0 && (int64_t)at.y * plan.tile_rows < rows ? shared_tokens(a, at.x, range) : 0;
        t.p0 = t.p1 = t.end - 1;
        t.first_step = t.sink_steps = 0;
        t.steps = t.end / kStep;
        t.carried = false;
        return t;
    } else {
        const int b = plan.row_tiles == 1 ? pair : pair / plan.row_tiles, len = length_of(a, b);
        return make_tile(a, plan, len, plan.row_tiles == 1 ? 0 : pair % plan.row_tiles,
                         P == kRest ? carried_tokens(a, b, len) : 0);
    }
}
// What an item takes of the list of all items' steps: its cost first.
template <Part P>
__device__ __forceinline__ int span_of(const Plan& plan, const Tile& tile) {
    return P == kPrefix && tile.steps == 0 ? 0 : tile.steps + plan.item_cost;
}

__device__ __forceinline__ uint32_t half2_bits(float lo, float hi) {
    const __half2 h = __floats2half2_rn(lo, hi);
    return *reinterpret_cast<const uint32_t*>(&h);
}
// 16 bytes, zeros unless real.
__device__ __forceinline__ void copy_async(uint32_t dst, const void* src, bool real) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(real ? 16u : 0u)
                 : "memory");
}
__device__ __forceinline__ void copy_async4(uint32_t dst, const void* src, bool real) {
    asm volatile("cp.async.ca.shared.global [%0], [%1], 4, %2;" ::"r"(dst), "l"(src), "r"(real ? 4u : 0u) : "memory");
}
template <int N>
__device__ __forceinline__ void copy_wait() {
    asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}
__device__ __forceinline__ void copy_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }

// 0x7f in each byte that holds a NaN code, else 0.
__device__ __forceinline__ uint32_t nan_bytes(uint32_t w) {
    return __vcmpeq4(w & 0x7f7f7f7fu, 0x7f7f7f7fu);
}

// Steps of an item at most.
inline int64_t most_steps(const CacheAttention& a) {
    const int64_t held = ((int64_t)a.table_pages << a.page_shift) / kStep;
    if (a.window == 0) return held;
    const int64_t seen = (a.window < INT_MAX ? a.window + a.T_q : INT_MAX) / kStep + 2 + (a.sinks + (int64_t)kStep - 1) / kStep;
    return seen < held ? seen : held;
}

// kRest: the steps that sequences are taken to have beyond their prefix, by the widths of the two tables (all of them,
// where these say nothing).  Whether items are cut, and which kernel takes them, goes by it.
inline int64_t rest_steps(const CacheAttention& a) {
    const int64_t rest = (int64_t)(a.table_pages > a.prefix_pages ? a.table_pages - a.prefix_pages : a.table_pages);
    return (rest << a.page_shift) / kStep;
}

// Whether one CTA an item is faster than equal shares of all items' steps.  Cutting costs each CTA a second start and
// end and a kernel that joins, together the time of `cutting` steps; whole items cost what the longest takes beyond
// the average load of the CTAs, where lengths are even from 0 to the longest: cap - items cap / (2 ctas) steps.
// No length is known here, only what the block table can hold, so that one long sequence among short ones is not cut then:
// up to `longest` steps.
inline bool whole_items_pay(int64_t cap, int64_t items, int64_t ctas, int64_t cutting, int64_t longest) {
    return cap <= longest && cap * (2 * ctas - items) <= 2 * ctas * cutting;
}

// A CTA's share of the list of all items' steps: [begin, end), which starts in pair `pair`
// (-1: nothing), whose first head begins at `base`.
struct Share {
    int64_t begin, end, share, base;
    int pair;
};

// Every thread of the CTA calls it; each sums up some pairs' steps.
template <int THREADS, Part P = kAll>
__device__ __forceinline__ Share find_share(const CacheAttention& a, const Plan& plan) {
    __shared__ int64_t warp_sum_s[THREADS / 32];
    __shared__ int64_t found_base;
    __shared__ int found_pair;
    const int pairs = P == kPrefix ? plan.pairs : a.B * plan.row_tiles;
    const int each = (pairs + THREADS - 1) / THREADS;
    const int q0 = threadIdx.x * each;
    int64_t mine = 0;
    for (int q = q0; q < q0 + each && q < pairs; ++q) mine += span_of<P>(plan, tile_of<P>(a, plan, q));
    int64_t before = mine;                                 // steps of one head, up to this thread's end
#pragma unroll
    for (int w = 1; w < 32; w <<= 1) {
        const int64_t x = __shfl_up_sync(0xffffffffu, before, w);
        if ((threadIdx.x & 31) >= w) before += x;
    }
    if ((threadIdx.x & 31) == 31) warp_sum_s[threadIdx.x >> 5] = before;
    if (threadIdx.x == 0) found_pair = -1;
    __syncthreads();
    int64_t total = 0;
#pragma unroll
    for (int w = 0; w < THREADS / 32; ++w) {
        if (w < (int)(threadIdx.x >> 5)) before += warp_sum_s[w];
        total += warp_sum_s[w];
    }
    before = (before - mine) * a.H_kv;
    total *= a.H_kv;
    Share s;
    s.share = (total + gridDim.x - 1) / gridDim.x;
    if (s.share < kMinShare) s.share = kMinShare;
    s.begin = s.share * blockIdx.x;
    s.end = s.begin + s.share < total ? s.begin + s.share : total;
    if (s.begin >= before && s.begin < before + mine * a.H_kv) {
        int64_t base = before;
        for (int q = q0; q < pairs; ++q) {
            // (its only pair: the one that its sum says)
            const int64_t w = each == 1 ? mine * a.H_kv : (int64_t)a.H_kv * span_of<P>(plan, tile_of<P>(a, plan, q));
            if (s.begin < base + w) {
                found_pair = q;
                found_base = base;
                break;
            }
            base += w;
        }
    }
    __syncthreads();
    s.pair = found_pair;
    s.base = found_base;
    return s;
}

// Calls f(pair, head, tile, from, to, slot, whole) for each piece of the share: steps [from, to) of
// an item; `whole` where that is all of it, else its sums go to the CTA's slot.  Returns the
// entry of `joins` for the item that begins here and ends in a later share.
template <Part P = kAll, typename F>
__device__ __forceinline__ int4 for_each_piece(const CacheAttention& a, const Plan& plan, const Share& s, F f) {
    int4 join = make_int4(-1, 0, 0, 0);
    if (s.pair < 0) return join;
    int pair = s.pair;
    int64_t base = s.base, at = s.begin;
    Tile tile = tile_of<P>(a, plan, pair);
    int span = span_of<P>(plan, tile);                     // of an item in the list
    int hk = (int)((s.begin - base) / span);
    base += (int64_t)hk * span;                            // where the item begins
    auto step_at = [&](int64_t x) {
        const int step = x - base > plan.item_cost ? (int)(x - base) - plan.item_cost : 0;
        return step == tile.steps ? step : step - step % plan.cut;
    };
    while (at < s.end) {
        const int64_t item_end = base + span;
        const int64_t stop = item_end < s.end ? item_end : s.end;
        const int from = step_at(at), to = step_at(stop);
        if (from < to) {
            const bool whole = from == 0 && to == tile.steps;
            const int slot = at == s.begin ? 0 : 1;
            f(pair, hk, tile, from, to, slot, whole);
            if (!whole && from == 0) join = make_int4(pair, hk, (int)((item_end - 1) / s.share), slot);
        }
        at = stop;
        base = item_end;
        if (++hk == a.H_kv && at < s.end) {
            hk = 0;
            do {
                ++pair;
                tile = tile_of<P>(a, plan, pair);
                span = span_of<P>(plan, tile);
            } while (P == kPrefix && span == 0);           // (the share goes on: there is one)
        }
    }
    return join;
}

// Row r of a tile, as a row of o and lse.
template <Part P = kAll>
__device__ __forceinline__ int64_t output_row(const CacheAttention& a, const Plan& plan, int b, int hk, int rt,
                                              int r) {
    const int row = rt * plan.tile_rows + r, i = row / plan.group;
    return (first_query<P>(a, b) + i) * a.H_q + hk * plan.group + row - i * plan.group;
}
__device__ __forceinline__ int rows_of_tile(const Plan& plan, int rt) {
    const int n = plan.rows - rt * plan.tile_rows;
    return n < plan.tile_rows ? n : plan.tile_rows;
}
template <Part P>
__device__ __forceinline__ int rows_of_tile(const CacheAttention& a, const Plan& plan, int b, int rt) {
    const int n = item_rows<P>(a, plan, b) - rt * plan.tile_rows;
    return n < plan.tile_rows ? n : plan.tile_rows;
}

// A row's sums of v, in units of 2^(m - dm - kWeightBits), become outputs by this factor.
__device__ __forceinline__ float row_factor(float DM, float L) {
    return L == 0.0f ? 0.0f : ex2(-DM - kWeightBits) / L;
}
__device__ __forceinline__ float row_lse(float M, float L) {
    return L == 0.0f ? -INFINITY : (M + log2f(L)) * 0.6931471805599453f;
}
// Channels ch .. ch + 3 of an output row.
template <typename T>
__device__ __forceinline__ void write_row(const CacheAttention& a, int64_t row, int ch, float4 o, float M,
                                          float DM, float L) {
    const float f = row_factor(DM, L);
    if (L == 0.0f) o = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
    if (ch < a.d) {
        T* to = static_cast<T*>(a.o) + row * a.d + ch;
        if constexpr (sizeof(T) == 2)
            *reinterpret_cast<uint2*>(to) =
                make_uint2(tc::pack_bf16x2(o.x * f, o.y * f), tc::pack_bf16x2(o.z * f, o.w * f));
        else
            *reinterpret_cast<float4*>(to) = make_float4(o.x * f, o.y * f, o.z * f, o.w * f);
    }
    if (ch == 0 && a.lse) a.lse[row] = row_lse(M, L);
}

// Sums (m, dm, l; o, four channels) and the sums (s; x) of other tokens: o becomes both's, (M, DM, L) their statistics.
__device__ __forceinline__ void join_sums(float4& o, float& M, float& DM, float& L, const float4& s, const float4& x) {
    const float m = fmaxf(M, s.x), dm = fminf(DM + (m - M), s.y + (m - s.x));
    const float keep = ex2(M - m + (dm - DM)), add = ex2(s.x - m + (dm - s.y));
    L = L * ex2(M - m) + s.z * ex2(s.x - m);
    o = make_float4(o.x * keep + x.x * add, o.y * keep + x.y * add, o.z * keep + x.z * add, o.w * keep + x.w * add);
    M = m;
    DM = dm;
}
// What becomes of a finished row's sums: outputs (kRest: with what the row carries), or (kPrefix) what it carries.
template <typename T, Part P, int D>
__device__ __forceinline__ void finish_row(const CacheAttention& a, int64_t row, int ch, float4 o, float M, float DM, float L,
                                           bool carried) {
    if constexpr (P == kPrefix) {
        *reinterpret_cast<float4*>(a.carry_sums + row * D + ch) = o;
        if (ch == 0) a.carry_stats[row] = make_float4(M, DM, L, 0.0f);
    } else {
        if (P == kRest && carried)
            join_sums(o, M, DM, L, a.carry_stats[row], *reinterpret_cast<const float4*>(a.carry_sums + row * D + ch));
        write_row<T>(a, row, ch, o, M, DM, L);
    }
}

}  // namespace attn

// Bytes of the pieces' sums behind `grid` CTAs, their division into plan.joins, stats and sums,
// and the kernel that joins them after one that wrote them.
size_t attention_piece_bytes(int64_t grid, int stored, int D);
void set_attention_pieces(attn::Plan& plan, void* workspace, int64_t grid);
cudaError_t run_attention_join(const CacheAttention& a, const attn::Plan& plan, bool bf16, int D, int64_t grid,
                               cudaStream_t stream);
cudaError_t run_attention_join_rest(const CacheAttention& a, const attn::Plan& plan, bool bf16, int D, int64_t grid,
                                    cudaStream_t stream);

// The kernels for few rows, by what they attend over (one source file each, so that they compile side by side).
size_t attention_rows_workspace_bytes(const CacheAttention& a, int num_sms);
size_t attention_rest_rows_workspace_bytes(const CacheAttention& a, int num_sms);
size_t attention_prefix_rows_workspace_bytes(const CacheAttention& a, int num_sms);
cudaError_t run_attention_rows(const CacheAttention& a, bool bf16, void* workspace, cudaStream_t stream, int num_sms);
cudaError_t run_attention_rest_rows(const CacheAttention& a, bool bf16, void* workspace, cudaStream_t stream, int num_sms);
cudaError_t run_attention_prefix_rows(const CacheAttention& a, bool bf16, void* workspace, cudaStream_t stream, int num_sms);

// What kda_selftest_attention_stall has set on this thread.
attn::Stall attention_stall();

// The kernel for the prefixes of bf16 rows (kda_cache_prefix_tc.cu).
size_t attention_prefix_tc_workspace_bytes(const CacheAttention& a, int num_sms);
cudaError_t run_attention_prefix_tc(const CacheAttention& a, void* workspace, cudaStream_t stream, int num_sms);

// The kernel for many bf16 rows (kda_cache_attention_tc.cu): its plan for these queries, how many CTAs share
// the work out (0: each item is one CTA's), and the launch.
bool attention_tc_takes(const CacheAttention& a, bool bf16);
attn::Plan attention_tc_plan(const CacheAttention& a);
int64_t attention_tc_grid(const CacheAttention& a, const attn::Plan& plan, int num_sms, attn::Part part = attn::kAll);
cudaError_t run_attention_tc(const CacheAttention& a, void* workspace, cudaStream_t stream, int num_sms);
cudaError_t run_attention_tc_rest(const CacheAttention& a, void* workspace, cudaStream_t stream, int num_sms);

}  // namespace kda
