// kda_cache_attention.cu -- attention of a sequence's newest tokens over the paged 8-bit cache.
//
// Row (b, i, h) is query head h of the i-th of T_q newest tokens; its position is
// p = lengths[b] - T_q + i and its keys are those of head h / (H_q / H_kv).  It sees
// token t if t <= p, t < sinks or t > p - window, and t's page is held:
//
//   s_t = scale q.k_t,   o = sum_t e^(s_t - m) v_t / sum_t e^(s_t - m),   m = max_t s_t
//
// one pass over the tokens with the running maximum and sum.  A row that sees
// nothing, or whose scores are all -inf, gives zeros and lse = -inf.
//
// What bounds it: reading the codes, as long as the rows that share a head's
// keys (T_q times H_q / H_kv) are few; the products' rate beyond some 32 rows.
//
// The tile.  16 rows x 16 tokens a step, on m16n8k16 products of fp16 with fp32
// sums: e4m3 codes are exact in fp16, and so are a page's scale (applied to
// the scores after the product, to the weights before it) and bf16 queries, once a
// power of two has brought their row under fp16's largest value.  fp32 queries
// and their weights go as two fp16 pieces (22 bits), two products instead of one.
// No operand passes through shared memory to change hands: the pairing of a
// product's k index with channels, of its n index with channels of v, is free, so
// each lane reads its own 16 consecutive bytes of a token's row, as they lie
// in the cache, and its words are the fragments; the scores' fragments are the
// weights' fragments.  Every lane copies what it will read itself (16-byte
// asynchronous copies into its own slots, three steps ahead), so a warp runs
// without a barrier; with more than 16 rows, MT warps share one ring of slots and
// one barrier a step.
//
// The work.  The lengths are on the device, so the host cannot cut the work up.
// All steps of all (sequence, row tile, head) items are one list, cut into equal
// shares, one for each of a fixed number of CTAs; each finds its place by
// summing the lengths.  An item that lies within one share is finished there; pieces of
// the others are left in the workspace (fp32 sums with their maxima), at most
// two a CTA, and a second small kernel joins them in a fixed order, so that
// the same call gives the same bits.  Where one CTA takes any item whole
// (short tables, or very many row tiles) there is no second kernel.
//
// V's scale.  The weights are e^(s - m) times the page's scale of v, whose range
// is far beyond fp16's.  So the sums of v have a reference of their own, mo = max(s
// + log2 scale), beside the maximum m that the sum of weights has; weights go
// to fp16 as 2^(s + log2 scale - mo + 12), at most 2^13, with full precision down to
// 2^-26 of the largest.
//
// NaN that a row does not see.  0 times NaN is NaN, so tokens past the last that
// any row of the tile sees are never copied (zeros instead), and a step that
// some rows see and others do not is looked through for NaN codes of v: if there are
// any they count as zeros, and a product of the rows' sight with the places of
// the NaN marks the outputs that they do reach.
#include <climits>

#include "kda_cache.cuh"
#include "kda_internal.h"
#include "tc_util.cuh"

namespace kda {
namespace {

constexpr int kWarps = 4;
constexpr int kThreads = 32 * kWarps;
constexpr int kStep = 16;             // tokens of a step
constexpr int kMinShare = 8;          // steps below which no item is cut further
constexpr int kJoinThreads = 256;
constexpr int kMaxScan = 8192;        // (sequence, row tile) pairs that every CTA sums up
constexpr float kWeightBits = 12.0f;

struct Plan {
    int group;          // query heads of a head of keys
    int rows;           // T_q * group
    int row_tiles;
    int stored;         // rows of a tile that exist: min(rows, 16 MT)
    float* sums;        // [grid][2][stored][D]
    float4* stats;      // [grid][2][stored]: m, mo, l
    int4* joins;        // [grid]: pair (sequence, row tile), head, last CTA, slot; pair < 0: none
};

// What a row tile of a sequence sees, in steps.
struct Tile {
    int p0, p1;         // positions of its first and last row
    int end;            // tokens [0, end) at most
    int first_step;     // of the window (or 0), after sink_steps steps from 0
    int sink_steps;
    int steps;          // at least 1, so that a row that sees nothing is written too
    __device__ __forceinline__ int token(int s) const {
        return (s < sink_steps ? s : first_step + s - sink_steps) * kStep;
    }
};

template <int ROWS>
__device__ __forceinline__ Tile make_tile(const CacheAttention& a, const Plan& plan, int len, int rt) {
    Tile t;
    const int r0 = rt * ROWS;
    const int r1 = (plan.rows < r0 + ROWS ? plan.rows : r0 + ROWS) - 1;
    t.p0 = len - a.T_q + r0 / plan.group;
    t.p1 = len - a.T_q + r1 / plan.group;
    t.end = t.p1 + 1 > 0 ? t.p1 + 1 : 0;
    int lo = 0, sink_end = 0;
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
__device__ __forceinline__ float quad_max(float x) {
    x = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, 1));
    return fmaxf(x, __shfl_xor_sync(0xffffffffu, x, 2));
}
__device__ __forceinline__ float quad_sum(float x) {
    x += __shfl_xor_sync(0xffffffffu, x, 1);
    return x + __shfl_xor_sync(0xffffffffu, x, 2);
}
__device__ __forceinline__ float or_zero(float m) { return m == -INFINITY ? 0.0f : m; }

__device__ __forceinline__ uint32_t half2_bits(float lo, float hi) {
    const __half2 h = __floats2half2_rn(lo, hi);
    return *reinterpret_cast<const uint32_t*>(&h);
}
// What half2_bits lost of (lo, hi).
__device__ __forceinline__ uint32_t half2_rest(float lo, float hi, uint32_t bits) {
    const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&bits));
    return half2_bits(lo - f.x, hi - f.y);
}

// The two fp16 pairs of a word of four codes.
__device__ __forceinline__ void word_to_half2x2(uint32_t w, uint32_t& lo, uint32_t& hi) {
    asm("{\n\t.reg .b16 l, h;\n\tmov.b32 {l, h}, %2;\n\t"
        "cvt.rn.f16x2.e4m3x2 %0, l;\n\tcvt.rn.f16x2.e4m3x2 %1, h;\n\t}"
        : "=r"(lo), "=r"(hi)
        : "r"(w));
}

// c += a b: a is 16 x 16 (rows g and g + 8; k 2c, 2c + 1, then 8 more), b 16 x 8
// (n = g), c 16 x 8 (rows g and g + 8, n 2c and 2c + 1), of lane 4 g + c.
__device__ __forceinline__ void mma16816(float (&c)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, "
        "{%0,%1,%2,%3};"
        : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

template <int BYTES>
__device__ __forceinline__ void copy_async(uint32_t dst, const void* src, bool real) {
    const uint32_t n = real ? BYTES : 0;
    if constexpr (BYTES == 16)
        asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(n) : "memory");
    else
        asm volatile("cp.async.ca.shared.global [%0], [%1], %2, %3;" ::"r"(dst), "l"(src), "n"(BYTES), "r"(n)
                     : "memory");
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

// The sizes that go together: MT warps share the tokens of their 16 MT rows,
// NG groups of them take steps in turn, each with a ring of STAGES steps.
template <typename T, int D, int MT>
struct Shape {
    static constexpr int NG = kWarps / MT;
    static constexpr int ROWS = 16 * MT;
    static constexpr int STAGES = MT == 1 ? 4 : MT == 2 ? 6 : 8;
    static constexpr int KC = D / 64;                 // 16-byte pieces of a key that a lane reads
    static constexpr int VB = D / 8;                  // bytes of a value that a lane reads
    static constexpr int K_BYTES = 2 * KC * 512;      // of a step: 16 keys
    static constexpr int STAGE = K_BYTES + 4 * 32 * VB + 16;   // + the two scales
    static constexpr int RING = NG * STAGES * STAGE;
    static constexpr int JOIN = NG * ROWS * (D + 4) * 4 + NG * ROWS * 16;
    static constexpr int SMEM = RING > JOIN ? RING : JOIN;
    static constexpr int PIECES = sizeof(T) == 4 ? 2 : 1;   // fp16 pieces of a query and a weight
    static constexpr int CTAS = PIECES == 1 ? 3 : 2;        // resident a SM
};

// One piece of an item: steps [from, to) of a tile's `steps`.
template <typename T, int D, int MT>
struct Piece {
    using S = Shape<T, D, MT>;
    const CacheAttention& a;
    const Plan& plan;
    uint8_t* smem;
    int b, hk, rt, from, to;
    Tile tile;

    __device__ __forceinline__ void run(int cta, int slot, bool whole) {
        const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
        const int g = lane >> 2, c = lane & 3;
        const int grp = warp / MT, wt = warp % MT;
        uint8_t* ring = smem + grp * S::STAGES * S::STAGE;
        const uint32_t ring_u = tc::smem_u32(ring);
        const int d = a.d;
        const int32_t* table = a.table + (int64_t)b * a.table_pages;
        const int page_mask = (1 << a.page_shift) - 1;

        auto page_at = [&](int s) -> int {
            const int t = tile.token(s);
            if (s >= to || t >= tile.end) return -1;
            return __ldg(table + (t >> a.page_shift));
        };
        // Copies step s (its page's id is pg) into stage st.
        auto issue = [&](int s, int pg, int st) {
            const uint32_t stage = ring_u + st * S::STAGE;
            const uint32_t scales = stage + S::STAGE - 16;
            if (pg >= 0 && pg < a.n_pages) {
                const int t0 = tile.token(s);
                const int64_t block = (int64_t)pg * a.H_kv + hk;
                const int64_t at = ((block << a.page_shift) + (t0 & page_mask)) * d;
                const uint8_t* k = a.k_codes + at;
                const uint8_t* v = a.v_codes + at;
                const int n = tile.end - t0;               // tokens of the step that exist
#pragma unroll
                for (int i = 0; i < 2 * S::KC; ++i)
                    if (MT == 1 || i % MT == wt) {
                        const int token = 8 * (i / S::KC) + g, byte = 64 * (i % S::KC) + 16 * c;
                        const bool real = token < n && byte < d;
                        copy_async<16>(stage + i * 512 + lane * 16, real ? k + token * d + byte : a.k_codes,
                                       real);
                    }
#pragma unroll
                for (int i = 0; i < 4; ++i)
                    if (MT == 1 || i % MT == wt) {
                        const int token = 8 * (i / 2) + 2 * c + (i & 1), byte = S::VB * g;
                        const bool real = token < n && byte < d;
                        copy_async<S::VB>(stage + S::K_BYTES + i * 32 * S::VB + lane * S::VB,
                                          real ? v + token * d + byte : a.v_codes, real);
                    }
                if (wt == 0 && lane < 2)
                    copy_async<4>(scales + 4 * lane, (lane ? a.v_scale : a.k_scale) + block, true);
            } else if (wt == 0 && lane < 2) {
                asm volatile("st.shared.b32 [%0], %1;" ::"r"(scales + 4 * lane), "r"(0) : "memory");
            }
            copy_commit();
        };

        const int s0 = from + grp;
        {
            int pg[S::STAGES - 1];
#pragma unroll
            for (int i = 0; i < S::STAGES - 1; ++i) pg[i] = page_at(s0 + i * S::NG);
#pragma unroll
            for (int i = 0; i < S::STAGES - 1; ++i) issue(s0 + i * S::NG, pg[i], i);
        }
        int next_page = page_at(s0 + (S::STAGES - 1) * S::NG);

        // Queries: rows ra and rb of this lane, 16 channels from 64 j + 16 c on.
        const int r_local[2] = {wt * 16 + g, wt * 16 + g + 8};
        uint32_t qf[S::PIECES][4 * S::KC][4];
        float factor[2];
        int pos[2];
#pragma unroll
        for (int r = 0; r < 2; ++r) {
            const int row = rt * S::ROWS + r_local[r];
            const bool real = row < plan.rows;
            const int i = real ? row / plan.group : 0;
            pos[r] = real ? tile.p0 - rt * S::ROWS / plan.group + i : -1;
            const T* q = static_cast<const T*>(a.q) + ((int64_t)b * a.T_q + i) * a.q_stride +
                         (int64_t)(hk * plan.group + (real ? row - i * plan.group : 0)) * d;
            float x[S::KC][16];
            float amax = 0.0f;
#pragma unroll
            for (int j = 0; j < S::KC; ++j) {
                uint4 raw[sizeof(T)];
                const bool in = real && 64 * j + 16 * c < d;
#pragma unroll
                for (int w = 0; w < (int)sizeof(T); ++w)
                    raw[w] = in ? __ldg(reinterpret_cast<const uint4*>(q + 64 * j + 16 * c) + w)
                                : make_uint4(0, 0, 0, 0);
                const T* e = reinterpret_cast<const T*>(raw);
#pragma unroll
                for (int w = 0; w < 16; ++w) {
                    x[j][w] = to_f32(e[w]);
                    amax = fmaxf(amax, finite_abs(x[j][w]));
                }
            }
            amax = quad_max(amax);
            // 2^ex <= amax < 2^(ex + 1): times 2^(14 - ex), under fp16's largest value
            int ex = (int)(__float_as_uint(amax) >> 23) - 127;
            ex = ex < -112 ? -112 : ex;
            const float up = __uint_as_float((uint32_t)(127 + 14 - ex) << 23);
            factor[r] = a.scale * 1.4426950408889634f * __uint_as_float((uint32_t)(127 + ex - 14) << 23);
#pragma unroll
            for (int j = 0; j < S::KC; ++j)
#pragma unroll
                for (int w = 0; w < 4; ++w)
#pragma unroll
                    for (int h = 0; h < 2; ++h) {
                        const float lo = x[j][4 * w + 2 * h] * up, hi = x[j][4 * w + 2 * h + 1] * up;
                        const uint32_t bits = half2_bits(lo, hi);
                        qf[0][4 * j + w][2 * h + r] = bits;
                        if constexpr (S::PIECES == 2) qf[1][4 * j + w][2 * h + r] = half2_rest(lo, hi, bits);
                    }
        }

        float acc[S::VB][4];
#pragma unroll
        for (int n = 0; n < S::VB; ++n)
#pragma unroll
            for (int w = 0; w < 4; ++w) acc[n][w] = 0.0f;
        float m[2] = {-INFINITY, -INFINITY}, mo[2] = {-INFINITY, -INFINITY}, l[2] = {0.0f, 0.0f};

        int st = 0;
        for (int s = s0; s < to; s += S::NG) {
            copy_wait<S::STAGES - 2>();
            if constexpr (MT == 1) __syncwarp();
            else tc::named_bar_sync(1 + grp, 32 * MT);
            const uint8_t* stage = ring + st * S::STAGE;
            const float2 scales = *reinterpret_cast<const float2*>(stage + S::STAGE - 16);
            {
                const int ahead = s + (S::STAGES - 1) * S::NG;
                const int into = st == 0 ? S::STAGES - 1 : st - 1;
                issue(ahead, next_page, into);
                next_page = page_at(ahead + S::NG);
            }
            st = st == S::STAGES - 1 ? 0 : st + 1;
            if (scales.y == 0.0f) continue;                // a page that is not held

            float sc[2][4];
#pragma unroll
            for (int t = 0; t < 2; ++t) {
#pragma unroll
                for (int w = 0; w < 4; ++w) sc[t][w] = 0.0f;
#pragma unroll
                for (int j = 0; j < S::KC; ++j) {
                    const uint4 raw = *reinterpret_cast<const uint4*>(stage + (t * S::KC + j) * 512 + lane * 16);
                    const uint32_t word[4] = {raw.x, raw.y, raw.z, raw.w};
#pragma unroll
                    for (int w = 0; w < 4; ++w) {
                        uint32_t b0, b1;
                        word_to_half2x2(word[w], b0, b1);
#pragma unroll
                        for (int pc = 0; pc < S::PIECES; ++pc) mma16816(sc[t], qf[pc][4 * j + w], b0, b1);
                    }
                }
            }
            const float f0 = factor[0] * scales.x, f1 = factor[1] * scales.x;
#pragma unroll
            for (int t = 0; t < 2; ++t) {
                sc[t][0] *= f0;
                sc[t][1] *= f0;
                sc[t][2] *= f1;
                sc[t][3] *= f1;
            }
            const int t0 = tile.token(s);
            const bool partly = t0 + kStep - 1 > tile.p0 ||
                                (a.window > 0 && t0 <= tile.p1 - a.window && t0 + kStep - 1 >= a.sinks);
            uint32_t sight = 0xffu;                        // bit 4 t + w: sc[t][w] is seen
            if (partly) {
                sight = 0;
#pragma unroll
                for (int t = 0; t < 2; ++t)
#pragma unroll
                    for (int w = 0; w < 4; ++w) {
                        const int at = t0 + 8 * t + 2 * c + (w & 1), p = pos[w >> 1];
                        const bool sees = at <= p && (a.window == 0 || at > p - a.window || at < a.sinks);
                        if (sees) sight |= 1u << (4 * t + w);
                        else sc[t][w] = -INFINITY;
                    }
            }
            // log2 of v's scale: its exponent, and what remains (1 for these pages' powers of two)
            const float e = (float)((int)(__float_as_uint(scales.y) >> 23) - 127);
            const float mantissa = __uint_as_float((__float_as_uint(scales.y) & 0x7fffffu) | 0x3f800000u);
            uint32_t pf[S::PIECES][4];
            float keep[2];
            bool moved = false;
#pragma unroll
            for (int r = 0; r < 2; ++r) {
                const float top = quad_max(fmaxf(fmaxf(sc[0][2 * r], sc[0][2 * r + 1]),
                                                 fmaxf(sc[1][2 * r], sc[1][2 * r + 1])));
                const float m_new = fmaxf(m[r], top), mo_new = fmaxf(mo[r], top + e);
                const float ref = or_zero(m_new), oref = or_zero(mo_new);
                keep[r] = ex2(mo[r] - oref);
                moved |= mo_new > mo[r];
                const float lift = ex2(fminf(ref + e - oref + kWeightBits, 126.0f)) * mantissa;
                float p[4];
#pragma unroll
                for (int w = 0; w < 4; ++w) p[w] = ex2(sc[w >> 1][2 * r + (w & 1)] - ref);
                l[r] = l[r] * ex2(m[r] - ref) + ((p[0] + p[1]) + (p[2] + p[3]));
                m[r] = m_new;
                mo[r] = mo_new;
#pragma unroll
                for (int t = 0; t < 2; ++t) {
                    const float lo = p[2 * t] * lift, hi = p[2 * t + 1] * lift;
                    const uint32_t bits = half2_bits(lo, hi);
                    pf[0][2 * t + r] = bits;
                    if constexpr (S::PIECES == 2) pf[1][2 * t + r] = half2_rest(lo, hi, bits);
                }
            }
            if (__any_sync(0xffffffffu, moved)) {
#pragma unroll
                for (int n = 0; n < S::VB; ++n) {
                    acc[n][0] *= keep[0];
                    acc[n][1] *= keep[0];
                    acc[n][2] *= keep[1];
                    acc[n][3] *= keep[1];
                }
            }
            // Values: four tokens' words; a product's b pairs two tokens of one channel.
            const uint8_t* vs = stage + S::K_BYTES + lane * S::VB;
            bool nan_here = false;
            if (partly) {
#pragma unroll
                for (int i = 0; i < 4; ++i)
#pragma unroll
                    for (int w = 0; w < S::VB / 4; ++w)
                        nan_here |= nan_bytes(*reinterpret_cast<const uint32_t*>(vs + i * 32 * S::VB + 4 * w)) != 0;
                nan_here = __any_sync(0xffffffffu, nan_here);
            }
            if (!nan_here) {
#pragma unroll
                for (int w = 0; w < S::VB / 4; w += 2) {
                    uint2 two[4];
#pragma unroll
                    for (int i = 0; i < 4; ++i)
                        two[i] = *reinterpret_cast<const uint2*>(vs + i * 32 * S::VB + 4 * w);
#pragma unroll
                    for (int x = 0; x < 2; ++x) {
                        const uint32_t v0 = x ? two[0].y : two[0].x, v1 = x ? two[1].y : two[1].x;
                        const uint32_t v2 = x ? two[2].y : two[2].x, v3 = x ? two[3].y : two[3].x;
                        add_values(acc, 4 * (w + x), pf, v0, v1, v2, v3);
                    }
                }
            } else {
                uint32_t seen[4];                          // the rows' sight as a fragment of ones
#pragma unroll
                for (int t = 0; t < 2; ++t)
#pragma unroll
                    for (int r = 0; r < 2; ++r)
                        seen[2 * t + r] = (sight >> (4 * t + 2 * r) & 1 ? 0x3c00u : 0u) |
                                          (sight >> (4 * t + 2 * r + 1) & 1 ? 0x3c000000u : 0u);
#pragma unroll
                for (int w = 0; w < S::VB / 4; ++w) {
                    uint32_t v[4], bad[4];
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        v[i] = *reinterpret_cast<const uint32_t*>(vs + i * 32 * S::VB + 4 * w);
                        bad[i] = nan_bytes(v[i]);
                        v[i] &= ~bad[i];
                        bad[i] &= 0x38383838u;             // 1 in e4m3
                    }
                    add_values(acc, 4 * w, pf, v[0], v[1], v[2], v[3]);
                    float hit[4][4] = {};
                    uint32_t ones[1][4] = {{seen[0], seen[1], seen[2], seen[3]}};
                    add_values<4, 1>(hit, 0, ones, bad[0], bad[1], bad[2], bad[3]);
#pragma unroll
                    for (int n = 0; n < 4; ++n)
#pragma unroll
                        for (int x = 0; x < 4; ++x)
                            if (hit[n][x] > 0.0f) acc[4 * w + n][x] = NAN;
                }
            }
        }
        copy_wait<0>();
        __syncthreads();                                   // the ring becomes the place to join in

        // Join the groups.  Lane (g, c) holds channels [2 c VB, 2 (c + 1) VB) of its rows.
        float* o_s = reinterpret_cast<float*>(smem);
        float4* stat_s = reinterpret_cast<float4*>(smem + S::NG * S::ROWS * (D + 4) * 4);
#pragma unroll
        for (int r = 0; r < 2; ++r) {
            l[r] = quad_sum(l[r]);
            if (r_local[r] >= plan.stored) continue;
            float* to_s = o_s + (grp * S::ROWS + r_local[r]) * (D + 4) + 2 * c * S::VB;
#pragma unroll
            for (int h = 0; h < 2; ++h)
#pragma unroll
                for (int n = 0; n < S::VB; n += 4)
                    *reinterpret_cast<float4*>(to_s + h * S::VB + n) =
                        make_float4(acc[n][2 * r + h], acc[n + 1][2 * r + h], acc[n + 2][2 * r + h],
                                    acc[n + 3][2 * r + h]);
            if (c == 0) stat_s[grp * S::ROWS + r_local[r]] = make_float4(m[r], mo[r], l[r], 0.0f);
        }
        __syncthreads();
        const int rows_here = plan.rows - rt * S::ROWS < S::ROWS ? plan.rows - rt * S::ROWS : S::ROWS;
        for (int u = threadIdx.x; u < rows_here * (D / 4); u += kThreads) {
            const int r = u / (D / 4), ch = u % (D / 4) * 4;
            float M = -INFINITY, MO = -INFINITY, L = 0.0f;
            float4 stat[S::NG];
#pragma unroll
            for (int i = 0; i < S::NG; ++i) {
                stat[i] = stat_s[i * S::ROWS + r];
                M = fmaxf(M, stat[i].x);
                MO = fmaxf(MO, stat[i].y);
            }
            float4 o = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
#pragma unroll
            for (int i = 0; i < S::NG; ++i) {
                L += stat[i].z * ex2(stat[i].x - or_zero(M));
                const float f = ex2(stat[i].y - or_zero(MO));
                const float4 x = *reinterpret_cast<const float4*>(o_s + (i * S::ROWS + r) * (D + 4) + ch);
                o.x += f * x.x;
                o.y += f * x.y;
                o.z += f * x.z;
                o.w += f * x.w;
            }
            if (whole) {
                const int row = rt * S::ROWS + r, i = row / plan.group;
                write_row<T>(a, ((int64_t)b * a.T_q + i) * a.H_q + hk * plan.group + row - i * plan.group, ch, o,
                             M, MO, L);
            } else {
                const int64_t at = ((int64_t)cta * 2 + slot) * plan.stored + r;
                *reinterpret_cast<float4*>(plan.sums + at * D + ch) = o;
                if (ch == 0) plan.stats[at] = make_float4(M, MO, L, 0.0f);
            }
        }
        __syncthreads();
    }

    // acc[n0 + x] += weights x channels n0 + x of four tokens, x = 0 .. 3.
    template <int N, int PCS>
    static __device__ __forceinline__ void add_values(float (&acc)[N][4], int n0, const uint32_t (&pf)[PCS][4],
                                                      uint32_t v0, uint32_t v1, uint32_t v2, uint32_t v3) {
        uint32_t b0[4], b1[4];
        word_to_half2x2(__byte_perm(v0, v1, 0x5140), b0[0], b0[1]);
        word_to_half2x2(__byte_perm(v0, v1, 0x7362), b0[2], b0[3]);
        word_to_half2x2(__byte_perm(v2, v3, 0x5140), b1[0], b1[1]);
        word_to_half2x2(__byte_perm(v2, v3, 0x7362), b1[2], b1[3]);
#pragma unroll
        for (int x = 0; x < 4; ++x)
#pragma unroll
            for (int pc = 0; pc < PCS; ++pc) mma16816(acc[n0 + x], pf[pc], b0[x], b1[x]);
    }

    template <typename U>
    static __device__ __forceinline__ void write_row(const CacheAttention& a, int64_t row, int ch, float4 o,
                                                     float M, float MO, float L) {
        const float f = L == 0.0f ? 0.0f : ex2(or_zero(MO) - or_zero(M) - kWeightBits) / L;
        if (L == 0.0f) o = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
        if (ch < a.d) {
            U* to = static_cast<U*>(a.o) + row * a.d + ch;
            if constexpr (sizeof(U) == 2) {
                const uint2 w = make_uint2(tc::pack_bf16x2(o.x * f, o.y * f), tc::pack_bf16x2(o.z * f, o.w * f));
                *reinterpret_cast<uint2*>(to) = w;
            } else {
                *reinterpret_cast<float4*>(to) = make_float4(o.x * f, o.y * f, o.z * f, o.w * f);
            }
        }
        if (ch == 0 && a.lse) a.lse[row] = L == 0.0f ? -INFINITY : (M + log2f(L)) * 0.6931471805599453f;
    }
};

// Every CTA one item: (sequence, row tile, head), heads innermost.
template <typename T, int D, int MT>
__global__ void __launch_bounds__(kThreads, Shape<T, D, MT>::CTAS)
attention_whole_kernel(const CacheAttention a, const Plan plan) {
    extern __shared__ __align__(16) uint8_t smem[];
    const int pair = blockIdx.x / a.H_kv, hk = blockIdx.x % a.H_kv;
    const int b = pair / plan.row_tiles, rt = pair % plan.row_tiles;
    const Tile tile = make_tile<16 * MT>(a, plan, length_of(a, b), rt);
    Piece<T, D, MT> piece{a, plan, smem, b, hk, rt, 0, tile.steps, tile};
    piece.run(0, 0, true);
}

// Every CTA an equal share of all items' steps.
template <typename T, int D, int MT>
__global__ void __launch_bounds__(kThreads, Shape<T, D, MT>::CTAS)
attention_share_kernel(const CacheAttention a, const Plan plan) {
    extern __shared__ __align__(16) uint8_t smem[];
    __shared__ int64_t warp_sum_s[kWarps];
    __shared__ int64_t found_base;
    __shared__ int found_pair;
    asm volatile("griddepcontrol.launch_dependents;");
    constexpr int ROWS = 16 * MT;
    const int pairs = a.B * plan.row_tiles;
    const int each = (pairs + kThreads - 1) / kThreads;
    const int q0 = threadIdx.x * each;
    int64_t mine = 0;
    for (int q = q0; q < q0 + each && q < pairs; ++q)
        mine += make_tile<ROWS>(a, plan, length_of(a, q / plan.row_tiles), q % plan.row_tiles).steps;
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
    for (int w = 0; w < kWarps; ++w) {
        if (w < (int)(threadIdx.x >> 5)) before += warp_sum_s[w];
        total += warp_sum_s[w];
    }
    before = (before - mine) * a.H_kv;
    total *= a.H_kv;
    int64_t share = (total + gridDim.x - 1) / gridDim.x;
    if (share < kMinShare) share = kMinShare;
    const int64_t begin = share * blockIdx.x;
    const int64_t end = begin + share < total ? begin + share : total;
    if (begin >= before && begin < before + mine * a.H_kv) {
        int64_t base = before;
        for (int q = q0; q < pairs; ++q) {
            const int64_t w = (int64_t)a.H_kv *
                make_tile<ROWS>(a, plan, length_of(a, q / plan.row_tiles), q % plan.row_tiles).steps;
            if (begin < base + w) {
                found_pair = q;
                found_base = base;
                break;
            }
            base += w;
        }
    }
    __syncthreads();
    int pair = found_pair;
    int4 join = make_int4(-1, 0, 0, 0);
    if (pair >= 0) {
        int64_t base = found_base, at = begin;
        Tile tile = make_tile<ROWS>(a, plan, length_of(a, pair / plan.row_tiles), pair % plan.row_tiles);
        int hk = (int)((begin - base) / tile.steps);
        base += (int64_t)hk * tile.steps;                  // where the item begins in the list
        while (at < end) {
            const int64_t item_end = base + tile.steps;
            const int64_t stop = item_end < end ? item_end : end;
            const bool whole = at == base && stop == item_end;
            const int slot = at == begin ? 0 : 1;
            Piece<T, D, MT> piece{a, plan, smem, pair / plan.row_tiles, hk, pair % plan.row_tiles,
                                  (int)(at - base), (int)(stop - base), tile};
            piece.run(blockIdx.x, slot, whole);
            if (!whole && at == base) join = make_int4(pair, hk, (int)((item_end - 1) / share), slot);
            at = stop;
            base = item_end;
            if (++hk == a.H_kv && at < end) {
                hk = 0;
                ++pair;
                tile = make_tile<ROWS>(a, plan, length_of(a, pair / plan.row_tiles), pair % plan.row_tiles);
            }
        }
    }
    if (threadIdx.x == 0) plan.joins[blockIdx.x] = join;
}

// The pieces of the item that begins in CTA blockIdx.x's share and ends in a later
// one, joined in order: the first from its slot, the later ones from slot 0.  A
// row a CTA at a time; eight warps take pieces in turn.
template <typename T, int D, int MT>
__global__ void __launch_bounds__(kJoinThreads)
attention_join_kernel(const CacheAttention a, const Plan plan) {
    constexpr int WARPS = kJoinThreads / 32, PER = D / 32;
    __shared__ float o_s[WARPS][D];
    __shared__ float l_s[WARPS];
    __shared__ float2 top_s[WARPS];
    asm volatile("griddepcontrol.wait;" ::: "memory");
    const int4 join = plan.joins[blockIdx.x];
    if (join.x < 0) return;
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int first = blockIdx.x, n = join.z - first + 1;
    const int b = join.x / plan.row_tiles, rt = join.x % plan.row_tiles;
    const int rows_here = plan.rows - rt * 16 * MT < 16 * MT ? plan.rows - rt * 16 * MT : 16 * MT;
    for (int r = blockIdx.y; r < rows_here; r += gridDim.y) {
        auto place = [&](int i) -> int64_t {
            return ((int64_t)(first + i) * 2 + (i == 0 ? join.w : 0)) * plan.stored + r;
        };
        float M = -INFINITY, MO = -INFINITY;
        for (int i = threadIdx.x; i < n; i += kJoinThreads) {
            const float4 s = plan.stats[place(i)];
            M = fmaxf(M, s.x);
            MO = fmaxf(MO, s.y);
        }
#pragma unroll
        for (int w = 16; w > 0; w >>= 1) {
            M = fmaxf(M, __shfl_xor_sync(0xffffffffu, M, w));
            MO = fmaxf(MO, __shfl_xor_sync(0xffffffffu, MO, w));
        }
        if (lane == 0) top_s[warp] = make_float2(M, MO);
        __syncthreads();
#pragma unroll
        for (int w = 0; w < WARPS; ++w) {
            M = fmaxf(M, top_s[w].x);
            MO = fmaxf(MO, top_s[w].y);
        }
        float o[PER] = {}, L = 0.0f;
#pragma unroll 4
        for (int i = warp; i < n; i += WARPS) {
            const int64_t at = place(i);
            const float4 s = plan.stats[at];
            const float f = ex2(s.y - or_zero(MO));
            L += s.z * ex2(s.x - or_zero(M));
#pragma unroll
            for (int x = 0; x < PER; ++x) o[x] += f * plan.sums[at * D + 32 * x + lane];
        }
#pragma unroll
        for (int x = 0; x < PER; ++x) o_s[warp][32 * x + lane] = o[x];
        if (lane == 0) l_s[warp] = L;
        __syncthreads();
        if (threadIdx.x < D / 4) {
            float4 sum = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
            L = 0.0f;
#pragma unroll
            for (int w = 0; w < WARPS; ++w) {
                const float4 x = *reinterpret_cast<const float4*>(&o_s[w][4 * threadIdx.x]);
                sum.x += x.x;
                sum.y += x.y;
                sum.z += x.z;
                sum.w += x.w;
                L += l_s[w];
            }
            const int row = rt * 16 * MT + r, i = row / plan.group;
            Piece<T, D, MT>::template write_row<T>(
                a, ((int64_t)b * a.T_q + i) * a.H_q + join.y * plan.group + row - i * plan.group,
                4 * threadIdx.x, sum, M, MO, L);
        }
        __syncthreads();
    }
}

int rows_of(const CacheAttention& a) { return a.T_q * (a.H_q / a.H_kv); }
// Row tiles of 16, of 32 (two warps share the tokens) or of 64 rows (four).
int tile_warps(const CacheAttention& a) { return rows_of(a) <= 16 ? 1 : rows_of(a) <= 32 ? 2 : 4; }
int padded_d(const CacheAttention& a) { return a.d <= 64 ? 64 : 128; }

// CTAs of the shared-out form; 0 where each item is one CTA's.
int64_t share_grid(const CacheAttention& a, int num_sms, int ctas) {
    const int mt = tile_warps(a);
    const int64_t row_tiles = (rows_of(a) + 16 * mt - 1) / (16 * mt);
    const int64_t cap = ((int64_t)a.table_pages << a.page_shift) / kStep;
    if (cap <= kMinShare || a.B * row_tiles > kMaxScan) return 0;
    const int64_t all = a.B * row_tiles * a.H_kv * cap;
    const int64_t most = (int64_t)num_sms * ctas, useful = (all + kMinShare - 1) / kMinShare;
    return useful < most ? useful : most;
}

template <typename T, int D, int MT>
cudaError_t launch(const CacheAttention& a, void* workspace, cudaStream_t stream, int num_sms) {
    using S = Shape<T, D, MT>;
    Plan plan = {};
    plan.group = a.H_q / a.H_kv;
    plan.rows = rows_of(a);
    plan.row_tiles = (plan.rows + S::ROWS - 1) / S::ROWS;
    plan.stored = plan.rows < S::ROWS ? plan.rows : S::ROWS;
    const int64_t grid = share_grid(a, num_sms, S::CTAS);
    if (grid == 0) {
        const int64_t items = (int64_t)a.B * plan.row_tiles * a.H_kv;
        cudaError_t e = cudaFuncSetAttribute(attention_whole_kernel<T, D, MT>,
                                             cudaFuncAttributeMaxDynamicSharedMemorySize, S::SMEM);
        if (e != cudaSuccess) return e;
        attention_whole_kernel<T, D, MT><<<(unsigned)items, kThreads, S::SMEM, stream>>>(a, plan);
        return cudaGetLastError();
    }
    const int64_t slots = grid * 2 * plan.stored;
    plan.joins = static_cast<int4*>(workspace);
    plan.stats = reinterpret_cast<float4*>(plan.joins + grid);
    plan.sums = reinterpret_cast<float*>(plan.stats + slots);
    cudaError_t e = cudaFuncSetAttribute(attention_share_kernel<T, D, MT>,
                                         cudaFuncAttributeMaxDynamicSharedMemorySize, S::SMEM);
    if (e != cudaSuccess) return e;
    attention_share_kernel<T, D, MT><<<(unsigned)grid, kThreads, S::SMEM, stream>>>(a, plan);
    e = cudaGetLastError();
    if (e != cudaSuccess) return e;
    // The second kernel's CTAs come up while the first ends, and wait for it.
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)grid, (unsigned)(plan.stored < 8 ? plan.stored : 8));
    cfg.blockDim = dim3(kJoinThreads);
    cfg.stream = stream;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, attention_join_kernel<T, D, MT>, a, plan);
}

template <typename T, int D>
cudaError_t by_rows(const CacheAttention& a, void* ws, cudaStream_t stream, int num_sms) {
    switch (tile_warps(a)) {
        case 1: return launch<T, D, 1>(a, ws, stream, num_sms);
        case 2: return launch<T, D, 2>(a, ws, stream, num_sms);
        default: return launch<T, D, 4>(a, ws, stream, num_sms);
    }
}

template <typename T>
cudaError_t by_d(const CacheAttention& a, void* ws, cudaStream_t stream, int num_sms) {
    return padded_d(a) == 64 ? by_rows<T, 64>(a, ws, stream, num_sms)
                             : by_rows<T, 128>(a, ws, stream, num_sms);
}

}  // namespace

size_t cache_attention_workspace_bytes(const CacheAttention& a, int num_sms) {
    const int mt = tile_warps(a);
    const int64_t stored = rows_of(a) < 16 * mt ? rows_of(a) : 16 * mt;
    // 3 CTAs a SM: the larger of what the two types of query run
    const int64_t grid = share_grid(a, num_sms, 3);
    return (size_t)grid * (16 + 2 * stored * (16 + padded_d(a) * 4));
}

cudaError_t run_cache_attention(const CacheAttention& a, bool bf16, void* workspace, cudaStream_t stream,
                                int num_sms) {
    return bf16 ? by_d<__nv_bfloat16>(a, workspace, stream, num_sms)
                : by_d<float>(a, workspace, stream, num_sms);
}

}  // namespace kda
