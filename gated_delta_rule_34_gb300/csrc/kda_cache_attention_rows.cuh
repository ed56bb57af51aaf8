// kda_cache_attention_rows.cuh -- attention of a sequence's newest tokens over the paged 8-bit cache, few rows a head.
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
// keys (T_q times H_q / H_kv) are few.  Measured with 8 heads of keys, 32 of queries, d = 128, bf16: a
// million tokens 349 us, 6.2 TB/s; 256 sequences of up to 4096 tokens 186 us, 5.8 TB/s; 77 tokens
// 4.0 us (8.2 to 8.9 under a block table with room for 1,024 to a million).  Beyond 16 rows the conversion of codes and
// the products bound it (537 MB of codes: 99 us under 4 rows, 108 us under 16, 170 us under 32), which is where kda_cache_attention_tc.cu
// takes over for bf16 rows of more than 64 channels.
//
// The tile.  16 tokens a step against NT tiles of 8 rows, on m16n8k16 products of
// fp16 with fp32 sums, tokens and then channels of v on the side of 16: a decode
// step has few rows a head, and 8 waste less than 16.  e4m3 codes are exact in
// fp16, and so are a page's scale (applied to the scores after the product,
// to the weights before it) and bf16 queries, once a power of two has brought
// their row under fp16's largest value.  fp32 queries and their weights go as
// two fp16 pieces (22 bits), two products instead of one.
// No code passes through shared memory to change hands: the pairing of a
// product's k index with channels, of its m index with channels of v, is free, so
// each lane reads its own 16 consecutive bytes of a token's row, as they lie
// in the cache, and its words are the fragments; the scores become the weights'
// fragments by a transposition of 8 x 8 within the warp.  A warp copies its steps
// itself, 16 bytes a lane, some steps ahead, so it runs without a barrier; with
// more rows than one warp takes, MT warps share one ring and one barrier a step.
// The copies go along the rows, whole lines at a time (a million tokens of 8 heads took 448
// us without any arithmetic when every lane fetched the bytes that it reads, half a
// line a row, and 334 us so), and each lane puts its 16 bytes where the reading
// lane's load meets no other's bank.
//
// The maximum is not brought up to date at every step: as long as no score is
// above the last one by more than a factor of 4, sums keep their reference, and a
// vote of the warp is all that a step spends on it.
//
// The work.  The lengths are on the device, so the host cannot cut the work up.
// All steps of all (sequence, row tile, head) items are one list, cut into equal
// shares, one for each of a fixed number of CTAs; each finds its place by
// summing the lengths.  An item counts some steps more than it has, for what its
// start and end cost.  An item that lies within one share is finished there; pieces of
// the others are left in the workspace (fp32 sums with their maxima), at most
// two a CTA, and a second small kernel joins them in a fixed order, so that
// the same call gives the same bits.  Where one CTA takes any item whole
// (short tables, or very many row tiles) there is no second kernel.
//
// V's scale.  The weights are e^(s - m) times the page's scale of v, whose range
// is far beyond fp16's.  So the sums of v have a reference of their own, mo = max(s
// + log2 scale), beside the maximum m that the sum of weights has (kept as dm = m -
// mo, which is small where m is large); weights go to fp16 as 2^(s + log2 scale - mo
// + 12), at most 2^15, with full precision down to 2^-26 of the largest.
//
// NaN that a row does not see.  0 times NaN is NaN, so tokens past the last that
// any row of the tile sees are never copied (zeros instead), and a step that
// some rows see and others do not is looked through for NaN codes of v: if there are
// any they count as zeros, and a product of the rows' sight with the places of
// the NaN marks the outputs that they do reach.
//
// The same kernels take the prefix that a group of sequences shares (kPrefix: the group's rows are one item's, and
// their sums go to what the rows carry) and the rest of each sequence (kRest: joined with that).
#pragma once

#include "kda_attention_common.cuh"

namespace kda {
namespace {

using namespace attn;

constexpr int kWarps = 4;
constexpr int kThreads = 32 * kWarps;

__device__ __forceinline__ float quad_max(float x) {
    x = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, 1));
    return fmaxf(x, __shfl_xor_sync(0xffffffffu, x, 2));
}
// Over the eight lanes of one c.
__device__ __forceinline__ float column_max(float x) {
    x = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, 4));
    x = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, 8));
    return fmaxf(x, __shfl_xor_sync(0xffffffffu, x, 16));
}
__device__ __forceinline__ float column_sum(float x) {
    x += __shfl_xor_sync(0xffffffffu, x, 4);
    x += __shfl_xor_sync(0xffffffffu, x, 8);
    return x + __shfl_xor_sync(0xffffffffu, x, 16);
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

// c += a b: a is 16 x 16 (m = g and g + 8; k = 2c, 2c + 1, then 8 more), b 16 x 8
// (n = g), c 16 x 8 (m = g and g + 8, n = 2c and 2c + 1), of lane 4 g + c.
__device__ __forceinline__ void mma16816(float (&c)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
    asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, "
        "{%0,%1,%2,%3};"
        : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

// (x, y) += (a, b), each rounded: one instruction.
__device__ __forceinline__ void add_pair(float& x, float& y, float a, float b) {
    asm("{\n\t.reg .b64 s, t;\n\tmov.b64 s, {%0, %1};\n\tmov.b64 t, {%2, %3};\n\tadd.rn.f32x2 s, s, t;\n\t"
        "mov.b64 {%0, %1}, s;\n\t}"
        : "+f"(x), "+f"(y)
        : "f"(a), "f"(b));
}

// An 8 x 8 matrix of 16-bit values, a row a quad, transposed.
__device__ __forceinline__ uint32_t transposed(uint32_t x) {
    uint32_t y;
    asm("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(y) : "r"(x));
    return y;
}

// The sizes that go together: a warp takes NT tiles of 8 rows; MT warps share
// the tokens of their 8 NT MT rows; NG groups of them take steps in turn, each with a
// ring of STAGES steps.  The more rows a warp has, the fewer warps' registers an SM holds.  (Four CTAs
// and three stages with one tile of rows: a million tokens 369 us, against 359 us with three and four.)
template <typename T, int D, int NT_, int MT_>
struct Shape {
    static constexpr int NT = NT_, MT = MT_;
    static constexpr int PIECES = sizeof(T) == 4 ? 2 : 1;   // fp16 pieces of a query and a weight
    static constexpr int NG = kWarps / MT;
    static constexpr int ROWS = 8 * NT * MT;
    static constexpr int CTAS = PIECES == 1 ? (NT == 4 ? 2 : 3) : (NT == 1 ? 3 : 2);   // resident a SM
    static constexpr int STAGES = MT == 1 ? (NT == 4 ? 6 : 4) : MT == 2 ? 6 : 8;
    static constexpr int ITEM_COST = NT == 4 ? 32 : 12;     // what an item's start and end cost, in steps
    static constexpr bool Q_HELD = NT <= 2;           // queries in registers, or read again at every step
    static constexpr int KC = D / 64;                 // 16-byte pieces of a key that a lane reads
    static constexpr int VB = D / 8;                  // bytes of a value that a lane reads
    static constexpr int TILES = VB / 2;              // of 16 channels of v
    static constexpr int COPIES = D / 32;             // a warp's, of 16 rows of keys or of values
    static constexpr int ROW_LANES = D / 16;          // lanes that copy one row
    static constexpr int K_BYTES = kStep * D;         // of a step
    static constexpr int STAGE = 2 * K_BYTES + 16;    // + the two scales
    static constexpr int RING = NG * STAGES * STAGE;
    static constexpr int JOIN = NG * ROWS * (D + 4) * 4 + NG * ROWS * 16;
    static constexpr int Q_AT = RING > JOIN ? RING : JOIN;
    static constexpr int Q_BYTES = ROWS * D * 2;      // of one piece
    static constexpr int FACTOR_AT = Q_AT + PIECES * Q_BYTES;
    static constexpr int SMEM = FACTOR_AT + ROWS * 4;
};

// One piece of an item: steps [from, to) of a tile's `steps`.
template <Part P, typename T, int D, int NT, int MT>
struct Piece {
    using S = Shape<T, D, NT, MT>;
    const CacheAttention& a;
    const Plan& plan;
    uint8_t* smem;
    int b, hk, rt, from, to;
    Tile tile;

    // The tile's queries, as the fragments that the score products read: for 8 rows
    // and 64 channels, two 16-byte words of each lane (row g, channels 16 c ..).
    __device__ __forceinline__ void load_queries() {
        const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
        const int g = lane >> 2, c = lane & 3;
        uint4* to_s = reinterpret_cast<uint4*>(smem + S::Q_AT);
        float* factor_s = reinterpret_cast<float*>(smem + S::FACTOR_AT);
        const int64_t token0 = first_query<P>(a, b);
        const int rows = item_rows<P>(a, plan, b);
        for (int rows8 = warp; rows8 < S::ROWS / 8; rows8 += kWarps) {
            const int row = rt * S::ROWS + 8 * rows8 + g;
            const bool real = row < rows;
            const int i = real ? row / plan.group : 0;
            const T* q = static_cast<const T*>(a.q) + (token0 + i) * a.q_stride +
                         (int64_t)(hk * plan.group + (real ? row - i * plan.group : 0)) * a.d;
            uint4 raw[S::KC][sizeof(T)];
            float amax = 0.0f;
#pragma unroll
            for (int j = 0; j < S::KC; ++j) {
                const bool in = real && 64 * j + 16 * c < a.d;
#pragma unroll
                for (int w = 0; w < (int)sizeof(T); ++w)
                    raw[j][w] = in ? reinterpret_cast<const uint4*>(q + 64 * j + 16 * c)[w]
                                   : make_uint4(0, 0, 0, 0);
            }
#pragma unroll
            for (int j = 0; j < S::KC; ++j)
#pragma unroll
                for (int w = 0; w < 16; ++w)
                    amax = fmaxf(amax, fabsf(to_f32(reinterpret_cast<const T*>(raw[j])[w])));
            amax = quad_max(amax);
            // 2^ex <= amax < 2^(ex + 1): times 2^(14 - ex), under fp16's largest value.  A row with an infinity: its scores
            // are infinite or no numbers whatever its finite channels hold, so these count as zeros, under no scale.
            const bool infinite = amax == INFINITY;
            int ex = infinite ? 14 : (int)(__float_as_uint(amax) >> 23) - 127;
            ex = ex < -112 ? -112 : ex;
            const float up = __uint_as_float((uint32_t)(127 + 14 - ex) << 23);
            if (c == 0)
                factor_s[8 * rows8 + g] =
                    a.scale * 1.4426950408889634f * __uint_as_float((uint32_t)(127 + ex - 14) << 23);
#pragma unroll
            for (int j = 0; j < S::KC; ++j)
#pragma unroll
                for (int half = 0; half < 2; ++half) {
                    uint32_t bits[4], rest[4];
#pragma unroll
                    for (int w = 0; w < 4; ++w) {
                        const T* e = reinterpret_cast<const T*>(raw[j]) + 8 * half + 2 * w;
                        float lo = to_f32(e[0]) * up, hi = to_f32(e[1]) * up;
                        if (infinite) {
                            lo = fabsf(lo) < INFINITY ? 0.0f : lo;
                            hi = fabsf(hi) < INFINITY ? 0.0f : hi;
                        }
                        bits[w] = half2_bits(lo, hi);
                        rest[w] = infinite ? 0 : half2_rest(lo, hi, bits[w]);
                    }
                    const int at = ((rows8 * S::KC + j) * 2 + half) * 32 + lane;
                    to_s[at] = make_uint4(bits[0], bits[1], bits[2], bits[3]);
                    if constexpr (S::PIECES == 2)
                        to_s[S::Q_BYTES / 16 + at] = make_uint4(rest[0], rest[1], rest[2], rest[3]);
                }
        }
    }

    __device__ __forceinline__ void run(int cta, int slot, bool whole) {
        const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
        const int g = lane >> 2, c = lane & 3;
        const int grp = warp / MT, wt = warp % MT;
        uint8_t* ring = smem + grp * S::STAGES * S::STAGE;
        const uint32_t ring_u = tc::smem_u32(ring);
        const int d = a.d;
        const int32_t* table = P == kPrefix ? a.prefix_table + (int64_t)b * a.prefix_pages : a.table + (int64_t)b * a.table_pages;
        const int page_mask = (1 << a.page_shift) - 1;
        // What this lane copies: 16-byte piece `piece` of row `row` (and of every 32 / ROW_LANES rows
        // on), to where lane (g, c) will read it.  Keys: word j = piece / 4 of token g (or g + 8) is at
        // [token / 8][j][4 g + c, its bit 2 turned for j = 1].  Values: token 8 (q / 2) + 2 c + q % 2
        // is at [q][c], its pieces turned by c, so that the eight lanes of two g and four c differ.
        const int row = lane / S::ROW_LANES, piece = lane % S::ROW_LANES;
        const int from_lane = row * d + 16 * piece;
        uint32_t k_to_lane, v_to_lane[2];
        if constexpr (D == 128) {
            k_to_lane = (piece >> 2) * 512 + ((4 * row + (piece & 3)) ^ (piece & 4)) * 16;
#pragma unroll
            for (int i = 0; i < 2; ++i)
                v_to_lane[i] = (row & 1) * 512 + (2 * i + (row >> 1)) * 128 + (piece ^ (2 * (2 * i + (row >> 1)))) * 16;
        } else {
            k_to_lane = lane * 16;
            v_to_lane[0] = v_to_lane[1] =
                (row & 1) * 256 + ((row >> 1) ^ (row & 1)) * 64 + (piece ^ ((row >> 1) & 2)) * 16;
        }

        auto page_at = [&](int s) -> int {
            const int t = tile.token(s);
            if (s >= to || t >= tile.end) return -1;
            return table[t >> a.page_shift];
        };
        // Copies step s (its page's id is pg) into stage st.
        auto issue = [&](int s, int pg, int st) {
            const uint32_t stage = ring_u + st * S::STAGE;
            const uint32_t scales = stage + S::STAGE - 16;
            if (pg >= 0 && pg < a.n_pages) {
                const int t0 = tile.token(s);
                const int64_t block = (int64_t)pg * a.H_kv + hk;
                const int64_t at = ((block << a.page_shift) + (t0 & page_mask)) * d;
                const uint8_t* k = a.k_codes + at + from_lane;
                const uint8_t* v = a.v_codes + at + from_lane;
                const int n = tile.end - t0;               // tokens of the step that exist
                const uint32_t k_to = stage + k_to_lane, v_to = stage + S::K_BYTES;
                constexpr int ROWS_A_COPY = 32 / S::ROW_LANES;
                // copy i of a warp's 16 rows starts at row i ROWS_A_COPY
                auto k_at = [&](int i) { return k_to + (D == 128 ? (i >> 1) * 1024 + (i & 1) * 256 : i * 512); };
                auto v_at = [&](int i) {
                    return v_to + v_to_lane[D == 128 ? i & 1 : 0] + (D == 128 ? (i >> 1) * 1024 : i * 512);
                };
                if (d == D && n >= kStep) {
#pragma unroll
                    for (int i = 0; i < S::COPIES; ++i)
                        if (MT == 1 || i % MT == wt) copy_async(k_at(i), k + i * 512, true);
#pragma unroll
                    for (int i = 0; i < S::COPIES; ++i)
                        if (MT == 1 || (i + S::COPIES) % MT == wt) copy_async(v_at(i), v + i * 512, true);
                } else {
#pragma unroll
                    for (int i = 0; i < S::COPIES; ++i) {
                        const int up = i * ROWS_A_COPY;
                        const bool real = up + row < n && 16 * piece < d;
                        if (MT == 1 || i % MT == wt)
                            copy_async(k_at(i), real ? k + up * d : a.k_codes, real);
                        if (MT == 1 || (i + S::COPIES) % MT == wt)
                            copy_async(v_at(i), real ? v + up * d : a.v_codes, real);
                    }
                }
                if (wt == 0 && lane < 2)
                    copy_async4(scales + 4 * lane, (lane ? a.v_scale : a.k_scale) + block, true);
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

        load_queries();
        __syncthreads();
        const uint4* q_s = reinterpret_cast<const uint4*>(smem + S::Q_AT) + wt * NT * S::KC * 64 + lane;
        const float* factor_s = reinterpret_cast<const float*>(smem + S::FACTOR_AT) + wt * NT * 8 + 2 * c;
        uint4 qh[S::Q_HELD ? S::PIECES : 1][S::Q_HELD ? NT : 1][S::KC][2];
        float factor[NT][2], m[NT][2], dm[NT][2], l[NT][2];   // dm = m - mo
#pragma unroll
        for (int n = 0; n < NT; ++n) {
            if constexpr (S::Q_HELD)
#pragma unroll
                for (int pc = 0; pc < S::PIECES; ++pc)
#pragma unroll
                    for (int j = 0; j < S::KC; ++j)
#pragma unroll
                        for (int h = 0; h < 2; ++h)
                            qh[pc][n][j][h] = q_s[pc * (S::Q_BYTES / 16) + ((n * S::KC + j) * 2 + h) * 32];
#pragma unroll
            for (int r = 0; r < 2; ++r) {
                factor[n][r] = factor_s[8 * n + r];
                m[n][r] = kLowest;
                dm[n][r] = l[n][r] = 0.0f;
            }
        }
        float acc[S::TILES][NT][4];
#pragma unroll
        for (int x = 0; x < S::TILES; ++x)
#pragma unroll
            for (int n = 0; n < NT; ++n)
#pragma unroll
                for (int w = 0; w < 4; ++w) acc[x][n][w] = 0.0f;

        // Scores of a step's tokens g and g + 8 with rows 2 c and 2 c + 1 of each tile.  The products' own sums are
        // cut off, not rounded, at every step; with fp32 queries 32 channels' sum is added to the others' by a rounded addition
        // (errors of outputs 3e-7 instead of up to 1.4e-6 over 40 cases, the plain 32-bit form's up to 1.2e-6).
        auto scores = [&](const uint8_t* stage, float (&sc)[NT][4]) {
#pragma unroll
            for (int n = 0; n < NT; ++n)
#pragma unroll
                for (int w = 0; w < 4; ++w) sc[n][w] = 0.0f;
#pragma unroll
            for (int j = 0; j < S::KC; ++j) {
                const uint4 k0 = *reinterpret_cast<const uint4*>(stage + j * 512 + (lane ^ 4 * j) * 16);
                const uint4 k1 = *reinterpret_cast<const uint4*>(stage + (S::KC + j) * 512 + (lane ^ 4 * j) * 16);
                const uint32_t w0[4] = {k0.x, k0.y, k0.z, k0.w}, w1[4] = {k1.x, k1.y, k1.z, k1.w};
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                    uint32_t f[2][4];
#pragma unroll
                    for (int w = 0; w < 2; ++w) {
                        word_to_half2x2(w0[2 * h + w], f[w][0], f[w][2]);
                        word_to_half2x2(w1[2 * h + w], f[w][1], f[w][3]);
                    }
#pragma unroll
                    for (int n = 0; n < NT; ++n) {
                        float part[4] = {};
#pragma unroll
                        for (int pc = S::PIECES - 1; pc >= 0; --pc) {
                            const uint4 q = S::Q_HELD ? qh[S::Q_HELD ? pc : 0][S::Q_HELD ? n : 0][j][h]
                                                      : q_s[pc * (S::Q_BYTES / 16) + ((n * S::KC + j) * 2 + h) * 32];
                            float (&to)[4] = S::PIECES == 2 ? part : sc[n];
                            mma16816(to, f[0], q.x, q.y);
                            mma16816(to, f[1], q.z, q.w);
                        }
                        if constexpr (S::PIECES == 2) {
#pragma unroll
                            for (int w = 0; w < 4; ++w) sc[n][w] += part[w];
                        }
                    }
                }
            }
        };
        auto meet = [&]() {
            if constexpr (MT == 1) __syncwarp();
            else tc::named_bar_sync(1 + grp, 32 * MT);
        };

        int st = 0;
        for (int s = s0; s < to; s += S::NG) {
            copy_wait<S::STAGES - 2>();
            meet();
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
            float sc[NT][4];
            scores(stage, sc);
            const int t0 = tile.token(s);
            const bool partly = t0 + kStep - 1 > tile.p0 ||
                                (a.window > 0 && t0 <= tile.p1 - a.window && t0 + kStep - 1 >= a.sinks);
            uint32_t sight = 0xffffffffu;                  // bit 4 n + w: sc[n][w] is seen
            if (partly) {
                sight = 0;
#pragma unroll
                for (int n = 0; n < NT; ++n)
#pragma unroll
                    for (int r = 0; r < 2; ++r) {
                        const int row = rt * S::ROWS + (wt * NT + n) * 8 + 2 * c + r;
                        const int p = tile.p0 - rt * S::ROWS / plan.group + row / plan.group;
#pragma unroll
                        for (int h = 0; h < 2; ++h) {
                            const int at = t0 + 8 * h + g;
                            if (at <= p && (a.window == 0 || at > p - a.window || at < a.sinks))
                                sight |= 1u << (4 * n + 2 * h + r);
                        }
                    }
            }
            // log2 of v's scale: its exponent, and what remains (1 for the powers of two that cache writes give)
            const float e = (float)((int)(__float_as_uint(scales.y) >> 23) - 127);
            const float mantissa = __uint_as_float((__float_as_uint(scales.y) & 0x7fffffu) | 0x3f800000u);
            // x = score - m, in powers of two
            float x[NT][4];
#pragma unroll
            for (int n = 0; n < NT; ++n)
#pragma unroll
                for (int r = 0; r < 2; ++r) {
                    const float f = factor[n][r] * scales.x;
                    x[n][r] = fmaf(sc[n][r], f, -m[n][r]);
                    x[n][2 + r] = fmaf(sc[n][2 + r], f, -m[n][r]);
                }
            if (partly) {
#pragma unroll
                for (int n = 0; n < NT; ++n)
#pragma unroll
                    for (int w = 0; w < 4; ++w)
                        if (!(sight >> (4 * n + w) & 1)) x[n][w] = -INFINITY;
            }
            // Beyond m, or beyond mo with this page's scale: by how much, at most?
            float beyond = -INFINITY;
#pragma unroll
            for (int n = 0; n < NT; ++n)
#pragma unroll
                for (int r = 0; r < 2; ++r)
                    beyond = fmaxf(beyond, fmaxf(x[n][r], x[n][2 + r]) + fmaxf(dm[n][r] + e, 0.0f));
            if (__any_sync(0xffffffffu, beyond > kSlack)) {
                bool large = false;
#pragma unroll
                for (int n = 0; n < NT; ++n) {
                    float keep[2];
#pragma unroll
                    for (int r = 0; r < 2; ++r) {
                        const float f = factor[n][r] * scales.x;
                        const bool seen[2] = {(sight >> (4 * n + r) & 1) != 0, (sight >> (4 * n + 2 + r) & 1) != 0};
                        const float top = column_max(fmaxf(seen[0] ? sc[n][r] * f : -INFINITY,
                                                           seen[1] ? sc[n][2 + r] * f : -INFINITY));
                        const float m_new = fmaxf(m[n][r], top);
                        large |= fabsf(m_new) >= 65536.0f && m_new != kLowest;
                        const float dm_new = -fmaxf((m[n][r] - m_new) - dm[n][r], (top - m_new) + e);
                        keep[r] = ex2(m[n][r] - m_new + (dm_new - dm[n][r]));
                        l[n][r] *= ex2(m[n][r] - m_new);
                        m[n][r] = m_new;
                        dm[n][r] = dm_new;
#pragma unroll
                        for (int h = 0; h < 2; ++h)
                            x[n][2 * h + r] = seen[h] ? fmaf(sc[n][2 * h + r], f, -m_new) : -INFINITY;
                    }
#pragma unroll
                    for (int y = 0; y < S::TILES; ++y)
#pragma unroll
                        for (int w = 0; w < 4; ++w) acc[y][n][w] *= keep[w & 1];
                }
                // Scores beyond 2^23 have whole numbers for last places: less a maximum that is a rounded product they
                // would be that far off, and weights beyond fp16's range, were they not rounded products too.
                if (__any_sync(0xffffffffu, large)) {
#pragma unroll
                    for (int n = 0; n < NT; ++n)
#pragma unroll
                        for (int w = 0; w < 4; ++w)
                            if (x[n][w] != -INFINITY) x[n][w] = __fsub_rn(__fmul_rn(sc[n][w], factor[n][w & 1] * scales.x), m[n][w & 1]);
                }
            }
            uint32_t pf[S::PIECES][NT][2];                 // weights: tokens 2 c .. of row g, then 8 more
#pragma unroll
            for (int n = 0; n < NT; ++n) {
                float lift[2];
#pragma unroll
                for (int r = 0; r < 2; ++r) lift[r] = ex2(fminf(dm[n][r] + (e + kWeightBits), 126.0f)) * mantissa;
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                    const float p0 = ex2(x[n][2 * h]), p1 = ex2(x[n][2 * h + 1]);
                    l[n][0] += p0;
                    l[n][1] += p1;
                    const float lo = p0 * lift[0], hi = p1 * lift[1];
                    const uint32_t bits = half2_bits(lo, hi);
                    pf[0][n][h] = transposed(bits);
                    if constexpr (S::PIECES == 2) pf[1][n][h] = transposed(half2_rest(lo, hi, bits));
                }
            }
            // Values: four tokens' words; a product's a pairs two tokens of one channel.
            const uint8_t* vs = stage + S::K_BYTES;
            uint32_t v[4][S::VB / 4];
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                if constexpr (D == 128) {
                    const uint4 x = *reinterpret_cast<const uint4*>(vs + i * 512 + c * 128 + (g ^ 2 * c) * 16);
                    v[i][0] = x.x, v[i][1] = x.y, v[i][2] = x.z, v[i][3] = x.w;
                } else {
                    const uint2 x = *reinterpret_cast<const uint2*>(
                        vs + i * 256 + (c ^ (i & 1)) * 64 + ((g >> 1) ^ (c & 2)) * 16 + (g & 1) * 8);
                    v[i][0] = x.x, v[i][1] = x.y;
                }
            }
            if (partly) {
                uint32_t any = 0;
#pragma unroll
                for (int i = 0; i < 4; ++i)
#pragma unroll
                    for (int w = 0; w < S::VB / 4; ++w) any |= nan_bytes(v[i][w]);
                if (__any_sync(0xffffffffu, any != 0)) {
                    uint32_t ones[1][NT][2];               // the rows' sight as weights of 1
#pragma unroll
                    for (int n = 0; n < NT; ++n)
#pragma unroll
                        for (int h = 0; h < 2; ++h)
                            ones[0][n][h] = transposed((sight >> (4 * n + 2 * h) & 1 ? 0x3c00u : 0u) |
                                                       (sight >> (4 * n + 2 * h + 1) & 1 ? 0x3c000000u : 0u));
#pragma unroll
                    for (int w = 0; w < S::VB / 4; ++w) {
                        uint32_t bad[4];
#pragma unroll
                        for (int i = 0; i < 4; ++i) {
                            bad[i] = nan_bytes(v[i][w]);
                            v[i][w] &= ~bad[i];
                            bad[i] &= 0x38383838u;         // 1 in e4m3
                        }
                        float hit[2][NT][4] = {};
                        add_values<2, 1>(hit, 0, ones, bad[0], bad[1], bad[2], bad[3]);
#pragma unroll
                        for (int y = 0; y < 2; ++y)
#pragma unroll
                            for (int n = 0; n < NT; ++n)
#pragma unroll
                                for (int z = 0; z < 4; ++z)
                                    if (hit[y][n][z] > 0.0f) acc[2 * w + y][n][z] = NAN;
                    }
                }
            }
#pragma unroll
            for (int w = 0; w < S::VB / 4; ++w) add_values(acc, 2 * w, pf, v[0][w], v[1][w], v[2][w], v[3][w]);
        }
        copy_wait<0>();
        __syncthreads();                                   // the ring becomes the place to join in

        // Join the groups.  Lane (g, c) holds channels VB g .. of rows 2 c and 2 c + 1.
        float* o_s = reinterpret_cast<float*>(smem);
        float4* stat_s = reinterpret_cast<float4*>(smem + S::NG * S::ROWS * (D + 4) * 4);
#pragma unroll
        for (int n = 0; n < NT; ++n)
#pragma unroll
            for (int r = 0; r < 2; ++r) {
                const int row = (wt * NT + n) * 8 + 2 * c + r;
                l[n][r] = column_sum(l[n][r]);
                if (row >= plan.stored) continue;
                float* to_s = o_s + (grp * S::ROWS + row) * (D + 4) + S::VB * g;
#pragma unroll
                for (int y = 0; y < S::TILES; y += 2)
                    *reinterpret_cast<float4*>(to_s + 2 * y) =
                        make_float4(acc[y][n][r], acc[y][n][2 + r], acc[y + 1][n][r], acc[y + 1][n][2 + r]);
                if (g == 0) stat_s[grp * S::ROWS + row] = make_float4(m[n][r], dm[n][r], l[n][r], 0.0f);
            }
        __syncthreads();
        const int rows_here = rows_of_tile<P>(a, plan, b, rt);
        for (int u = threadIdx.x; u < rows_here * (D / 4); u += kThreads) {
            const int r = u / (D / 4), ch = u % (D / 4) * 4;
            float M = kLowest, DM = INFINITY, L = 0.0f;
            float4 stat[S::NG];
#pragma unroll
            for (int i = 0; i < S::NG; ++i) {
                stat[i] = stat_s[i * S::ROWS + r];
                M = fmaxf(M, stat[i].x);
            }
#pragma unroll
            for (int i = 0; i < S::NG; ++i) DM = fminf(DM, stat[i].y + (M - stat[i].x));
            float4 o = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
#pragma unroll
            for (int i = 0; i < S::NG; ++i) {
                L += stat[i].z * ex2(stat[i].x - M);
                const float f = ex2(stat[i].x - M + (DM - stat[i].y));
                const float4 x = *reinterpret_cast<const float4*>(o_s + (i * S::ROWS + r) * (D + 4) + ch);
                o.x += f * x.x;
                o.y += f * x.y;
                o.z += f * x.z;
                o.w += f * x.w;
            }
            if (whole) {
                finish_row<T, P, D>(a, output_row<P>(a, plan, b, hk, rt, r), ch, o, M, DM, L, tile.carried);
            } else {
                const int64_t at = ((int64_t)cta * 2 + slot) * plan.stored + r;
                *reinterpret_cast<float4*>(plan.sums + at * D + ch) = o;
                if (ch == 0) plan.stats[at] = make_float4(M, DM, L, 0.0f);
            }
        }
        __syncthreads();
    }

    // acc[y0], acc[y0 + 1] += four channels of four tokens x weights.  The products' own sums are cut off, not rounded, and
    // all the same way: sums kept in them over 131,072 tokens of one sign came out up to 8.5e-4 too small.  So a product
    // holds one step's tokens (and both pieces of a weight), and its sum is added to the others' by rounded additions.
    template <int N, int PCS>
    static __device__ __forceinline__ void add_values(float (&acc)[N][NT][4], int y0, const uint32_t (&pf)[PCS][NT][2],
                                                      uint32_t v0, uint32_t v1, uint32_t v2, uint32_t v3) {
        uint32_t f[2][4];
        word_to_half2x2(__byte_perm(v0, v1, 0x5140), f[0][0], f[0][1]);
        word_to_half2x2(__byte_perm(v0, v1, 0x7362), f[1][0], f[1][1]);
        word_to_half2x2(__byte_perm(v2, v3, 0x5140), f[0][2], f[0][3]);
        word_to_half2x2(__byte_perm(v2, v3, 0x7362), f[1][2], f[1][3]);
#pragma unroll
        for (int y = 0; y < 2; ++y)
#pragma unroll
            for (int n = 0; n < NT; ++n) {
                float part[4] = {};
#pragma unroll
                for (int pc = PCS - 1; pc >= 0; --pc) mma16816(part, f[y], pf[pc][n][0], pf[pc][n][1]);
                add_pair(acc[y0 + y][n][0], acc[y0 + y][n][1], part[0], part[1]);
                add_pair(acc[y0 + y][n][2], acc[y0 + y][n][3], part[2], part[3]);
            }
    }

};

// Every CTA one item: (sequence, row tile, head), heads innermost.
template <Part P, typename T, int D, int NT, int MT>
__global__ void __launch_bounds__(kThreads, Shape<T, D, NT, MT>::CTAS)
attention_whole_kernel(const CacheAttention a, const Plan plan) {
    extern __shared__ __align__(16) uint8_t smem[];
    after_the_kernel_before();
    const int pair = blockIdx.x / a.H_kv, hk = blockIdx.x % a.H_kv;
    const Tile tile = tile_of<P>(a, plan, pair);
    if (P == kPrefix && tile.steps == 0) return;
    const int2 at = split_pair<P>(a, plan, pair);
    Piece<P, T, D, NT, MT> piece{a, plan, smem, at.x, hk, at.y, 0, tile.steps, tile};
    piece.run(0, 0, true);
}

// Every CTA an equal share of all items' steps.
template <Part P, typename T, int D, int NT, int MT>
__global__ void __launch_bounds__(kThreads, Shape<T, D, NT, MT>::CTAS)
attention_share_kernel(const CacheAttention a, const Plan plan) {
    extern __shared__ __align__(16) uint8_t smem[];
    after_the_kernel_before();
    const Share share = find_share<kThreads, P>(a, plan);
    const int4 join = for_each_piece<P>(a, plan, share, [&](int pair, int hk, const Tile& tile, int from, int to, int slot,
                                                            bool whole) {
        const int2 at = split_pair<P>(a, plan, pair);
        Piece<P, T, D, NT, MT> piece{a, plan, smem, at.x, hk, at.y, from, to, tile};
        piece.run(blockIdx.x, slot, whole);
    });
    if (threadIdx.x == 0) plan.joins[blockIdx.x] = join;
}

// The pieces of the item that begins in CTA blockIdx.x's share and ends in a later
// one, joined in order: the first from its slot, the later ones from slot 0.  Few
// pieces: a warp a row, without a barrier; many: eight warps a row, each every
// eighth piece, their sums joined in shared memory.  A piece's statistics and sums are
// loaded together, the sums so far rescaled as they come, since what it takes is loads that wait for one another
// (8 sequences of 1,501 tokens, 16 heads, fp32: 15.3 us; 1.5 more with the largest of all statistics found first, 0.8 more
// with eight pieces at once, whose registers leave room for fewer CTAs).
template <Part P, typename T, int D>
__global__ void __launch_bounds__(kJoinThreads, 4)
attention_join_kernel(const CacheAttention a, const Plan plan) {
    constexpr int WARPS = kJoinThreads / 32, PER = D / 32;
    __shared__ float4 o_s[WARPS][D / PER];
    __shared__ float4 stat_s[WARPS];
    after_the_kernel_before();
    const int4 join = plan.joins[blockIdx.x];
    if (join.x < 0) return;
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int n = join.z - (int)blockIdx.x + 1;
    const int2 item = split_pair<P>(a, plan, join.x);
    const int b = item.x, rt = item.y;
    const int rows_here = rows_of_tile<P>(a, plan, b, rt);
    const bool carried = P == kRest && carried_tokens(a, b, length_of(a, b)) > 0;
    const bool few = n <= kJoinFew;
    const int at_once = few ? WARPS : 1, part = few ? 0 : warp, parts = few ? 1 : WARPS;
    for (int r0 = blockIdx.y * at_once; r0 < rows_here; r0 += gridDim.y * at_once) {
        const int r = r0 + (few ? warp : 0);
        if (r >= rows_here) return;                        // only where no barrier follows
        auto place = [&](int i) -> int64_t {
            return ((int64_t)(blockIdx.x + i) * 2 + (i == 0 ? join.w : 0)) * plan.stored + r;
        };
        // Sums (m, dm, l; x) join those so far, whose largest is M and, with the pages' scales, M - DM.  To M and DM from
        // m at least M and the least of dm over what joins, as seen from m.
        float o[4] = {}, M = kLowest, DM = 0.0f, L = 0.0f;
        auto rise = [&](float m_new, float dm) {
            const float dm_new = fminf(DM + (m_new - M), dm);
            const float keep = ex2(M - m_new + (dm_new - DM));
            L *= ex2(M - m_new);
#pragma unroll
            for (int c = 0; c < 4; ++c) o[c] *= keep;
            M = m_new;
            DM = dm_new;
        };
        auto add = [&](const float4& s, const float4& x) {
            const float f = ex2(s.x - M + (DM - s.y));
            L += s.z * ex2(s.x - M);
            o[0] += f * x.x, o[1] += f * x.y, o[2] += f * x.z, o[3] += f * x.w;
        };
        for (int i0 = part; i0 < n; i0 += kAtOnce * parts) {
            float4 s[kAtOnce], x[kAtOnce];
            float m = M, dm = INFINITY;
#pragma unroll
            for (int j = 0; j < kAtOnce; ++j) {
                const int i = i0 + j * parts;
                s[j] = make_float4(kLowest, 0.0f, 0.0f, 0.0f);
                x[j] = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
                if (i >= n) continue;
                const int64_t at = place(i);
                const float* from = plan.sums + at * D + PER * lane;
                s[j] = plan.stats[at];
                if constexpr (PER == 4) {
                    x[j] = *reinterpret_cast<const float4*>(from);
                } else {
                    const float2 two = *reinterpret_cast<const float2*>(from);
                    x[j].x = two.x, x[j].y = two.y;
                }
            }
#pragma unroll
            for (int j = 0; j < kAtOnce; ++j) m = fmaxf(m, s[j].x);
#pragma unroll
            for (int j = 0; j < kAtOnce; ++j) dm = fminf(dm, s[j].y + (m - s[j].x));
            rise(m, dm);
#pragma unroll
            for (int j = 0; j < kAtOnce; ++j) add(s[j], x[j]);
        }
        if (!few) {
            o_s[warp][lane] = make_float4(o[0], o[1], o[2], o[3]);
            if (lane == 0) stat_s[warp] = make_float4(M, DM, L, 0.0f);
            __syncthreads();
            if (warp == 0) {
                for (int w = 1; w < WARPS; ++w) {
                    const float4 s = stat_s[w];
                    const float m = fmaxf(M, s.x);
                    rise(m, s.y + (m - s.x));
                    add(s, o_s[w][lane]);
                }
            }
            __syncthreads();
            if (warp != 0) continue;
        }
        if constexpr (PER == 2) {                          // four channels a lane from here on
            o[2] = __shfl_down_sync(0xffffffffu, o[0], 1);
            o[3] = __shfl_down_sync(0xffffffffu, o[1], 1);
            if (lane & 1) continue;
        }
        finish_row<T, P, D>(a, output_row<P>(a, plan, b, join.y, rt, r), PER * lane,
                            make_float4(o[0], o[1], o[2], o[3]), M, DM, L, carried);
    }
}

// Rows of an item at most; of a group, the rows that it has where groups are alike.
template <Part P>
int64_t rows_of(const CacheAttention& a) {
    const int64_t rows = (int64_t)a.T_q * (a.H_q / a.H_kv);
    return P == kPrefix ? rows * ((a.B + a.n_groups - 1) / a.n_groups) : rows;
}
int padded_d(const CacheAttention& a) { return a.d <= 64 ? 64 : 128; }

// Calls f with the shape for these queries: as many rows a warp as registers allow
// before warps have to share tokens.  (More than 16 bf16 rows of more than 64 channels
// are the other kernels': attention_tc_takes.)
template <Part P, typename T, int D, typename F>
auto by_rows(const CacheAttention& a, F f) {
    const int64_t rows = rows_of<P>(a);
    if (rows <= 8) return f(Shape<T, D, 1, 1>{});
    if constexpr (sizeof(T) == 2 && D == 128) {
        // The rest behind a prefix is short, and 32 rows a CTA of two warps a group have fewer starts and ends: 40 sequences of
        // 256 rows a head, 128 tokens each, 141 us with the prefix, 161 with 16 rows a CTA, 137 with 64 of four warps; 32 rows, 42,
        // 45 and 47.  (Four tiles of rows a warp: slower than either.)
        if constexpr (P == kRest) {
            if (rows > 16) return f(Shape<T, D, 2, 2>{});
        }
        return f(Shape<T, D, 2, 1>{});
    } else {
        constexpr int MOST = sizeof(T) == 4 ? 2 : 4;
        if (rows <= 16) return f(Shape<T, D, 2, 1>{});
        if (rows <= 32) return f(Shape<T, D, MOST, 4 / MOST>{});
        return f(Shape<T, D, MOST, 8 / MOST>{});
    }
}
template <Part P, typename F>
auto by_shape(const CacheAttention& a, bool bf16, F f) {
    if (bf16) return padded_d(a) == 64 ? by_rows<P, __nv_bfloat16, 64>(a, f) : by_rows<P, __nv_bfloat16, 128>(a, f);
    return padded_d(a) == 64 ? by_rows<P, float, 64>(a, f) : by_rows<P, float, 128>(a, f);
}

template <Part P, typename S>
Plan make_plan(const CacheAttention& a) {
    Plan plan = {};
    plan.group = a.H_q / a.H_kv;
    const int64_t rows = (int64_t)a.T_q * plan.group * (P == kPrefix ? a.B : 1);
    plan.rows = (int)rows;
    plan.tile_rows = S::ROWS;
    plan.row_tiles = (int)((rows + S::ROWS - 1) / S::ROWS);
    plan.pairs = P == kPrefix ? plan.row_tiles + a.n_groups : 0;
    plan.stored = plan.rows < S::ROWS ? plan.rows : S::ROWS;
    plan.item_cost = S::ITEM_COST;
    plan.cut = 1;
    return plan;
}

// CTAs of the shared-out form; 0 where each item is one CTA's.  Measured both ways at 8 to 2,048 items of up to 256 to 4,096
// tokens: with 32 steps (512 tokens) 8.4 us whole and 9.3 cut (32 items), 8.5 and 12.1 (128), 34 and 35 (1,024); with 128
// steps 23 and 19 us (128), 65 and 54 (512), 175 and 184 (2,048); with 256 steps and lengths that differ 113 and 102 us (1,024).
template <Part P>
int64_t pairs_of(const CacheAttention& a, const Plan& plan) {
    return P == kPrefix ? plan.pairs : (int64_t)a.B * plan.row_tiles;
}
template <Part P>
int64_t share_grid(const CacheAttention& a, const Plan& plan, int64_t most) {
    const int64_t cap = P == kPrefix ? ((int64_t)a.prefix_pages << a.page_shift) / kStep : most_steps(a);
    const int64_t pairs = pairs_of<P>(a, plan), items = pairs * a.H_kv;
    if (whole_items_pay(P == kRest ? rest_steps(a) : cap, items, most, 32, 128) || pairs > kMaxScan) return 0;
    const int64_t useful = (items * (cap + plan.item_cost) + kMinShare - 1) / kMinShare;
    return useful < most ? useful : most;
}

template <Part P, typename T, int D>
cudaError_t launch_join(const CacheAttention& a, const Plan& plan, int64_t grid, cudaStream_t stream) {
    // A row a CTA where the items are so few that each ends in many pieces.
    const bool many = grid > kJoinFew * pairs_of<P>(a, plan) * a.H_kv;
    const dim3 ctas((unsigned)grid, (unsigned)(many ? plan.stored : (plan.stored + 7) / 8));
    return launch_chained(attention_join_kernel<P, T, D>, ctas, kJoinThreads, 0, stream, a, plan);
}

template <Part P, typename T, int D, int NT, int MT>
cudaError_t launch(Shape<T, D, NT, MT>, const CacheAttention& a, void* workspace, cudaStream_t stream, int num_sms) {
    using S = Shape<T, D, NT, MT>;
    Plan plan = make_plan<P, S>(a);
    const int64_t grid = share_grid<P>(a, plan, (int64_t)num_sms * S::CTAS);
    if (grid == 0) {
        const int64_t items = pairs_of<P>(a, plan) * a.H_kv;
        cudaError_t e = cudaFuncSetAttribute(attention_whole_kernel<P, T, D, NT, MT>,
                                             cudaFuncAttributeMaxDynamicSharedMemorySize, S::SMEM);
        if (e != cudaSuccess) return e;
        return launch_chained(attention_whole_kernel<P, T, D, NT, MT>, (unsigned)items, kThreads, S::SMEM, stream, a, plan);
    }
    set_attention_pieces(plan, workspace, grid);
    cudaError_t e = cudaFuncSetAttribute(attention_share_kernel<P, T, D, NT, MT>,
                                         cudaFuncAttributeMaxDynamicSharedMemorySize, S::SMEM);
    if (e != cudaSuccess) return e;
    e = launch_chained(attention_share_kernel<P, T, D, NT, MT>, (unsigned)grid, kThreads, S::SMEM, stream, a, plan);
    return e != cudaSuccess ? e : launch_join<P, T, D>(a, plan, grid, stream);
}

// The larger of what the two types of query need.
template <Part P>
size_t rows_workspace_bytes(const CacheAttention& a, int num_sms) {
    size_t most = 0;
    for (int bf16 = 0; bf16 < 2; ++bf16) {
        const size_t need = by_shape<P>(a, bf16 != 0, [&](auto shape) -> size_t {
            using S = decltype(shape);
            const Plan plan = make_plan<P, S>(a);
            return attention_piece_bytes(share_grid<P>(a, plan, (int64_t)num_sms * S::CTAS), plan.stored, padded_d(a));
        });
        most = need > most ? need : most;
    }
    return most;
}
template <Part P>
cudaError_t run_rows(const CacheAttention& a, bool bf16, void* workspace, cudaStream_t stream, int num_sms) {
    return by_shape<P>(a, bf16, [&](auto shape) { return launch<P>(shape, a, workspace, stream, num_sms); });
}
template <Part P>
cudaError_t run_join(const CacheAttention& a, const attn::Plan& plan, bool bf16, int D, int64_t grid, cudaStream_t stream) {
    if (bf16)
        return D == 64 ? launch_join<P, __nv_bfloat16, 64>(a, plan, grid, stream)
                       : launch_join<P, __nv_bfloat16, 128>(a, plan, grid, stream);
    return D == 64 ? launch_join<P, float, 64>(a, plan, grid, stream) : launch_join<P, float, 128>(a, plan, grid, stream);
}

}  // namespace
}  // namespace kda
