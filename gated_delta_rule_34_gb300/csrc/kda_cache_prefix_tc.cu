// kda_cache_prefix_tc.cu -- attention of a group's rows over the prefix that its sequences share, for bf16 queries.
//
// All sequences' query rows of one head of keys are the rows of one product with the prefix's keys, 128 of them to a
// product, and of one with its values:
//
//   S [128 rows x 128 tokens] = (q1 + q2) [128 x d] K^T        q1 e5m2, q2 e4m3: the 8 bits of a bf16 value exactly, down to
//                                                             2^-13 of its row's largest; K e4m3, as it lies in the cache
//   W = 2^(s f + c)                                           fp16, 11 bits: f the page's scale of keys, c = log2 of its scale
//                                                             of values less the row's reference, a whole number
//   O [128 rows x d]        += W [128 x 128] V                W from TMEM; V fp16, exact, converted once for 256 rows
//
// What bounds it: 4 d operations a row and token on the tensor cores (q in two fp8 pieces costs what one bf16 product
// does), with the exponentials and conversions beside them; under 128 rows, reading the codes.  256 sequences of 4 rows a head, 8
// heads of 128, behind 32,768 tokens: 147 us, where the products take 72; the tensor pipe runs 42% of it.  A stream's products are
// 1,024 cycles a tile, two streams' tiles take 4,150: softmax 1,770, scores 1,100 (their operands take all that shared memory gives),
// values 700, the rest hand-overs.
//
// One CTA an SM takes items (group, head of keys, 256 rows): two streams of 128 rows, each with softmax threads
// that own a row (no shuffles), so that one stream's products run under the other's softmax. Keys and values are loaded and
// converted once for both. Where 128 rows or fewer are left, both streams take them, the tiles of tokens in turn. Roles:
//   16 softmax   scores from TMEM, weights back into the same columns: eight warps a stream, half of a tile's tokens each
//   4 converters values from e4m3 to fp16
//   1 issuer     S of a stream's next tile after the O of its last one, since S and W share their columns
//   1 loader     pages by TMA, 128-byte-swizzled rows, a box a page (of up to 128 tokens); their scales
//   1 planner    the CTA's pieces, told to the others through shared memory
// A row's references, m of its scores and m + dr of its weights times their pages' scales of values, are whole numbers, so that
// moving them rounds nothing.  A weight is 2^7 at most where they were set; they move when one would pass 2^15, or a score 2^64 times
// 2^m.  l sums the exponentials in fp32, before they are rounded to the fp16 weights (11 bits) that meet the values.
//
// The products' sums are cut off, not rounded: every 64 tiles O goes to sums in the workspace by rounded additions.
//
// The work is one list in equal shares, as in kda_attention_common.cuh, but of tiles of 128 tokens a stream. What a share
// leaves of an item goes to the workspace; a second small kernel joins it.
//
// A wait that gives up (about 2 s) makes the sums of the piece and of the CTA's later ones NaN; see kda_cache_attention_tc.cu.
#include <cuda.h>
#include <cudaTypedefs.h>

#include <mutex>

#include "kda_attention_common.cuh"

namespace kda {
namespace {

using namespace attn;
using tc::smem_u32;

constexpr int kRows = 128;                 // of a stream
constexpr int kPair = 2 * kRows;           // of an item
constexpr int kTokens = 128;               // of a tile: 8 steps
constexpr int kSteps = kTokens / kStep;
constexpr int kTile = kTokens * 128;       // bytes of a tile's keys, or values
constexpr int kKeySlots = 3, kRawSlots = 2, kValueSlots = 2;
constexpr int kScaleSlots = 8;             // more than tiles that softmax may be behind the loader
constexpr int kWarpgroup = 128;
constexpr int kStream = 256;               // softmax threads of a stream
constexpr int kThreads = 768;
constexpr int kConverterWarp = 16, kIssuerWarp = 20, kLoaderWarp = 21, kPlannerWarp = 22;
constexpr int kPieceSlots = 4;
constexpr int kPatience = 8;               // waits' limits that roles wait for one another's pieces
// 80 registers a thread at launch: 512 x 96 + 256 x 48 = 768 x 80.
constexpr int kSoftmaxRegs = 96, kOtherRegs = 48;
static_assert(2 * kStream * kSoftmaxRegs + (kThreads - 2 * kStream) * kOtherRegs <= kThreads * 80, "registers at launch");
constexpr int kItemCost = 4;               // what an item's start and end cost, in tiles of a stream
constexpr int kLeastShare = 8;
constexpr int kRun = 64;                   // tiles that O sums up
constexpr float kBits = 7.0f, kFar = 8.0f; // log2 of the largest weight at its reference, and of how far above it
constexpr float kFarScore = 64.0f;         // and of how far a score may be above m: l is a sum of 2^(s - m)
constexpr float kNear = 4194304.0f;        // 2^22: below, scores have places behind the point
// Named barriers: 1 to 8 of the two warps that have the same rows, 9 and 10 of a stream's, 11 of both streams'.
constexpr int kBarRows = 1, kBarStream = 9, kBarBoth = 11;

// Shared memory, from a 1024-byte boundary.
constexpr int kQueriesAt = 0;                                      // [2 streams][2 pieces][128 rows][128 channels]
constexpr int kKeysAt = kQueriesAt + 4 * kTile;
constexpr int kRawAt = kKeysAt + kKeySlots * kTile;
constexpr int kValuesAt = kRawAt + kRawSlots * kTile;              // [2 halves of the channels][128 tokens][64 channels] fp16
constexpr int kValueTile = 2 * kTile;
constexpr int kSmallAt = kValuesAt + kValueSlots * kValueTile;

// What a CTA does next: a piece of an item. The planner writes these, so that the other roles' registers are free of the
// walk through the list.
struct PrefixPiece {
    int g, hk;
    int rows256;                           // which 256 rows of the group's
    int two;                               // two streams of 128 rows, or one of 128 or fewer that both take
    int from, to;                          // tiles; none: the end
    int slot, whole;
    int first_seq;                         // of the group,
    int tokens;                            // its prefix,
    int64_t rows;                          // and all its rows
};
struct Scales {
    alignas(16) float2 step[kSteps];       // of keys; log2 of that of values
    uint32_t mask;                         // steps that exist, a bit each
    float lowest;                          // of their values' logarithms
};
struct Small {
    PrefixPiece piece[kPieceSlots];
    Scales scales[kScaleSlots];
    float factor[kPair];                   // of the scores, to powers of two
    float4 stat[kRows];                    // of the second stream's sums, where both have the same rows
    float top[2][2][kRows], reach[2][2][kRows];   // what the halves of a stream tell each other
    uint64_t k_full[kKeySlots], k_empty[kKeySlots], raw_full[kRawSlots], raw_empty[kRawSlots], v_full[kValueSlots],
        v_empty[kValueSlots], scale_full[kScaleSlots], s_full[2], p_full[2], o_done[2], q_full[2], piece_full[kPieceSlots],
        piece_empty[kPieceSlots], drained;
    uint32_t tmem;
};
constexpr int kSmem = kSmallAt + (int)sizeof(Small) + 1024;
static_assert(kSmem <= 227 * 1024, "shared memory");

constexpr uint32_t kTmemCols = 512;        // S (and W) 2 x 128, O 2 x 128
constexpr uint32_t kTmemO = 256;

struct PrefixPlan {
    int group;
    int D;                                 // of a row of carried sums: 64 or 128
    float4* stats;                         // [grid][2][256]
    float* sums;                           // [grid][2][256][D]
    float* runs;                           // [grid][2 streams][32][128 rows][4]
    int4* joins;                           // [grid]: group (< 0: none), head, last CTA, 2 (256 rows) + slot
    Stall stall;
};

constexpr uint32_t idesc(uint32_t M, uint32_t N, uint32_t a_format, bool b_mn) {
    return (1u << 4) | (a_format << 7) | ((b_mn ? 1u : 0u) << 16) | ((N >> 3) << 17) | ((M >> 4) << 24);
}
// Shared-memory descriptors by their lower words (address and the stride along the 128-byte rows); the upper words are
// constant: 1024 bytes from eight rows to the next, version 1, 128-byte swizzle.
constexpr uint32_t kDescHigh = (1024u >> 4) | 1u << 14 | 2u << 29;
__device__ __forceinline__ uint32_t desc_low(uint32_t addr, uint32_t lbo) { return (addr >> 4 & 0x3FFFu) | lbo >> 4 << 16; }
// fp8 (a_format 0 e4m3, 1 e5m2; B e4m3), both from shared memory.
template <bool ADD>
__device__ __forceinline__ void mma_f8(uint32_t d_tmem, uint32_t a, uint32_t b, uint32_t desc) {
    asm volatile(
        "{\n\t.reg .b64 da, db;\n\t.reg .pred p;\n\t"
        "mov.b64 da, {%1, %4};\n\tmov.b64 db, {%2, %4};\n\tsetp.ne.b32 p, %5, 0;\n\t"
        "tcgen05.mma.cta_group::1.kind::f8f6f4 [%0], da, db, %3, p;\n\t}" ::"r"(d_tmem), "r"(a), "r"(b), "r"(desc),
        "n"(kDescHigh), "n"(ADD ? 1 : 0)
        : "memory");
}
// fp16, A from TMEM.
__device__ __forceinline__ void mma_f16_ta(uint32_t d_tmem, uint32_t a_tmem, uint32_t b, uint32_t desc, bool accumulate) {
    asm volatile(
        "{\n\t.reg .b64 db;\n\t.reg .pred p;\n\t"
        "mov.b64 db, {%2, %5};\n\tsetp.ne.b32 p, %4, 0;\n\t"
        "tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], db, %3, p;\n\t}" ::"r"(d_tmem), "r"(a_tmem), "r"(b), "r"(desc),
        "r"((uint32_t)accumulate), "n"(kDescHigh)
        : "memory");
}
// 32 columns of the warp's 32 lanes, a lane a thread.
__device__ __forceinline__ void load32(uint32_t taddr, float* v) {
    uint32_t r[32];
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x32.b32 "
        "{%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16,%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31},"
        " [%32];"
        : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), "=r"(r[8]),
          "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15]), "=r"(r[16]),
          "=r"(r[17]), "=r"(r[18]), "=r"(r[19]), "=r"(r[20]), "=r"(r[21]), "=r"(r[22]), "=r"(r[23]), "=r"(r[24]),
          "=r"(r[25]), "=r"(r[26]), "=r"(r[27]), "=r"(r[28]), "=r"(r[29]), "=r"(r[30]), "=r"(r[31])
        : "r"(taddr));
#pragma unroll
    for (int i = 0; i < 32; ++i) v[i] = __uint_as_float(r[i]);
}
// This thread's loads from TMEM have come; what they gave is used after it only.
__device__ __forceinline__ void loaded16(float* v) {
    asm volatile("tcgen05.wait::ld.sync.aligned;"
                 : "+f"(v[0]), "+f"(v[1]), "+f"(v[2]), "+f"(v[3]), "+f"(v[4]), "+f"(v[5]), "+f"(v[6]), "+f"(v[7]),
                   "+f"(v[8]), "+f"(v[9]), "+f"(v[10]), "+f"(v[11]), "+f"(v[12]), "+f"(v[13]), "+f"(v[14]), "+f"(v[15])
                 :
                 : "memory");
}

__device__ __forceinline__ uint64_t add_pair(uint64_t a, uint64_t b) {
    uint64_t r;
    asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
    return r;
}

__device__ __forceinline__ void store8(float* to, const float* v) {
    asm volatile("st.global.v8.f32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8};" ::"l"(to), "f"(v[0]), "f"(v[1]), "f"(v[2]), "f"(v[3]),
                 "f"(v[4]), "f"(v[5]), "f"(v[6]), "f"(v[7])
                 : "memory");
}
// The two fp16 pairs of a word of four codes.
__device__ __forceinline__ void word_to_half2x2(uint32_t w, uint32_t& lo, uint32_t& hi) {
    asm("{\n\t.reg .b16 l, h;\n\tmov.b32 {l, h}, %2;\n\t"
        "cvt.rn.f16x2.e4m3x2 %0, l;\n\tcvt.rn.f16x2.e4m3x2 %1, h;\n\t}"
        : "=r"(lo), "=r"(hi)
        : "r"(w));
}

// Four values to e5m2 (nearest) and back: an e5m2 code is the upper byte of an fp16 number.
__device__ __forceinline__ uint32_t to_e5m2x4(float a, float b, float c, float d) {
    const uint32_t lo = __nv_cvt_float2_to_fp8x2(make_float2(a, b), __NV_SATFINITE, __NV_E5M2);
    const uint32_t hi = __nv_cvt_float2_to_fp8x2(make_float2(c, d), __NV_SATFINITE, __NV_E5M2);
    return lo | hi << 16;
}
__device__ __forceinline__ void from_e5m2x4(uint32_t four, float* f) {
    const uint32_t lo = __byte_perm(four, 0, 0x1404), hi = __byte_perm(four, 0, 0x3424);
    const float2 a = __half22float2(*reinterpret_cast<const __half2*>(&lo));
    const float2 b = __half22float2(*reinterpret_cast<const __half2*>(&hi));
    f[0] = a.x; f[1] = a.y; f[2] = b.x; f[3] = b.y;
}

// One lane of the warp, the same each time.
__device__ __forceinline__ bool elected() {
    uint32_t r;
    asm volatile("{\n\t.reg .pred p;\n\telect.sync _|p, 0xffffffff;\n\tselp.u32 %0, 1, 0, p;\n\t}" : "=r"(r));
    return r != 0;
}

// tc::mbar_wait with a limit of the caller's, in microseconds, counted in cycles of 2 GHz.  A try may rest for 10 us before it
// says no, so that waiting warps take no issue slots from working ones.
__device__ __forceinline__ bool try_long(uint64_t* bar, uint32_t parity) {
    uint32_t ok;
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "mbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2, %3;\n\t"
        "selp.u32 %0, 1, 0, p;\n\t}"
        : "=r"(ok)
        : "r"(smem_u32(bar)), "r"(parity), "r"(10000u)
        : "memory");
    return ok != 0;
}
// Without a rest.
__device__ __forceinline__ bool has_come(uint64_t* bar, uint32_t parity) {
    uint32_t ok;
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "mbarrier.test_wait.parity.shared::cta.b64 p, [%1], %2;\n\t"
        "selp.u32 %0, 1, 0, p;\n\t}"
        : "=r"(ok)
        : "r"(smem_u32(bar)), "r"(parity)
        : "memory");
    return ok != 0;
}
__device__ __forceinline__ bool wait_up_to(uint64_t* bar, uint32_t parity, int limit) {
    if (try_long(bar, parity)) return true;
    const long long t0 = clock64();
    for (uint32_t i = 0; i < (1u << 30); ++i) {
        if (try_long(bar, parity)) return true;
        if (clock64() - t0 > 2000ll * limit) break;
    }
    return false;
}

// ------------------------------------------------------------------ the list of work

// What a group brings: its rows in items of 256 (the last of 128 or fewer counts as one stream's), and its tiles.
struct GroupWork {
    int2 range;                            // sequences
    int tokens, tiles;
    int64_t rows;
    int pairs;                             // items of two streams a head
    bool half;                             // one of one stream behind them
    int64_t span;                          // of a head in the list

    __device__ __forceinline__ int64_t whole() const { return 2 * (int64_t)tiles + kItemCost; }
};
__device__ __forceinline__ GroupWork group_work(const CacheAttention& a, const PrefixPlan& plan, int g) {
    GroupWork w;
    w.range = group_range(a, g, a.B);
    w.tokens = shared_tokens(a, g, w.range);
    w.tiles = (int)(((int64_t)w.tokens + kTokens - 1) / kTokens);   // (tokens may be close to 2^31)
    w.rows = (int64_t)(w.range.y - w.range.x) * a.T_q * plan.group;
    const int left = (int)(w.rows % kPair);
    w.pairs = (int)(w.rows / kPair) + (left > kRows);
    w.half = left > 0 && left <= kRows;
    w.span = w.tiles == 0 ? 0 : w.pairs * w.whole() + (w.half ? w.tiles + kItemCost : 0);
    return w;
}

struct PrefixShare {
    int64_t begin, end, share, base;       // base: where group g begins in the list
    int g;                                 // -1: nothing
};

// One warp calls it; its lanes sum up some groups' spans each.
__device__ __forceinline__ PrefixShare find_prefix_share(const CacheAttention& a, const PrefixPlan& plan) {
    const int lane = threadIdx.x & 31;
    const int each = (a.n_groups + 31) / 32, g0 = lane * each;
    int64_t mine = 0;
    for (int g = g0; g < g0 + each && g < a.n_groups; ++g) mine += group_work(a, plan, g).span * a.H_kv;
    int64_t up = mine;
#pragma unroll
    for (int w = 1; w < 32; w <<= 1) {
        const int64_t x = __shfl_up_sync(0xffffffffu, up, w);
        if (lane >= w) up += x;
    }
    const int64_t total = __shfl_sync(0xffffffffu, up, 31);
    PrefixShare s;
    s.share = (total + gridDim.x - 1) / gridDim.x;
    if (s.share < kLeastShare) s.share = kLeastShare;
    s.begin = s.share * blockIdx.x;
    s.end = s.begin + s.share < total ? s.begin + s.share : total;
    int found = -1;
    int64_t base = up - mine;
    if (s.begin >= base && s.begin < up) {
        for (int g = g0; g < a.n_groups; ++g) {
            const int64_t w = group_work(a, plan, g).span * a.H_kv;
            if (s.begin < base + w) {
                found = g;
                break;
            }
            base += w;
        }
    }
    const uint32_t who = __ballot_sync(0xffffffffu, found >= 0);
    const int from = who ? __ffs(who) - 1 : 0;
    s.g = __shfl_sync(0xffffffffu, found, from);
    s.base = __shfl_sync(0xffffffffu, base, from);
    return s;
}

// Calls f(piece) for each piece of the share; returns the entry of `joins` for the item that begins here
// and ends in a later share.
template <typename F>
__device__ __forceinline__ int4 for_each_prefix_piece(const CacheAttention& a, const PrefixPlan& plan, const PrefixShare& s,
                                                      F f) {
    int4 join = make_int4(-1, 0, 0, 0);
    if (s.g < 0) return join;
    PrefixPiece p;
    p.g = s.g;
    int64_t base = s.base, at = s.begin;
    GroupWork w = group_work(a, plan, p.g);
    while (at < s.end) {
        while (at >= base + w.span * a.H_kv) {             // (the share goes on: there is one)
            base += w.span * a.H_kv;
            w = group_work(a, plan, ++p.g);
        }
        p.hk = (int)((at - base) / w.span);
        const int64_t in_head = (at - base) % w.span;
        p.rows256 = (int)(in_head / w.whole());
        p.two = p.rows256 < w.pairs;
        const int64_t item = at - (in_head - p.rows256 * w.whole());
        const int64_t item_end = item + (p.two ? w.whole() : w.tiles + kItemCost);
        const int64_t stop = item_end < s.end ? item_end : s.end;
        auto tile_at = [&](int64_t x) { return x <= kItemCost ? 0 : (int)((x - kItemCost) >> (p.two ? 1 : 0)); };
        p.from = tile_at(at - item);
        p.to = tile_at(stop - item);
        if (p.from < p.to) {
            p.whole = p.from == 0 && p.to == w.tiles;
            p.slot = at == s.begin ? 0 : 1;
            p.first_seq = w.range.x;
            p.tokens = w.tokens;
            p.rows = w.rows;
            f(p);
            if (!p.whole && p.from == 0) join = make_int4(p.g, p.hk, (int)((item_end - 1) / s.share), 2 * p.rows256 + p.slot);
        }
        at = stop;
    }
    return join;
}

// Row r of a group's rows, as a row of o.
__device__ __forceinline__ int64_t prefix_row(const CacheAttention& a, const PrefixPlan& plan, int first_seq, int hk,
                                              int64_t r) {
    const int64_t i = r / plan.group;
    return ((int64_t)first_seq * a.T_q + i) * a.H_q + hk * plan.group + (int)(r - i * plan.group);
}

struct Cta {
    const CacheAttention& a;
    const PrefixPlan& plan;
    uint8_t* sm;
    Small* small;
    uint32_t tmem;
};

__device__ __forceinline__ float max3(float a, float b, float c) {
    float r;
    asm("max.f32 %0, %1, %2, %3;" : "=f"(r) : "f"(a), "f"(b), "f"(c));
    return r;
}

// An arrival for a whole warp: what its lanes did before is done.  (Arrivals of single lanes at one barrier follow one
// another.)
__device__ __forceinline__ void arrive_warp(uint64_t* bar) {
    __syncwarp();
    if ((threadIdx.x & 31) == 0) tc::mbar_arrive(bar);
}

// A ring's next slot and the parity of its use.
template <int N>
struct Ring {
    int slot = 0;
    uint32_t phase = 0;
    bool again = false;                    // every slot has been used
    __device__ __forceinline__ void next() {
        if (++slot == N) {
            slot = 0;
            phase ^= 1;
            again = true;
        }
    }
    __device__ __forceinline__ void skip(int n) {
        const int at = slot + n % N;
        phase ^= (uint32_t)(n / N + at / N) & 1u;
        slot = at % N;
    }
};

// Calls f for each piece that the planner writes; whole warps.
template <typename F>
__device__ __forceinline__ void for_each_piece_told(const Cta& c, F f) {
    Ring<kPieceSlots> ring;
    for (;;) {
        if (!__all_sync(0xffffffffu, wait_up_to(&c.small->piece_full[ring.slot], ring.phase, kPatience * c.plan.stall.wait_us))) return;
        const PrefixPiece& p = c.small->piece[ring.slot];
        if (p.from >= p.to) return;
        f(p);
        arrive_warp(&c.small->piece_empty[ring.slot]);
        ring.next();
    }
}

// ------------------------------------------------------------------ loader
struct Loader {
    Cta c;
    const CUtensorMap* k_map;
    const CUtensorMap* v_map;
    Ring<kKeySlots> k;
    Ring<kRawSlots> raw;
    Ring<kScaleSlots> scale;
    int n = 0;                             // tiles begun
    bool dead = false;

    // All lanes call it, and agree.
    __device__ __forceinline__ void wait(uint64_t* bar, uint32_t parity) {
        if (!__all_sync(0xffffffffu, wait_up_to(bar, parity, c.plan.stall.wait_us))) dead = true;
    }

    __device__ __forceinline__ void piece(const PrefixPiece& told) {
        const CacheAttention& a = c.a;
        const int lane = threadIdx.x & 31;
        const struct { int hk, from, to, tokens; } p{told.hk, told.from, told.to, told.tokens};
        const int32_t* table = a.prefix_table + (int64_t)told.g * a.prefix_pages;
        const int page_mask = (1 << a.page_shift) - 1;
        const int box = a.page_shift >= 7 ? kSteps : 1 << (a.page_shift - 4);   // steps that one copy brings
        const bool leads = lane < kSteps && (lane & (box - 1)) == 0;
        const uint32_t box_bytes = box * kStep * 128;
        // Lane k < 8: step k of a tile.
        auto page_of = [&](int tile) -> int {
            const uint32_t t = (uint32_t)(tile * kSteps + lane) * kStep;
            const int id = lane < kSteps && tile < p.to && t < (uint32_t)p.tokens ? table[t >> a.page_shift] : -1;
            return id >= 0 && id < a.n_pages ? id : -1;
        };
        auto scales_of = [&](int id, float& ks, float& vs) {
            const int64_t at = (int64_t)id * a.H_kv + p.hk;
            ks = id >= 0 ? a.k_scale[at] : 0.0f;
            vs = id >= 0 ? a.v_scale[at] : 0.0f;
        };
        int id = page_of(p.from), id_next = page_of(p.from + 1);
        float ks, vs;
        scales_of(id, ks, vs);
        for (int tile = p.from; tile < p.to; ++tile, ++n) {
            if (n >= c.plan.stall.loads) dead = true;
            if (dead) return;
            const int t0 = (tile * kSteps + lane) * kStep;
            const int y = p.hk * (page_mask + 1) + (t0 & page_mask);
            const uint32_t held = __ballot_sync(0xffffffffu, id >= 0) & 0xffu;
            const uint32_t bytes = __popc(__ballot_sync(0xffffffffu, leads && id >= 0)) * box_bytes;
            const int id_now = id;
            const float ks_now = ks, vs_now = vs;
            id = id_next;
            scales_of(id, ks, vs);
            id_next = page_of(tile + 2);

            if (n >= kKeySlots) wait(&c.small->k_empty[k.slot], k.phase ^ 1);
            if (dead) return;
            if (lane == 0) tc::mbar_expect_tx(&c.small->k_full[k.slot], bytes);
            __syncwarp();
            if (leads && id_now >= 0)
                tc::tma_load_3d(c.sm + kKeysAt + k.slot * kTile + lane * kStep * 128, k_map, 0, y, id_now,
                                &c.small->k_full[k.slot]);
            k.next();

            // Scales of values are powers of two but where a caller made them otherwise; what has none does not exist.
            const uint32_t bits = __float_as_uint(vs_now);
            const bool real = vs_now > 0.0f && bits < 0x7f800000u;
            float log_vs = (float)((int)(bits >> 23) - 127);
            if (bits & 0x7fffffu) log_vs += log2f(__uint_as_float((bits & 0x7fffffu) | 0x3f800000u));
            const uint32_t mask = held & __ballot_sync(0xffffffffu, real);
            Scales* to = &c.small->scales[scale.slot];
            if (lane < kSteps) to->step[lane] = make_float2(real ? ks_now : 0.0f, real ? log_vs : 0.0f);
            float lowest = real && id_now >= 0 ? log_vs : INFINITY;
#pragma unroll
            for (int x = 1; x < kSteps; x <<= 1) lowest = fminf(lowest, __shfl_xor_sync(0xffffffffu, lowest, x));
            if (lane == 0) {
                to->mask = mask;
                to->lowest = lowest;
            }
            __syncwarp();
            if (lane == 0) tc::mbar_arrive(&c.small->scale_full[scale.slot]);
            scale.next();

            if (n >= kRawSlots) wait(&c.small->raw_empty[raw.slot], raw.phase ^ 1);
            if (dead) return;
            if (lane == 0) tc::mbar_expect_tx(&c.small->raw_full[raw.slot], bytes);
            __syncwarp();
            if (leads && id_now >= 0)
                tc::tma_load_3d(c.sm + kRawAt + raw.slot * kTile + lane * kStep * 128, v_map, 0, y, id_now,
                                &c.small->raw_full[raw.slot]);
            raw.next();
        }
    }
    // No copy is under way when the CTA ends: what was asked for and not waited for by others is waited for here.
    __device__ __forceinline__ void finish() {
        for (int i = 0; i < kKeySlots; ++i) {
            if (k.slot > i || k.again) tc::mbar_wait(&c.small->k_full[i], k.slot > i ? k.phase : k.phase ^ 1);
        }
        for (int i = 0; i < kRawSlots; ++i) {
            if (raw.slot > i || raw.again) tc::mbar_wait(&c.small->raw_full[i], raw.slot > i ? raw.phase : raw.phase ^ 1);
        }
    }
};

// ------------------------------------------------------------------ converters
struct Converter {
    Cta c;
    Ring<kRawSlots> raw;
    Ring<kValueSlots> v;
    Ring<kScaleSlots> scale;
    int n = 0;
    bool dead = false;

    __device__ __forceinline__ void wait(uint64_t* bar, uint32_t parity) {
        if (!dead && !__all_sync(0xffffffffu, wait_up_to(bar, parity, c.plan.stall.wait_us))) dead = true;
    }

    __device__ __forceinline__ void piece(const PrefixPiece& p) {
        const int tid = threadIdx.x - kConverterWarp * 32;
        const int row0 = tid >> 3, chunk = tid & 7;        // eight threads a token, 16 channels each
        for (int left = p.to - p.from; left > 0; --left, ++n) {
            wait(&c.small->scale_full[scale.slot], scale.phase);
            wait(&c.small->raw_full[raw.slot], raw.phase);
            if (n >= kValueSlots) wait(&c.small->v_empty[v.slot], v.phase ^ 1);
            if (dead) return;
            const uint32_t mask = c.small->scales[scale.slot].mask;
            const uint8_t* from = c.sm + kRawAt + raw.slot * kTile;
            uint8_t* to = c.sm + kValuesAt + v.slot * kValueTile + (chunk >> 2) * kTile;
#pragma unroll 2
            for (int j = 0; j < kSteps; ++j) {
                const int t = j * kStep + row0;
                uint4 code = *reinterpret_cast<const uint4*>(from + tc::sw128(t, chunk));
                if (!(mask >> j & 1)) code = make_uint4(0, 0, 0, 0);
                const uint32_t word[4] = {code.x, code.y, code.z, code.w};
                uint32_t half[8];
#pragma unroll
                for (int i = 0; i < 4; ++i) word_to_half2x2(word[i], half[2 * i], half[2 * i + 1]);
                // (the upper four threads of a token store their second piece first: no two meet in a bank)
                const int c0 = 2 * (chunk & 3), late = chunk >> 2;
                const uint4 first = late ? make_uint4(half[4], half[5], half[6], half[7]) : make_uint4(half[0], half[1], half[2], half[3]);
                const uint4 second = late ? make_uint4(half[0], half[1], half[2], half[3]) : make_uint4(half[4], half[5], half[6], half[7]);
                *reinterpret_cast<uint4*>(to + tc::sw128(t, c0 + late)) = first;
                *reinterpret_cast<uint4*>(to + tc::sw128(t, c0 + 1 - late)) = second;
            }
            tc::fence_async_smem();
            arrive_warp(&c.small->v_full[v.slot]);
            arrive_warp(&c.small->raw_empty[raw.slot]);
            raw.next();
            v.next();
            scale.next();
        }
    }
};

// ------------------------------------------------------------------ issuer
// A unit is a stream's tile: O += W V of it, then, once these products have read W, S of the stream's next tile,
// which goes where W lies.  Both streams' units are taken as their weights come, each to its end: so one stream's
// products run under the other's softmax, and not both under neither.  (An issuer a stream, or one that takes whatever products are
// ready: the streams fall into step, both softmaxes at once and then all products; 23 to 34 us more for 256 sequences behind
// 32,768 tokens.)
struct Issuer {
    Cta c;
    Ring<kKeySlots> k[2];                  // of each stream's next unit
    Ring<kValueSlots> v[2];
    bool k_here[2] = {false, false}, v_here[2] = {false, false};   // their tiles have been seen to be there
    uint32_t phase[2] = {0, 0};            // of each stream's weights
    uint32_t q_phase = 0;
    int tiles = 0;
    bool dead = false;

    // All lanes call everything, and agree; one of them issues.  (With one thread alone a product took 105 cycles to issue,
    // its descriptors moved to uniform registers one by one; the product takes 64.)
    __device__ __forceinline__ void wait(uint64_t* bar, uint32_t parity) {
        if (!dead && !__all_sync(0xffffffffu, wait_up_to(bar, parity, c.plan.stall.wait_us))) dead = true;
    }
    template <int CHUNKS>
    static __device__ __forceinline__ void score_products(uint32_t d_tmem, uint32_t q, uint32_t keys) {
        mma_f8<false>(d_tmem, q, keys, idesc(128, kTokens, 1, false));
#pragma unroll
        for (int x = 1; x < CHUNKS; ++x) mma_f8<true>(d_tmem, q + 2 * x, keys + 2 * x, idesc(128, kTokens, 1, false));
#pragma unroll
        for (int x = 0; x < CHUNKS; ++x)
            mma_f8<true>(d_tmem, q + (kTile >> 4) + 2 * x, keys + 2 * x, idesc(128, kTokens, 0, false));
    }
    // A tile that both streams read is given back by both; one that only one does, by that one twice.
    static __device__ __forceinline__ void give_back(uint64_t* bar, bool two) {
        tc::mma_commit(bar);
        if (!two) tc::mma_commit(bar);
    }
    template <int STREAM>
    __device__ __forceinline__ void scores(bool two, bool later) {
        if (tiles++ / 2 >= c.plan.stall.tiles) dead = true;
        const int slot = k[STREAM].slot;
        if (!k_here[STREAM]) wait(&c.small->k_full[slot], k[STREAM].phase);
        if (later) wait(&c.small->o_done[STREAM], phase[STREAM] ^ 1);
        if (dead) return;
        tc::tc_fence_after();
        const uint32_t base = smem_u32(c.sm), keys = desc_low(base + kKeysAt + slot * kTile, 16);
        const uint32_t q = desc_low(base + kQueriesAt + 2 * STREAM * kTile, 16), to = c.tmem + 128 * STREAM;
        const int chunks = (c.a.d + 31) / 32;              // 32 channels a product
        if (elected()) {
            if (chunks == 4) score_products<4>(to, q, keys);
            else if (chunks == 3) score_products<3>(to, q, keys);
            else if (chunks == 2) score_products<2>(to, q, keys);
            else score_products<1>(to, q, keys);
            tc::mma_commit(&c.small->s_full[STREAM]);
            give_back(&c.small->k_empty[slot], two);
        }
        __syncwarp();
        k[STREAM].next();
        if (!two) k[STREAM].next();
    }
    // `fresh`: O has no sums yet.  The weights have come.
    template <int STREAM>
    __device__ __forceinline__ void values(bool two, bool fresh) {
        const int slot = v[STREAM].slot;
        if (!v_here[STREAM]) wait(&c.small->v_full[slot], v[STREAM].phase);
        if (dead) return;
        tc::tc_fence_after();
        const uint32_t values = desc_low(smem_u32(c.sm) + kValuesAt + slot * kValueTile, kTile);
        const uint32_t from = c.tmem + 128 * STREAM, to = from + kTmemO, desc = idesc(128, c.a.d, 0, true);
        if (elected()) {
            mma_f16_ta(to, from, values, desc, !fresh);
#pragma unroll
            for (int x = 1; x < kSteps; ++x)               // 16 tokens a product
                mma_f16_ta(to, from + 8 * x + (x >= kSteps / 2 ? 32 : 0), values + x * (kStep * 128 >> 4), desc, true);
            tc::mma_commit(&c.small->o_done[STREAM]);
            give_back(&c.small->v_empty[slot], two);
        }
        __syncwarp();
        phase[STREAM] ^= 1;
        v[STREAM].next();
        if (!two) v[STREAM].next();
    }
    // `done` units of this stream are, and `others` of the other's.  A stream is at most one unit ahead, and the second not at all
    // where it has the odd tiles: then the slots that the unit's tiles, and all tiles before them, lie in were given back by products
    // already issued, so that no wait here is for products that come after it, and a slot's barrier is at most one phase behind.
    template <int STREAM>
    static __device__ __forceinline__ bool in_turn(bool two, int done, int others) { return done <= others + (STREAM == 0 || two); }
    template <int STREAM>
    __device__ __forceinline__ bool unit(bool two, int done, int units, int others) {
        if (done == units || !in_turn<STREAM>(two, done, others) ||
            !__all_sync(0xffffffffu, has_come(&c.small->p_full[STREAM], phase[STREAM])))
            return false;
        values<STREAM>(two, done % kRun == 0);
        if (done + 1 < units && !dead) scores<STREAM>(two, true);
        look<STREAM>(two);
        return true;
    }
    // Whether the next unit's tiles are there, asked while products run and not when they are needed.  (Keys where this stream
    // has had every tile: what lay in the slot before may else be the other's, and still to come.)
    template <int STREAM>
    __device__ __forceinline__ void look(bool two) {
        k_here[STREAM] = two && __all_sync(0xffffffffu, has_come(&c.small->k_full[k[STREAM].slot], k[STREAM].phase));
        v_here[STREAM] = __all_sync(0xffffffffu, has_come(&c.small->v_full[v[STREAM].slot], v[STREAM].phase));
    }
    __device__ __forceinline__ void piece(const PrefixPiece& p) {
        const bool two = p.two;
        const int n = p.to - p.from, n0 = two ? n : (n + 1) >> 1, n1 = two ? n : n >> 1;
        wait(&c.small->q_full[0], q_phase);
        wait(&c.small->q_full[1], q_phase);
        q_phase ^= 1;
        Ring<kKeySlots> k_begin = k[0];
        Ring<kValueSlots> v_begin = v[0];
        if (!two) {                                        // the second stream's first tile is the second
            k[1].next();
            v[1].next();
        }
        k_here[0] = k_here[1] = v_here[0] = v_here[1] = false;
        if (!dead) scores<0>(two, false);
        if (n1 > 0 && !dead) scores<1>(two, false);
        int d0 = 0, d1 = 0;
        long long t0 = 0;
        for (uint32_t idle = 0; (d0 < n0 || d1 < n1) && !dead;) {
            const bool a = unit<0>(two, d0, n0, d1);
            d0 += a;
            const bool b = !dead && unit<1>(two, d1, n1, d0);
            d1 += b;
            if (a || b) {
                idle = 0;
            } else if ((++idle & 15u) == 0) {              // as in wait_up_to
                if (idle == 16) t0 = clock64();
                dead = __any_sync(0xffffffffu, clock64() - t0 > 2000ll * c.plan.stall.wait_us);
            }
        }
        k_begin.skip(n);
        v_begin.skip(n);
        k[0] = k[1] = k_begin;
        v[0] = v[1] = v_begin;
    }
    // Every product issued has ended, whether or not a wait gave up before, so that TMEM may go.
    __device__ __forceinline__ void finish() {
        if (elected()) tc::mma_commit(&c.small->drained);
        tc::mbar_wait(&c.small->drained, 0);
    }
};

// ------------------------------------------------------------------ softmax
// Whether any of the 64 threads at barrier `id` says yes.
__device__ __forceinline__ bool vote_rows(bool yes, uint32_t id) {
    uint32_t r;
    __syncwarp();
    asm volatile(
        "{\n\t.reg .pred p, q;\n\tsetp.ne.u32 p, %1, 0;\n\t"
        "bar.red.or.pred q, %2, 64, p;\n\tselp.u32 %0, 1, 0, q;\n\t}"
        : "=r"(r)
        : "r"((uint32_t)yes), "r"(id)
        : "memory");
    return r != 0;
}

// A stream's two warpgroups: a thread has one row and half of a tile's tokens, then half of O's columns.  References are the
// same in both halves.
struct Softmax {
    Cta c;
    int stream, half;
    Ring<kScaleSlots> scale;
    uint32_t s_phase = 0;                  // of this stream's units
    bool bad = false;                      // a wait of this warp gave up: it waits no more, its numbers are none

    __device__ __forceinline__ void wait(uint64_t* bar, uint32_t parity) {
        if (!bad && !__all_sync(0xffffffffu, wait_up_to(bar, parity, c.plan.stall.wait_us))) bad = true;
        __syncwarp();                                      // (what follows is done by whole warps)
    }

    // The stream's 128 queries: eight threads a row, 16 channels each.  (A loop, the next row's loads under this one's
    // work: unrolled, its instructions took longer to come than the queries.)
    __device__ __forceinline__ void load_queries(const PrefixPiece& p) {
        const CacheAttention& a = c.a;
        const int tid = threadIdx.x & (kStream - 1), part = tid & 7;
        constexpr int kStride = kStream / 8;
        const int64_t first = (int64_t)p.rows256 * kPair + (p.two ? stream * kRows : 0), rows = p.rows;
        const int64_t token0 = (int64_t)p.first_seq * a.T_q;
        const int head0 = p.hk * c.plan.group;
        const float sign = a.scale < 0.0f ? -1.0f : 1.0f;
        uint8_t* to = c.sm + kQueriesAt + 2 * stream * kTile;
        auto load = [&](int r, uint4 (&raw)[2]) {
            const int64_t at = first + r;
            const bool real = r < kRows && at < rows;
            const int64_t i = real ? at / c.plan.group : 0;
            const __nv_bfloat16* q = static_cast<const __nv_bfloat16*>(a.q) + (token0 + i) * a.q_stride +
                                     (int64_t)(head0 + (real ? (int)(at - i * c.plan.group) : 0)) * a.d + 16 * part;
#pragma unroll
            for (int x = 0; x < 2; ++x)
                raw[x] = real && 16 * part < a.d ? reinterpret_cast<const uint4*>(q)[x] : make_uint4(0, 0, 0, 0);
        };
        uint4 next[2];
        load(tid >> 3, next);
#pragma unroll 1
        for (int r = tid >> 3; r < kRows; r += kStride) {
            uint4 raw[2] = {next[0], next[1]};
            load(r + kStride, next);
            const __nv_bfloat16* e = reinterpret_cast<const __nv_bfloat16*>(raw);
            float amax = 0.0f;
            bool number = true;
#pragma unroll
            for (int x = 0; x < 16; ++x) {
                const float f = fabsf(to_f32(e[x]));
                number &= f <= INFINITY;
                amax = fmaxf(amax, f);
            }
#pragma unroll
            for (int s = 1; s < 8; s <<= 1) amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, s));
            number = (__ballot_sync(0xffffffffu, !number) >> (threadIdx.x & 24) & 255u) == 0;
            // 2^ex <= amax < 2^(ex + 1): times 2^(11 - ex), so that what e5m2 leaves, 2^-4 of it at most, is under e4m3's
            // largest value.  A row with an infinity: its scores are infinite or no numbers whatever its finite channels
            // hold, so these count as zeros, under no scale.  A row with a NaN has it from its factor.
            const bool infinite = amax == INFINITY;
            int ex = infinite ? 11 : (int)(__float_as_uint(amax) >> 23) - 127;
            ex = ex < -112 ? -112 : ex;
            const float up = sign * __uint_as_float((uint32_t)(127 + 11 - ex) << 23);
            uint32_t one[4], two[4];
#pragma unroll
            for (int v = 0; v < 4; ++v) {
                float x[4], f[4];
#pragma unroll
                for (int y = 0; y < 4; ++y) x[y] = number ? to_f32(e[4 * v + y]) * up : 0.0f;
                one[v] = to_e5m2x4(x[0], x[1], x[2], x[3]);
                from_e5m2x4(one[v], f);
                two[v] = to_e4m3x4(x[0] - f[0], x[1] - f[1], x[2] - f[2], x[3] - f[3]);
                if (infinite) {                            // its infinities alone: 7c
                    one[v] = two[v] = 0;
#pragma unroll
                    for (int y = 0; y < 4; ++y) {
                        const uint32_t bits = __float_as_uint(to_f32(e[4 * v + y]) * sign);
                        if (number && (bits & 0x7fffffffu) == 0x7f800000u) one[v] |= (bits >> 24 & 0x80u | 0x7cu) << (8 * y);
                    }
                }
            }
            *reinterpret_cast<uint4*>(to + tc::sw128(r, part)) = make_uint4(one[0], one[1], one[2], one[3]);
            *reinterpret_cast<uint4*>(to + kTile + tc::sw128(r, part)) = make_uint4(two[0], two[1], two[2], two[3]);
            if (part == 0)
                c.small->factor[stream * kRows + r] =
                    number ? fabsf(a.scale) * 1.4426950408889634f * __uint_as_float((uint32_t)(127 + ex - 11) << 23) : NAN;
        }
    }

    __device__ __forceinline__ float4* run_at(int row) const {
        return reinterpret_cast<float4*>(c.plan.runs) + ((int64_t)blockIdx.x * 2 + stream) * 32 * kRows + row;
    }

    // Columns [c0, c1) of O, its products ended, go to the sums of runs, which are 2^shift of what they were.  (`first`:
    // there are none.)
    static __device__ __noinline__ void add_run(uint32_t at, float4* runs, int c0, int c1, bool first, float shift) {
        const float keep = ex2(shift);
#pragma unroll 1
        for (int ch = c0; ch < c1; ch += 16) {
            float o[16];
            tc::tmem_ld16(at + ch, o);
            loaded16(o);
#pragma unroll
            for (int x = 0; x < 4; ++x) {
                float4* to = runs + (ch / 4 + x) * kRows;
                float4 r = first ? make_float4(0.0f, 0.0f, 0.0f, 0.0f) : *to;
                r = make_float4(fmaf(r.x, keep, o[4 * x]), fmaf(r.y, keep, o[4 * x + 1]), fmaf(r.z, keep, o[4 * x + 2]),
                                fmaf(r.w, keep, o[4 * x + 3]));
                *to = r;
            }
        }
    }

    // Columns [c0, c1) of O multiplied in place.
    static __device__ __noinline__ void scale_sums(uint32_t at, int c0, int c1, float keep) {
#pragma unroll 1
        for (int ch = c0; ch < c1; ch += 32) {             // (16 columns at the end are read twice, and one of the two kept)
            const bool two = ch + 16 < c1;
            float o[32];
            tc::tmem_ld16(at + ch, *reinterpret_cast<float(*)[16]>(o));
            tc::tmem_ld16(at + ch + (two ? 16 : 0), *reinterpret_cast<float(*)[16]>(o + 16));
            loaded16(o);
            loaded16(o + 16);
            uint32_t out[32];
#pragma unroll
            for (int x = 0; x < 32; ++x) out[x] = __float_as_uint(o[x] * keep);
            tc::tmem_st16(at + ch, *reinterpret_cast<uint32_t(*)[16]>(out));
            if (two) tc::tmem_st16(at + ch + 16, *reinterpret_cast<uint32_t(*)[16]>(out + 16));
        }
    }
    // Weights where steps are missing, scores are beyond 2^22, or pages of values so small beside others that their weights
    // are lost: the sum of weights by itself, which it returns.
    static __device__ __noinline__ float far_weights(uint32_t at, const Scales* sc, int half, float factor, float m, float dr) {
        float l = 0.0f;
#pragma unroll 1
        for (int h = 0; h < 2; ++h) {
            uint32_t out[16];
#pragma unroll 1
            for (int j = 0; j < 2; ++j) {
                float s[16];
                tc::tmem_ld16(at + 32 * h + 16 * j, s);
                loaded16(s);
                const float2 st = sc->step[4 * half + 2 * h + j];
                const bool real = sc->mask >> (4 * half + 2 * h + j) & 1;
                const float f = factor * st.x, lift = st.y - dr + kBits;
                uint32_t eight[8];
#pragma unroll
                for (int x = 0; x < 8; ++x) {
                    const float z0 = __fsub_rn(__fmul_rn(s[2 * x], f), m);
                    const float z1 = __fsub_rn(__fmul_rn(s[2 * x + 1], f), m);
                    if (real) l += ex2(z0) + ex2(z1);
                    eight[x] = real ? half2_bits(ex2(z0 + lift), ex2(z1 + lift)) : 0u;
                }
#pragma unroll
                for (int x = 0; x < 8; ++x) {
                    out[x] = j == 0 ? eight[x] : out[x];
                    out[8 + x] = eight[x];
                }
            }
            tc::tmem_st16(at + 16 * h, out);
        }
        return l;
    }

    __device__ __forceinline__ void piece(const PrefixPiece& p) {
        const CacheAttention& a = c.a;
        const int row = threadIdx.x & (kRows - 1);
        const uint32_t id = kBarRows + 4 * stream + (row >> 5);
        const uint32_t lanes = (uint32_t)(row & 96) << 16;
        // This thread's scores, then (from their first column on) its weights.
        const uint32_t s_at = c.tmem + lanes + 128 * stream + 64 * half, o_at = c.tmem + lanes + 128 * stream + kTmemO;
        const int middle = (a.d / 16 + 1) / 2 * 16, c0 = half ? middle : 0, c1 = half ? a.d : middle;
        load_queries(p);
        tc::fence_async_smem();
        tc::named_bar_sync(kBarStream + stream, kStream);
        if (threadIdx.x % kStream == 0) tc::mbar_arrive(&c.small->q_full[stream]);
        const float factor = c.small->factor[stream * kRows + row];

        // m: the largest score so far, rounded up (or 0: none); weights are relative to m + dr.
        float m = 0.0f, dr = 0.0f, l = 0.0f, shift = 0.0f;
        bool seen = false;
        const bool two = p.two;
        const int tiles = p.to - p.from, units = two ? tiles : (tiles + 1 - stream) >> 1;
        if (!two && stream) scale.next();
#pragma unroll 1
        for (int k = 0; k < units; ++k) {
            wait(&c.small->scale_full[scale.slot], scale.phase);
            wait(&c.small->s_full[stream], s_phase);
            tc::tc_fence_after();
            const Scales* sc = &c.small->scales[scale.slot];
            const bool fresh = k % kRun == 0;              // no sums in O
            if (fresh && k > 0) {
                wait(&c.small->o_done[stream], s_phase ^ 1);
                tc::tc_fence_after();
                if (!bad) add_run(o_at, run_at(row), c0, c1, k == kRun, shift);
                shift = 0.0f;
            }
            // Scores are loaded twice, 32 tokens at a time: for the largest, then for the weights.
            const uint32_t mine = sc->mask >> (kSteps / 2 * half);
            float xs[kSteps / 2], top = -INFINITY, reach = -INFINITY;
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                float now[32];
                load32(s_at + 32 * h, now);
                const float4 st = *reinterpret_cast<const float4*>(&sc->step[kSteps / 2 * half + 2 * h]);
                loaded16(now);
                loaded16(now + 16);
#pragma unroll
                for (int j = 0; j < 2; ++j) {
                    float some[5];
#pragma unroll
                    for (int x = 0; x < 5; ++x) some[x] = max3(now[16 * j + 3 * x], now[16 * j + 3 * x + 1], now[16 * j + 3 * x + 2]);
                    const float most = fmaxf(max3(some[0], some[1], some[2]), max3(some[3], some[4], now[16 * j + 15]));
                    const float x = mine >> (2 * h + j) & 1 ? __fmul_rn(most, factor * (j ? st.z : st.x)) : -INFINITY;
                    xs[2 * h + j] = x;
                    top = fmaxf(top, x);
                    reach = fmaxf(reach, (x - m) + (j ? st.w : st.y));   // (m first: it may have no places to add to)
                }
            }
            // Where a weight would be too large, by its page's values or (on pages of values far smaller than others) by its score
            // alone, all references of the two warps' rows move to the largest so far.
            if (vote_rows(reach - dr > kFar || top - m > kFarScore || (!seen && top > -INFINITY), id)) {
                c.small->top[stream][half][row] = top;
                tc::named_bar_sync(id, 64);
                top = fmaxf(top, c.small->top[stream][half ^ 1][row]);
                const bool found = top > -INFINITY;
                const float m_new = !found ? m : seen ? fmaxf(m, ceilf(top)) : ceilf(top);
                // (differences of rounded products: scores whose last places are whole numbers still give the largest
                // one's value)
                reach = -INFINITY;
#pragma unroll
                for (int j = 0; j < kSteps / 2; ++j) reach = fmaxf(reach, __fsub_rn(xs[j], m_new) + sc->step[kSteps / 2 * half + j].y);
                c.small->reach[stream][half][row] = reach;
                tc::named_bar_sync(id, 64);
                reach = fmaxf(reach, c.small->reach[stream][half ^ 1][row]);
                const float dr_old = dr + (seen ? m - m_new : 0.0f);
                const bool moves = found && (!seen || reach > dr_old);
                const float dr_new = moves ? ceilf(reach) : dr_old;
                const float move = seen && moves ? dr_old - dr_new : 0.0f;
                if (!fresh && __any_sync(0xffffffffu, move != 0.0f)) {
                    wait(&c.small->o_done[stream], s_phase ^ 1);
                    tc::tc_fence_after();
                    if (!bad) scale_sums(o_at, c0, c1, ex2(move));
                }
                l *= seen ? ex2(m - m_new) : 1.0f;
                shift += move;
                m = m_new;
                dr = dr_new;
                seen |= found;
            }
            // (the same in both halves)
            const bool near = __all_sync(0xffffffffu, fabsf(m) < kNear && dr - sc->lowest < 90.0f);
            if (near && sc->mask == (1u << kSteps) - 1) {
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                    float now[32];
                    load32(s_at + 32 * h, now);
                    const float4 st = *reinterpret_cast<const float4*>(&sc->step[kSteps / 2 * half + 2 * h]);
                    uint32_t out[16];
                    loaded16(now);
                    loaded16(now + 16);
#pragma unroll
                    for (int j = 0; j < 2; ++j) {
                        const float f = factor * (j ? st.z : st.x), lv = j ? st.w : st.y, less = (lv - dr + kBits) - m;
                        const uint64_t ff = f2_pack(f, f), cc = f2_pack(less, less);
                        uint64_t both = 0;
#pragma unroll
                        for (int x = 0; x < 8; ++x) {
                            const float2 e = f2_unpack(f2_fma(f2_pack(now[16 * j + 2 * x], now[16 * j + 2 * x + 1]), ff, cc));
                            const float w0 = ex2(e.x), w1 = ex2(e.y);
                            both = x == 0 ? f2_pack(w0, w1) : add_pair(both, f2_pack(w0, w1));
                            out[8 * j + x] = half2_bits(w0, w1);
                        }
                        const float2 two = f2_unpack(both);
                        l = fmaf(two.x + two.y, ex2(dr - kBits - lv), l);
                    }
                    tc::tmem_st16(s_at + 16 * h, out);
                }
            } else {
                l += far_weights(s_at, sc, half, factor, m, dr);
            }
            tc::tmem_wait_st();
            tc::tc_fence_before();
            arrive_warp(&c.small->p_full[stream]);
            s_phase ^= 1;
            scale.next();
            if (!two && 2 * k + stream + 1 < tiles) scale.next();
        }
        if (units > 0) wait(&c.small->o_done[stream], s_phase ^ 1);
        tc::tc_fence_after();

        // The end: both halves' sums of weights, and each half's columns.
        c.small->reach[stream][half][row] = bad ? NAN : l;
        tc::named_bar_sync(kBarStream + stream, kStream);
        const float L = c.small->reach[stream][0][row] + c.small->reach[stream][1][row];
        const float M = seen ? m : kLowest, DM = seen ? -dr - (kWeightBits - kBits) : 0.0f;
        const bool runs = units > kRun, none = units == 0;
        const float keep = ex2(shift);
        auto sums = [&](int ch, float (&o)[16]) {
            tc::tmem_ld16(o_at + ch, o);
            loaded16(o);
            if (runs) {
#pragma unroll
                for (int x = 0; x < 4; ++x) {
                    const float4 r = run_at(row)[(ch / 4 + x) * kRows];
                    o[4 * x] = fmaf(r.x, keep, o[4 * x]);
                    o[4 * x + 1] = fmaf(r.y, keep, o[4 * x + 1]);
                    o[4 * x + 2] = fmaf(r.z, keep, o[4 * x + 2]);
                    o[4 * x + 3] = fmaf(r.w, keep, o[4 * x + 3]);
                }
            }
            if (bad || none) {
#pragma unroll
                for (int x = 0; x < 16; ++x) o[x] = bad ? NAN : 0.0f;
            }
        };
        // Where both streams have the same rows, the second's sums go through the queries' place, whose products have ended.
        float4* other = two ? nullptr : reinterpret_cast<float4*>(c.sm + kQueriesAt) + row;
        float4 stat = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
        if (!two) {
            tc::named_bar_sync(kBarBoth, 2 * kStream);
            if (stream == 1) {
#pragma unroll 1
                for (int ch = c0; ch < c1; ch += 16) {
                    float o[16];
                    sums(ch, o);
#pragma unroll
                    for (int x = 0; x < 4; ++x)
                        other[(ch / 4 + x) * kRows] = make_float4(o[4 * x], o[4 * x + 1], o[4 * x + 2], o[4 * x + 3]);
                }
                if (half == 0) c.small->stat[row] = make_float4(M, DM, L, 0.0f);
            }
            tc::named_bar_sync(kBarBoth, 2 * kStream);
            stat = c.small->stat[row];
        }
        if (two || stream == 0) {
            // To what the row carries, or to the share's slot.
            const int r = (two ? stream * kRows : 0) + row;
            const int64_t at = (int64_t)p.rows256 * kPair + r;
            const bool real = at < p.rows;
            const int64_t out = !real    ? 0
                                : p.whole ? prefix_row(a, c.plan, p.first_seq, p.hk, at)
                                          : ((int64_t)blockIdx.x * 2 + p.slot) * kPair + r;
            float* to = (p.whole ? a.carry_sums : c.plan.sums) + out * c.plan.D;
            // (join_sums' factors, once)
            const float m_all = other ? fmaxf(M, stat.x) : M, dm_all = other ? fminf(DM + (m_all - M), stat.y + (m_all - stat.x)) : DM;
            const float mine = other ? ex2(M - m_all + (dm_all - DM)) : 1.0f, its = other ? ex2(stat.x - m_all + (dm_all - stat.y)) : 0.0f;
#pragma unroll 1
            for (int ch = c0; ch < c1; ch += 16) {
                float o[16];
                sums(ch, o);                               // (by whole warps: from TMEM)
                if (other) {
#pragma unroll
                    for (int x = 0; x < 4; ++x) {
                        const float4 y = other[(ch / 4 + x) * kRows];
                        o[4 * x] = o[4 * x] * mine + y.x * its;
                        o[4 * x + 1] = o[4 * x + 1] * mine + y.y * its;
                        o[4 * x + 2] = o[4 * x + 2] * mine + y.z * its;
                        o[4 * x + 3] = o[4 * x + 3] * mine + y.w * its;
                    }
                }
                // (a thread has a row: whole sectors of 32 bytes at a time)
                if (real) {
                    store8(to + ch, o);
                    store8(to + ch + 8, o + 8);
                }
            }
            const float l_all = other ? L * ex2(M - m_all) + stat.z * ex2(stat.x - m_all) : L;
            if (real && half == 0) (p.whole ? a.carry_stats : c.plan.stats)[out] = make_float4(m_all, dm_all, l_all, 0.0f);
        }
        if (!two) tc::named_bar_sync(kBarBoth, 2 * kStream);   // before the queries' place is theirs again
        tc::tc_fence_before();                             // the next piece's products may overwrite the sums
    }
};

__global__ void __launch_bounds__(kThreads, 1)
    prefix_tc_kernel(const __grid_constant__ CacheAttention a, const __grid_constant__ PrefixPlan plan,
                     const __grid_constant__ CUtensorMap k_map, const __grid_constant__ CUtensorMap v_map) {
    extern __shared__ uint8_t smem_raw[];
    uint8_t* sm = smem_raw + ((1024u - (smem_u32(smem_raw) & 1023u)) & 1023u);
    Small* small = reinterpret_cast<Small*>(sm + kSmallAt);
    const int warp = threadIdx.x >> 5;
    after_the_kernel_before();
    if (threadIdx.x == 0) {
        for (int i = 0; i < kKeySlots; ++i) {
            tc::mbar_init(&small->k_full[i], 1);
            tc::mbar_init(&small->k_empty[i], 2);
        }
        for (int i = 0; i < kRawSlots; ++i) {
            tc::mbar_init(&small->raw_full[i], 1);
            tc::mbar_init(&small->raw_empty[i], kWarpgroup / 32);
        }
        for (int i = 0; i < kValueSlots; ++i) {
            tc::mbar_init(&small->v_full[i], kWarpgroup / 32);
            tc::mbar_init(&small->v_empty[i], 2);
        }
        for (int i = 0; i < kScaleSlots; ++i) tc::mbar_init(&small->scale_full[i], 1);
        for (int i = 0; i < kPieceSlots; ++i) {
            tc::mbar_init(&small->piece_full[i], 1);
            tc::mbar_init(&small->piece_empty[i], kPlannerWarp);   // the warps of the roles before the planner
        }
        for (int i = 0; i < 2; ++i) {
            tc::mbar_init(&small->s_full[i], 1);
            tc::mbar_init(&small->p_full[i], kStream / 32);
            tc::mbar_init(&small->o_done[i], 1);
            tc::mbar_init(&small->q_full[i], 1);
        }
        tc::mbar_init(&small->drained, 1);
        tc::fence_mbar_init();
    }
    if (warp == kIssuerWarp) tc::tmem_alloc<kTmemCols>(&small->tmem);
    tc::tc_fence_before();
    __syncthreads();
    tc::tc_fence_after();
    const Cta cta{a, plan, sm, small, small->tmem};
    if (warp < kConverterWarp) {
        asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(kSoftmaxRegs));
        Softmax role{cta, warp >> 3, warp >> 2 & 1};
        for_each_piece_told(cta, [&](const PrefixPiece& p) { role.piece(p); });
    } else {
        asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kOtherRegs));
        if (warp < kIssuerWarp) {
            Converter role{cta};
            for_each_piece_told(cta, [&](const PrefixPiece& p) {
                if (!role.dead) role.piece(p);
            });
        } else if (warp == kLoaderWarp) {
            Loader role{cta, &k_map, &v_map};
            for_each_piece_told(cta, [&](const PrefixPiece& p) {
                if (!role.dead) role.piece(p);
            });
            role.finish();
        } else if (warp == kIssuerWarp) {
            Issuer role{cta};
            for_each_piece_told(cta, [&](const PrefixPiece& p) {
                if (!role.dead) role.piece(p);
            });
            role.finish();
        } else if (warp == kPlannerWarp) {
            const PrefixShare share = find_prefix_share(a, plan);
            Ring<kPieceSlots> ring;
            auto tell = [&](const PrefixPiece& p) {
                if (ring.again)
                    __all_sync(0xffffffffu, wait_up_to(&small->piece_empty[ring.slot], ring.phase ^ 1, kPatience * plan.stall.wait_us));
                if (elected()) {
                    small->piece[ring.slot] = p;
                    tc::mbar_arrive(&small->piece_full[ring.slot]);
                }
                __syncwarp();
                ring.next();
            };
            const int4 join = for_each_prefix_piece(a, plan, share, tell);
            PrefixPiece end = {};
            tell(end);
            if (elected()) plan.joins[blockIdx.x] = join;
        }
    }
    __syncwarp();
    tc::tc_fence_before();
    __syncthreads();
    if (warp == kIssuerWarp) {
        tc::tc_fence_after();
        tc::tmem_dealloc<kTmemCols>(cta.tmem);
    }
}

// The pieces of the item that begins in CTA blockIdx.x's share and ends in a later one, joined in order to what its rows
// carry: a warp a row, four channels a lane.
constexpr int kJoinRows = 8;

__global__ void __launch_bounds__(32 * kJoinRows) prefix_join_kernel(const CacheAttention a, const PrefixPlan plan) {
    after_the_kernel_before();
    const int4 join = plan.joins[blockIdx.x];
    if (join.x < 0) return;
    const GroupWork w = group_work(a, plan, join.x);
    const int lane = threadIdx.x & 31, r = blockIdx.y * kJoinRows + (threadIdx.x >> 5);
    const int64_t at = (int64_t)(join.w >> 1) * kPair + r;
    if (at >= w.rows) return;
    const int n = join.z - (int)blockIdx.x + 1;
    const int ch = 4 * lane;
    float4 o = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
    float M = kLowest, DM = 0.0f, L = 0.0f;
    for (int i = 0; i < n; ++i) {
        const int64_t place = ((int64_t)(blockIdx.x + i) * 2 + (i == 0 ? join.w & 1 : 0)) * kPair + r;
        const float4 x = ch < a.d ? *reinterpret_cast<const float4*>(plan.sums + place * plan.D + ch) : make_float4(0.0f, 0.0f, 0.0f, 0.0f);
        const float4 s = plan.stats[place];
        if (i == 0) {
            o = x, M = s.x, DM = s.y, L = s.z;
        } else {
            join_sums(o, M, DM, L, s, x);
        }
    }
    const int64_t out = prefix_row(a, plan, w.range.x, join.y, at);
    if (ch < a.d) *reinterpret_cast<float4*>(a.carry_sums + out * plan.D + ch) = o;
    if (lane == 0) a.carry_stats[out] = make_float4(M, DM, L, 0.0f);
}

// cuTensorMapEncodeTiled through the runtime, so that the library does not link against the driver's.
PFN_cuTensorMapEncodeTiled_v12000 map_encoder() {
    static PFN_cuTensorMapEncodeTiled_v12000 fn = nullptr;
    static std::once_flag once;
    std::call_once(once, [] {
        void* p = nullptr;
        cudaDriverEntryPointQueryResult q;
        if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &p, 12000, cudaEnableDefault, &q) == cudaSuccess &&
            q == cudaDriverEntryPointSuccess)
            fn = reinterpret_cast<PFN_cuTensorMapEncodeTiled_v12000>(p);
    });
    return fn;
}
// The pool's codes: [page][head, token][channel], in boxes of up to 128 tokens whose channels from d to 128 come as zeros.
bool make_pool_map(CUtensorMap* map, const void* codes, const CacheAttention& a) {
    const PFN_cuTensorMapEncodeTiled_v12000 encode = map_encoder();
    if (!encode) return false;
    const int page = 1 << a.page_shift;
    cuuint64_t dims[3] = {(cuuint64_t)a.d, (cuuint64_t)a.H_kv * page, (cuuint64_t)a.n_pages};
    cuuint64_t strides[2] = {(cuuint64_t)a.d, (cuuint64_t)a.H_kv * page * a.d};
    cuuint32_t box[3] = {128, (cuuint32_t)(page < kTokens ? page : kTokens), 1};
    cuuint32_t one[3] = {1, 1, 1};
    return encode(map, CU_TENSOR_MAP_DATA_TYPE_UINT8, 3, const_cast<void*>(codes), dims, strides, box, one,
                  CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                  CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// CTAs: one an SM, or as many as have a share of the least size.
int64_t prefix_grid(const CacheAttention& a, int num_sms) {
    const int64_t rows = (int64_t)a.B * a.T_q * (a.H_q / a.H_kv);
    const int64_t tiles = (((int64_t)a.prefix_pages << a.page_shift) + kTokens - 1) / kTokens;
    const int64_t most = a.H_kv * (rows / kPair + a.n_groups) * (2 * tiles + kItemCost) / kLeastShare + 1;
    return most < num_sms ? most : num_sms;
}
size_t up256(size_t n) { return (n + 255) / 256 * 256; }

}  // namespace

size_t attention_prefix_tc_workspace_bytes(const CacheAttention& a, int num_sms) {
    const size_t grid = prefix_grid(a, num_sms), D = a.d <= 64 ? 64 : 128;
    return up256(grid * sizeof(int4)) + up256(grid * 2 * kPair * sizeof(float4)) + up256(grid * 2 * kPair * D * sizeof(float)) +
           grid * 2 * kRows * 128 * sizeof(float);
}

cudaError_t run_attention_prefix_tc(const CacheAttention& a, void* workspace, cudaStream_t stream, int num_sms) {
    const int64_t grid = prefix_grid(a, num_sms);
    PrefixPlan plan = {};
    plan.group = a.H_q / a.H_kv;
    plan.D = a.d <= 64 ? 64 : 128;
    plan.stall = attention_stall();
    uint8_t* at = static_cast<uint8_t*>(workspace);
    plan.joins = reinterpret_cast<int4*>(at);
    at += up256(grid * sizeof(int4));
    plan.stats = reinterpret_cast<float4*>(at);
    at += up256(grid * 2 * kPair * sizeof(float4));
    plan.sums = reinterpret_cast<float*>(at);
    at += up256(grid * 2 * kPair * plan.D * sizeof(float));
    plan.runs = reinterpret_cast<float*>(at);
    CUtensorMap k_map, v_map;
    if (!make_pool_map(&k_map, a.k_codes, a) || !make_pool_map(&v_map, a.v_codes, a)) return cudaErrorInvalidValue;
    cudaError_t e = cudaFuncSetAttribute(prefix_tc_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, kSmem);
    if (e != cudaSuccess) return e;
    e = launch_chained(prefix_tc_kernel, (unsigned)grid, kThreads, kSmem, stream, a, plan, k_map, v_map);
    if (e != cudaSuccess) return e;
    const int64_t rows = (int64_t)a.B * a.T_q * plan.group;
    const unsigned strips = (unsigned)((rows < kPair ? rows : kPair) + kJoinRows - 1) / kJoinRows;
    return launch_chained(prefix_join_kernel, dim3((unsigned)grid, strips), 32 * kJoinRows, 0, stream, a, plan);
}

}  // namespace kda
