// kda_cache_attention_tc.cu -- attention over the paged 8-bit cache for many bf16 rows: draft
// tokens and prompts, whose rows share each head's keys.
//
// The mathematics is that of kda_cache_attention.cu.  With more than some 16 rows a head the
// products there bound it (537 MB of codes under 32 rows: 170 us; here 134 us, 4.0 TB/s; 64 rows 330 and 240 us),
// above all the conversion of every code to fp16.  Here the codes go to the tensor cores as they lie in
// the cache, as e4m3 operands; what is not 8 bits is split instead:
//
//   S^T [128 tokens x 32]  = K [128 x d] (q1 + q2 + q3)^T      e5m2 pieces, which hold the 8 bits of a bf16 value exactly,
//                                                             down to 2^-30 of its row's largest
//   O^T [128 channels x 128] += V^T [128 x 128 tokens] (w1 | w2 | w3 | w4)
//                                                             w = w1 + w2 / 4 + w3 / 16 + w4 / 64, e5m2: a weight in fp16,
//                                                             cut into the top bytes of what remains of it
//
// Tokens (and then channels) are the 128 rows of a product and the pieces of 32 query rows its
// columns, so a thread has 16 rows' scores of one token, and writes their weights 16 bytes at a time.
// Weights keep 11 bits down to 2^-22 of the row's reference and are lost below 2^-30 of it.
//
// Roles of a CTA's eleven warps, two CTAs a SM, handing over by mbarriers:
//   8 softmax   scores from TMEM, weights to shared memory; two threads a token (four warps of
//               32 rows a thread took twice as long over a tile as the memory)
//   2 loaders   a ring of five half tiles (keys or values of 128 tokens, 16 KB), 16-byte asynchronous copies along
//               the rows into 128-byte-swizzled rows, zeros where there is no token
//   1 issuer    the score product of the next tile, then the value product of this one
// The maximum m and the reference of v's sums (kept as dm) are common to the CTA and move only when a
// score passes them by more than a factor of 128, which a vote of the four warps of its row tells; the sums in
// TMEM are then multiplied in place.  (A move takes 2,750 cycles, its wait for the products before it included; of pages
// that differ by 2^6 in size 19% of the tiles have one, with a factor of 4 every third had.)
//
// The products' own sums are cut off, not rounded, all the same way: values of one sign over 131,072 tokens came out 1.2e-4
// too small, and more so with the length.  So they hold kRun tiles (256 products, cut off by less than 2^-15 of their sum), then go to
// sums in TMEM by rounded additions.  (0.5 to 1% of the time of 65,536 tokens.)
//
// NaN that a row does not see (0 times NaN is NaN): see Softmax::mend_values.
//
// A wait that gives up (about 2 s) makes the outputs of the item and of the CTA's later ones NaN.  The lanes of a warp give up
// together, since what follows a wait is done by whole warps (loads from TMEM, shuffles); a warp that gave up waits no
// more, but still arrives where others wait; and TMEM is given back after the end of all products that were issued, by a barrier of
// their own.  kda_selftest_attention_stall has them run out.
#include "kda_attention_common.cuh"

namespace kda {
namespace {

using namespace attn;
using tc::smem_u32;

constexpr int kRows = 32;                  // query rows of a tile
constexpr int kTokens = 128;               // tokens of a tile: 8 steps
constexpr int kTileSteps = kTokens / kStep;
constexpr int kHalf = kTokens * 128;       // bytes of a tile's keys, or values
constexpr int kSlots = 5;
constexpr int kSoftmax = 256;              // threads of warps 0-7; then the loaders', and the issuer's warp
constexpr int kLoaders = 64;               // eight rows at a time
constexpr int kThreads = kSoftmax + 128;   // (whole warpgroups, for setmaxnreg: the last warp has no role)
constexpr int kIssuerWarp = (kSoftmax + kLoaders) / 32;
// Registers: 80 a thread at launch, then 96 for softmax and 48 for the others, all there are: 256 x 96 + 128 x 48 = 384 x 80.
// (40 for the others: their loops spill; 4 x 65,536 tokens of one size under 32 rows 129.9 us, 123.1 so.)
constexpr int kSoftmaxRegs = 96, kOtherRegs = 48;
static_assert(kSoftmax * kSoftmaxRegs + (kThreads - kSoftmax) * kOtherRegs <= kThreads * 80, "registers at launch");
constexpr int kMine = kRows / 2;           // rows of a softmax thread
constexpr float kBits = 8.0f, kFar = 7.0f;    // log2 of the largest weight at its reference, and of how far above it
constexpr float kToPlan = 16.0f;           // 2^(kWeightBits - kBits)
constexpr int kCtas = 2;                   // a SM
constexpr int kBarSoftmax = 1;             // named barriers: of all softmax warps,
constexpr int kBarHalf = 2;                // and (2 and 3) of the four that have the same 16 rows

// Shared memory, from a 1024-byte boundary.
constexpr int kRingAt = 0;
constexpr int kWeightsAt = kRingAt + kSlots * kHalf;            // [128 tokens][128 columns] e5m2
constexpr int kQueriesAt = kWeightsAt + kTokens * 128;          // [3 pieces][32][128 channels] e5m2
constexpr int kScalesAt = kQueriesAt + 3 * kRows * 128;         // [4 tiles][k, v][8 steps]
constexpr int kRowsAt = kScalesAt + 4 * 2 * kTileSteps * 4;     // Rows
constexpr int kRowsBytes = 2560;
constexpr int kBarriersAt = kRowsAt + kRowsBytes;
constexpr int kSmem = kBarriersAt + 256 + 1024;

struct alignas(16) Rows {
    float factor[kRows];                   // of the scores, to powers of two
    float m[kRows], dm[kRows];
    float lift[kRows];                     // 2^(dm + kWeightBits)
    float up[kRows];                       // by how much a reference moved,
    float keep_o[kRows], keep_l[kRows];    // and what that multiplies the sums by
    float dm_most[4];                      // of each 16 rows: the largest dm,
    uint32_t unset[2];                     // and those that have seen no score yet, a bit each: m = 0 is none of theirs
    uint32_t empty[2];                     // at the end: those whose sum of weights is 0
    float part[4][kRows], part_e[4][kRows];
    uint32_t nan[kRows][4];                // channels whose output is NaN, a bit each
};
static_assert(sizeof(Rows) <= kRowsBytes, "Rows");

struct Barriers {
    uint64_t full[kSlots], empty[kSlots], s_full[2], s_free[2], w_full, pv_done, q_full, drained;
    uint32_t tmem;
};

constexpr uint32_t kTmemCols = 256;        // S 2 x 32, sums 32, O 128
constexpr uint32_t kTmemSums = 64;
constexpr uint32_t kTmemO = 128;
constexpr int kRun = 64;                   // tiles that O sums up before it goes to the rounded sums

// kind::f8f6f4, fp32 sums: M x N, A e4m3; B e4m3 (0) or e5m2 (1); bits 15 and 16: A, B with M, N along
// the rows.
constexpr uint32_t idesc_f8(uint32_t M, uint32_t N, uint32_t b_format, bool a_mn, bool b_mn) {
    return (1u << 4) | (b_format << 10) | ((a_mn ? 1u : 0u) << 15) | ((b_mn ? 1u : 0u) << 16) | ((N >> 3) << 17) |
           ((M >> 4) << 24);
}
__device__ __forceinline__ void mma_f8(uint32_t d_tmem, uint64_t a, uint64_t b, uint32_t idesc, bool accumulate) {
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "setp.ne.b32 p, %4, 0;\n\t"
        "tcgen05.mma.cta_group::1.kind::f8f6f4 [%0], %1, %2, %3, p;\n\t}" ::"r"(d_tmem),
        "l"(a), "l"(b), "r"(idesc), "r"((uint32_t)accumulate)
        : "memory");
}

// Whether any of the `count` threads at barrier `id` says yes.
__device__ __forceinline__ bool vote(bool yes, uint32_t id, uint32_t count) {
    uint32_t r;
    asm volatile(
        "{\n\t.reg .pred p, q;\n\t"
        "setp.ne.u32 p, %1, 0;\n\t"
        "bar.red.or.pred q, %2, %3, p;\n\t"
        "selp.u32 %0, 1, 0, q;\n\t}"
        : "=r"(r)
        : "r"((uint32_t)yes), "r"(id), "r"(count)
        : "memory");
    return r != 0;
}

// Lanes 2 r and 2 r + 1 get the reduction over the warp of v[r]: halves are exchanged, 16 shuffles for
// 16 rows.
template <typename Op>
__device__ __forceinline__ float reduce_rows(const float (&v)[kMine], Op op) {
    const int lane = threadIdx.x & 31;
    float u[kMine];
#pragma unroll
    for (int i = 0; i < kMine; ++i) u[i] = v[i];
#pragma unroll
    for (int w = 16; w > 1; w >>= 1) {
        const bool up = lane & w;
#pragma unroll
        for (int i = 0; i < w / 2; ++i)
            u[i] = op(up ? u[i + w / 2] : u[i], __shfl_xor_sync(0xffffffffu, up ? u[i] : u[i + w / 2], w));
    }
    return op(u[0], __shfl_xor_sync(0xffffffffu, u[0], 1));
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

__device__ __forceinline__ uint32_t half2_sub(uint32_t a, uint32_t b) {
    uint32_t r;
    asm("sub.rn.f16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
    return r;
}
__device__ __forceinline__ uint32_t half2_times4(uint32_t a) {
    uint32_t r;
    asm("mul.rn.f16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(0x44004400u));
    return r;
}

// Waits for this thread's loads from TMEM; what they gave is used after it only.
__device__ __forceinline__ void loaded(float (&v)[16]) {
    asm volatile("tcgen05.wait::ld.sync.aligned;"
                 : "+f"(v[0]), "+f"(v[1]), "+f"(v[2]), "+f"(v[3]), "+f"(v[4]), "+f"(v[5]), "+f"(v[6]), "+f"(v[7]),
                   "+f"(v[8]), "+f"(v[9]), "+f"(v[10]), "+f"(v[11]), "+f"(v[12]), "+f"(v[13]), "+f"(v[14]), "+f"(v[15])
                 :
                 : "memory");
}

// tc::mbar_wait with a limit of the caller's, in microseconds.
__device__ __forceinline__ bool wait_up_to(uint64_t* bar, uint32_t parity, int limit) {
    if (tc::mbar_try_wait(bar, parity)) return true;
    const uint64_t t0 = tc::global_ns();
    for (uint32_t i = 0; i < (1u << 30); ++i) {
        if (tc::mbar_try_wait(bar, parity)) return true;
        if ((i & 15u) == 15u && tc::global_ns() - t0 > 1000ull * limit) break;
    }
    return false;
}

struct Cta {
    const CacheAttention& a;
    const Plan& plan;
    uint8_t* sm;
    Barriers* bar;
    Rows* rows;
    uint32_t tmem;
};

// ------------------------------------------------------------------ loaders
struct Loader {
    Cta c;
    int next = 0;                          // half tiles begun
    bool dead = false;

    __device__ __forceinline__ void piece(int pair, int hk, const Tile& tile, int from, int to) {
        const CacheAttention& a = c.a;
        const int tid = threadIdx.x - kSoftmax, lane = tid & 31;
        const int r = tid >> 3, chunk = tid & 7;           // row 0 .. 7 of a step (and 8 on), 16-byte piece of it
        const int32_t* table = a.table + (int64_t)(pair / c.plan.row_tiles) * a.table_pages;
        const int page_mask = (1 << a.page_shift) - 1;
        const bool in_row = chunk * 16 < a.d;
        const int lane_off = r * a.d + chunk * 16, eight_rows = in_row ? 8 * a.d : 0;
        const uint32_t lane_to = r * 128 + ((chunk ^ r) << 4);
        // Lane k < 8: where step k of the tile at step s0 is in the pool, and how many of its tokens exist.
        auto page_of = [&](int s0) -> int {
            const int s = s0 + lane, t = tile.token(s);
            return lane < kTileSteps && s < to && t < tile.end ? table[t >> a.page_shift] : -1;
        };
        int id = page_of(from);
        for (int s0 = from; s0 < to && !dead; s0 += kTileSteps) {
            const int id_next = page_of(s0 + kTileSteps);
            const int t0 = tile.token(s0 + lane);
            const bool held = id >= 0 && id < a.n_pages;
            const int64_t block = (int64_t)id * a.H_kv + hk;
            const int64_t off = held ? ((block << a.page_shift) + (t0 & page_mask)) * a.d : 0;
            const int n = held ? (tile.end - t0 < kStep ? tile.end - t0 : kStep) : 0;
            const bool whole = __all_sync(0xffffffffu, n == kStep || lane >= kTileSteps);
            int64_t offs[kTileSteps];
#pragma unroll
            for (int k = 0; k < kTileSteps; ++k) offs[k] = __shfl_sync(0xffffffffu, off, k) + lane_off;
#pragma unroll 1
            for (int kv = 0; kv < 2; ++kv) {
                const int slot = next % kSlots;
                if (next >= kSlots && !__all_sync(0xffffffffu, wait_up_to(&c.bar->empty[slot], (next / kSlots - 1) & 1,
                                                                         c.plan.stall.wait_us))) {
                    dead = true;
                    break;
                }
                const uint8_t* codes = kv ? a.v_codes : a.k_codes;
                const uint32_t to_s = smem_u32(c.sm + kRingAt + slot * kHalf) + lane_to;
                if (whole) {
#pragma unroll
                    for (int k = 0; k < kTileSteps; ++k) {
                        const uint8_t* src = in_row ? codes + offs[k] : codes;
                        copy_async(to_s + k * kStep * 128, src, in_row);
                        copy_async(to_s + (k * kStep + 8) * 128, src + eight_rows, in_row);
                    }
                } else {
#pragma unroll
                    for (int k = 0; k < kTileSteps; ++k) {
                        const int n_all = __shfl_sync(0xffffffffu, n, k), n_k = in_row ? n_all : 0;
                        copy_async(to_s + k * kStep * 128, r < n_k ? codes + offs[k] : codes, r < n_k);
                        copy_async(to_s + (k * kStep + 8) * 128, r + 8 < n_k ? codes + offs[k] + eight_rows : codes,
                                   r + 8 < n_k);
                    }
                }
                if (tid < kTileSteps) {
                    const uint32_t scale_s =
                        smem_u32(c.sm + kScalesAt) + (((next / 2) & 3) * 2 + kv) * kTileSteps * 4 + tid * 4;
                    copy_async4(scale_s, held ? (kv ? a.v_scale : a.k_scale) + block : a.k_scale, held);
                }
                // An arrival of this thread once all of that has landed; nobody waits here, and the slots to
                // come are begun as they get free.
                asm volatile("cp.async.mbarrier.arrive.noinc.shared::cta.b64 [%0];" ::"r"(smem_u32(&c.bar->full[slot]))
                             : "memory");
                ++next;
            }
            id = id_next;
        }
    }

    __device__ __forceinline__ void finish() { tc::cp_async_wait_all(); }
};

// ------------------------------------------------------------------ issuer
struct Issuer {
    Cta c;
    int tile_n = 0;                        // tiles begun, over all pieces
    int piece_n = 0;
    bool dead = false;

    __device__ __forceinline__ void wait(uint64_t* b, uint32_t parity) {
        if (!dead && !wait_up_to(b, parity, c.plan.stall.wait_us)) dead = true;
    }
    // S[n & 1] = K (q1 + q2 + q3)^T of tile n.
    __device__ __forceinline__ void scores(int n) {
        const int j = 2 * n, slot = j % kSlots;
        if (n >= c.plan.stall.tiles) dead = true;
        wait(&c.bar->full[slot], (j / kSlots) & 1);
        if (n >= 2) wait(&c.bar->s_free[n & 1], ((n >> 1) - 1) & 1);
        if (dead) return;
        tc::fence_async_smem();                            // the copies are generic writes
        tc::tc_fence_after();
        const uint64_t k = tc::desc_sw128(smem_u32(c.sm + kRingAt + slot * kHalf));
        const uint64_t q = tc::desc_sw128(smem_u32(c.sm + kQueriesAt));
#pragma unroll
        for (int x = 0; x < 12; ++x)                       // 32 channels a product; a piece is 32 rows of 128 bytes
            mma_f8(c.tmem + kRows * (n & 1), k + 2 * (x & 3), q + 2 * (x & 3) + (x >> 2) * (kRows * 128 >> 4),
                   idesc_f8(128, kRows, 1, false, false), x > 0);
        tc::mma_commit(&c.bar->empty[slot]);
        tc::mma_commit(&c.bar->s_full[n & 1]);
    }
    // O^T (+)= V^T (w1 | w2 | w3 | w4) of tile n.
    __device__ __forceinline__ void values(int n, bool first) {
        const int j = 2 * n + 1, slot = j % kSlots;
        wait(&c.bar->full[slot], (j / kSlots) & 1);
        wait(&c.bar->w_full, n & 1);
        if (dead) return;
        tc::fence_async_smem();
        tc::tc_fence_after();
        const uint32_t v = smem_u32(c.sm + kRingAt + slot * kHalf), w = smem_u32(c.sm + kWeightsAt);
#pragma unroll
        for (int x = 0; x < 4; ++x)                        // 32 tokens a product
            mma_f8(c.tmem + kTmemO, tc::desc_sw128_mn(v + x * 4096, kHalf, 1024),
                   tc::desc_sw128_mn(w + x * 4096, kHalf, 1024), idesc_f8(128, 128, 1, true, true), !first || x > 0);
        tc::mma_commit(&c.bar->empty[slot]);
        tc::mma_commit(&c.bar->pv_done);
    }
    __device__ __forceinline__ void piece(int from, int to) {
        const int n = (to - from + kTileSteps - 1) / kTileSteps;
        wait(&c.bar->q_full, piece_n & 1);
        ++piece_n;
        if (!dead) scores(tile_n);
        for (int i = 0; i < n && !dead; ++i) {
            if (i + 1 < n) scores(tile_n + i + 1);
            values(tile_n + i, i == 0);
        }
        tile_n += n;
    }
    // Every product issued has ended, whether or not a wait gave up before, so that TMEM may go.
    __device__ __forceinline__ void finish() {
        tc::mma_commit(&c.bar->drained);
        tc::mbar_wait(&c.bar->drained, 0);
    }
};

// ------------------------------------------------------------------ softmax
struct Softmax {
    Cta c;
    int tile_n = 0;
    bool bad = false;                      // a wait of this warp gave up: it waits no more, its numbers are none
    bool dead = false;                     // some thread's did, as found at the piece's end: the same in all

    __device__ __forceinline__ void wait(uint64_t* b, uint32_t parity) {
        if (!bad && !dead && !__all_sync(0xffffffffu, wait_up_to(b, parity, c.plan.stall.wait_us))) bad = true;
    }

    // The item's queries: eight threads a row, 16 channels each.
    __device__ __forceinline__ void load_queries(int b, int hk, int rt) {
        const CacheAttention& a = c.a;
        const int row = threadIdx.x >> 3, part = threadIdx.x & 7;
        const int at = rt * kRows + row;
        const bool real = at < c.plan.rows;
        const int i = real ? at / c.plan.group : 0;
        const __nv_bfloat16* q = static_cast<const __nv_bfloat16*>(a.q) + ((int64_t)b * a.T_q + i) * a.q_stride +
                                 (int64_t)(hk * c.plan.group + (real ? at - i * c.plan.group : 0)) * a.d + 16 * part;
        uint4 raw[2];
#pragma unroll
        for (int x = 0; x < 2; ++x)
            raw[x] = real && 16 * part < a.d ? reinterpret_cast<const uint4*>(q)[x] : make_uint4(0, 0, 0, 0);
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
        for (int w = 1; w < 8; w <<= 1) amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, w));
        number = (__ballot_sync(0xffffffffu, !number) >> (threadIdx.x & 24) & 255u) == 0;
        // 2^ex <= amax < 2^(ex + 1): times 2^(14 - ex), under e5m2's largest value.  A row with an infinity: its scores are
        // infinite or no numbers whatever its finite channels hold, so these count as zeros, under no scale.  A row with a
        // NaN has it from its factor.
        const bool infinite = amax == INFINITY;
        int ex = infinite ? 14 : (int)(__float_as_uint(amax) >> 23) - 127;
        ex = ex < -112 ? -112 : ex;
        const float up = __uint_as_float((uint32_t)(127 + 14 - ex) << 23);
        float rest[16];
#pragma unroll
        for (int x = 0; x < 16; ++x) rest[x] = number ? to_f32(e[x]) * up : 0.0f;
#pragma unroll
        for (int k = 0; k < 3; ++k) {
            uint32_t word[4];
#pragma unroll
            for (int w = 0; w < 4; ++w) {
                word[w] = to_e5m2x4(rest[4 * w], rest[4 * w + 1], rest[4 * w + 2], rest[4 * w + 3]);
                float f[4];
                from_e5m2x4(word[w], f);
#pragma unroll
                for (int x = 0; x < 4; ++x) rest[4 * w + x] -= f[x];
                if (infinite) {                            // its infinities alone: 7c
                    uint32_t codes = 0;
#pragma unroll
                    for (int x = 0; x < 4; ++x) {
                        const uint32_t bits = k == 0 ? __float_as_uint(to_f32(e[4 * w + x])) : 0;
                        if (number && (bits & 0x7fffffffu) == 0x7f800000u) codes |= (bits >> 24 & 0x80u | 0x7cu) << (8 * x);
                    }
                    word[w] = codes;
                }
            }
            *reinterpret_cast<uint4*>(c.sm + kQueriesAt + tc::sw128(k * kRows + row, part)) =
                make_uint4(word[0], word[1], word[2], word[3]);
        }
        if (part == 0) {
            c.rows->factor[row] = number ? a.scale * 1.4426950408889634f * __uint_as_float((uint32_t)(127 + ex - 14) << 23)
                                          : NAN;
            c.rows->m[row] = 0.0f;                         // until the first tile's scores
        }
        if (part < 4) c.rows->nan[row][part] = 0;
    }

    // Which of rows r0 .. r0 + n - 1 see a token, a bit each.
    __device__ __forceinline__ uint32_t sight_of(const Tile& tile, int rt, int at, int r0, int n) {
        const CacheAttention& a = c.a;
        uint32_t sight = 0;
        for (int r = 0; r < n; ++r) {
            const int p = tile.p0 - rt * kRows / c.plan.group + (rt * kRows + r0 + r) / c.plan.group;
            if (at <= p && (a.window == 0 || at > p - a.window || at < a.sinks)) sight |= 1u << r;
        }
        return sight;
    }

    // A token that some rows see and others do not must bring no NaN to the others: its NaN codes become
    // zeros, and the rows that do see it are marked, a channel a bit.  (A token that no row sees
    // is either zeros already or treated the same, without marks.)
    __device__ __noinline__ void mend_values(uint8_t* v, int t, uint32_t sight) {
        for (int chunk = 0; chunk < 8; ++chunk) {
            uint4* at = reinterpret_cast<uint4*>(v + tc::sw128(t, chunk));
            uint4 x = *at;
            uint32_t* word = reinterpret_cast<uint32_t*>(&x);
            uint32_t found = 0;                            // a bit for each of the 16 channels
            for (int w = 0; w < 4; ++w) {
                const uint32_t n = nan_bytes(word[w]);
                word[w] &= ~n;
                found |= ((n & 1u) | (n >> 7 & 2u) | (n >> 14 & 4u) | (n >> 21 & 8u)) << (4 * w);
            }
            if (found == 0) continue;
            *at = x;
            for (uint32_t left = sight; left; left &= left - 1)
                atomicOr(&c.rows->nan[__ffs(left) - 1][chunk >> 1], found << (16 * (chunk & 1)));
        }
    }

    // The references move to the largest of this tile's scores (the first tile: there are none before).
    // s: scores less m, -inf where unseen, and so again afterwards; this thread's rows start at r0.
    __device__ __forceinline__ void move_references(float (&s)[kMine], float e, float (&l)[kMine], int r0, int i) {
        const bool first = i == 0;
        const int lane = threadIdx.x & 31, quarter = threadIdx.x >> 5 & 3;
        Rows* rows = c.rows;
        auto most = [](float x, float y) { return fmaxf(x, y); };
        rows->part[quarter][r0 + (lane >> 1)] = reduce_rows(s, most);
        float se[kMine];
#pragma unroll
        for (int r = 0; r < kMine; ++r) se[r] = s[r] + e;
        rows->part_e[quarter][r0 + (lane >> 1)] = reduce_rows(se, most);
        const int half = r0 / kMine, row = r0 + (lane & 15);
        const float m = rows->m[row], dm = first ? 0.0f : rows->dm[row];     // read by all before any writes
        const uint32_t unset_rows = first ? 0xffffu : rows->unset[half];
        tc::named_bar_sync(kBarHalf + half, kSoftmax / 2);
        // Every warp works out its 16 rows, a lane a row, and writes the same: no warp waits for another's.
        float top = rows->part[0][row], top_e = rows->part_e[0][row];
#pragma unroll
        for (int w = 1; w < 4; ++w) {
            top = fmaxf(top, rows->part[w][row]);
            top_e = fmaxf(top_e, rows->part_e[w][row]);
        }
        // relative to the old m: the new one is m + up, above it unless no score has set it yet
        const bool unset = unset_rows >> (lane & 15) & 1, seen = top != -INFINITY;
        const float up = unset ? (seen ? top : 0.0f) : fmaxf(top, 0.0f);
        const float dm_new = unset ? (seen ? up - top_e : 0.0f) : up - fmaxf(-dm, top_e);
        rows->m[row] = m + up;
        rows->dm[row] = dm_new;
        rows->up[row] = up;
        rows->lift[row] = ex2(dm_new + kBits);
        rows->keep_l[row] = unset ? 1.0f : ex2(-up);
        rows->keep_o[row] = unset ? 1.0f : ex2(dm_new - dm - up);
        const uint32_t still = __ballot_sync(0xffffffffu, unset && !seen) & 0xffffu;
        float most_dm = dm_new;
#pragma unroll
        for (int w = 8; w > 0; w >>= 1) most_dm = fmaxf(most_dm, __shfl_xor_sync(0xffffffffu, most_dm, w));
        if (lane == 0) {
            rows->dm_most[half] = most_dm;
            rows->unset[half] = still;
        }
        __syncwarp();
#pragma unroll
        for (int r = 0; r < kMine; ++r) s[r] -= rows->up[r0 + r];
        if (first) return;                                 // nothing summed yet
#pragma unroll
        for (int r = 0; r < kMine; ++r) l[r] *= rows->keep_l[r0 + r];
        wait(&c.bar->pv_done, (tile_n - 1) & 1);           // the sums rest until this tile's weights are told
        tc::tc_fence_after();
        if (bad) return;
        const uint32_t at = c.tmem + r0 + ((uint32_t)(32 * quarter) << 16);
        const int parts = i > kRun ? 5 : 4;                // (the run that ends at this tile is not in the sums yet)
#pragma unroll 1
        for (int k = 0; k < parts; ++k) {
            const uint32_t part = at + (k < 4 ? kTmemO + kRows * k : kTmemSums);
            float v[16];
            uint32_t out[16];
            tc::tmem_ld16(part, v);
            loaded(v);
#pragma unroll
            for (int r = 0; r < 16; ++r) out[r] = __float_as_uint(v[r] * rows->keep_o[r0 + r]);
            tc::tmem_st16(part, out);
        }
        tc::tmem_wait_st();
        tc::tc_fence_before();
    }

    // This thread's channel of its rows, from the four pieces' sums and the rounded ones.  (Unrolled, it costs the loop over
    // the tiles registers: 5% of 4 x 65,536 tokens under 32 rows.)
    static __device__ __forceinline__ void read_sums(uint32_t at, bool summed, float (&o)[kMine]) {
        tc::tmem_ld16(at + kTmemO, o);
        loaded(o);
#pragma unroll 1
        for (int k = 1; k < 4; ++k) {
            float x[kMine];
            tc::tmem_ld16(at + kTmemO + kRows * k, x);
            loaded(x);
            const float part = k == 1 ? 0.25f : k == 2 ? 0.0625f : 0.015625f;
#pragma unroll
            for (int r = 0; r < kMine; ++r) o[r] = fmaf(x[r], part, o[r]);
        }
        if (summed) {
            float x[kMine];
            tc::tmem_ld16(at + kTmemSums, x);
            loaded(x);
#pragma unroll
            for (int r = 0; r < kMine; ++r) o[r] += x[r];
        }
    }

    // What O holds, all its products ended, goes to the rounded sums, and O begins again from zeros.  (Inline, 1% slower.)
    static __device__ __noinline__ void add_run(uint32_t at, bool summed) {
        float o[kMine];
        read_sums(at, summed, o);
        uint32_t out[kMine];
#pragma unroll
        for (int r = 0; r < kMine; ++r) out[r] = __float_as_uint(o[r]);
        tc::tmem_st16(at + kTmemSums, out);
#pragma unroll
        for (int r = 0; r < kMine; ++r) out[r] = 0;
#pragma unroll
        for (int k = 0; k < 4; ++k) tc::tmem_st16(at + kTmemO + kRows * k, out);
        tc::tmem_wait_st();
        tc::tc_fence_before();
    }

    __device__ __forceinline__ void piece(int pair, int hk, const Tile& tile, int from, int to, int slot, bool whole) {
        const CacheAttention& a = c.a;
        const Plan& plan = c.plan;
        Rows* rows = c.rows;
        const int lane = threadIdx.x & 31, quarter = threadIdx.x >> 5 & 3;
        const int t = 32 * quarter + lane;                 // token of the tile, then channel
        const int half = threadIdx.x >> 7, r0 = kMine * half;
        const int b = pair / plan.row_tiles, rt = pair % plan.row_tiles;
        const uint32_t lanes = (uint32_t)(32 * quarter) << 16;
        // The products of the piece before have read its queries; all threads have left its rows.
        tc::named_bar_sync(kBarSoftmax, kSoftmax);
        load_queries(b, hk, rt);
        tc::fence_async_smem();
        tc::mbar_arrive(&c.bar->q_full);
        tc::named_bar_sync(kBarSoftmax, kSoftmax);

        float l[kMine];
#pragma unroll
        for (int r = 0; r < kMine; ++r) l[r] = 0.0f;
        const int n_tiles = (to - from + kTileSteps - 1) / kTileSteps;
#pragma unroll 1
        for (int i = 0; i < n_tiles; ++i, ++tile_n) {
            if (dead) continue;
            const int n = tile_n, v_slot = (2 * n + 1) % kSlots;
            wait(&c.bar->full[v_slot], ((2 * n + 1) / kSlots) & 1);
            const float* scales = reinterpret_cast<const float*>(c.sm + kScalesAt) + (n & 3) * 2 * kTileSteps;
            const int step = from + i * kTileSteps + (t >> 4);
            const float ks = scales[t >> 4], vs = scales[kTileSteps + (t >> 4)];
            const int at = tile.token(step) + (t & 15);
            const bool valid = step < to && at < tile.end && vs != 0.0f;
            const bool by_all = valid && at <= tile.p0 &&
                                (a.window == 0 || at > tile.p1 - a.window || at < a.sinks);
            wait(&c.bar->s_full[n & 1], (n >> 1) & 1);
            tc::tc_fence_after();

            float s[kMine];                                // scores less m, in powers of two
            tc::tmem_ld16(c.tmem + lanes + kRows * (n & 1) + r0, s);
            loaded(s);
#pragma unroll
            for (int r = 0; r < kMine; ++r) s[r] = fmaf(s[r], rows->factor[r0 + r] * ks, -rows->m[r0 + r]);
            tc::tc_fence_before();
            tc::mbar_arrive(&c.bar->s_free[n & 1]);

            if (!by_all) {
                const uint32_t sight = valid ? sight_of(tile, rt, at, r0, kMine) : 0;
#pragma unroll
                for (int r = 0; r < kMine; ++r)
                    if (!(sight >> r & 1)) s[r] = -INFINITY;
            }
            // log2 of v's scale, rounded up
            const uint32_t vs_bits = __float_as_uint(vs);
            const float e = (float)((int)(vs_bits >> 23) - 127 + ((vs_bits & 0x7fffffu) ? 1 : 0));
            // beyond m, or beyond the sums' reference by this page's scale (of any row: a move too many does no harm)
            float beyond = s[0];
#pragma unroll
            for (int r = 1; r < kMine; ++r) beyond = fmaxf(beyond, s[r]);
            if (i > 0) {
                beyond += fmaxf(rows->dm_most[half] + e, 0.0f);
                if (const uint32_t unset = rows->unset[half]) {
#pragma unroll
                    for (int r = 0; r < kMine; ++r)
                        if ((unset >> r & 1) && s[r] != -INFINITY) beyond = INFINITY;
                }
            }
            if (vote(beyond > kFar || i == 0, kBarHalf + half, kSoftmax / 2)) move_references(s, e, l, r0, i);
            if (i > 0) wait(&c.bar->pv_done, (n - 1) & 1);   // the weights before have been read
            if (i > 0 && i % kRun == 0 && !bad) {
                tc::tc_fence_after();
                add_run(c.tmem + lanes + r0, i > kRun);
            }

            // Weights: the pieces of 16 rows are 16 bytes each.
            uint32_t piece[4][4];
#pragma unroll
            for (int q = 0; q < 4; ++q) {
                uint32_t two[2];
#pragma unroll
                for (int x = 0; x < 2; ++x) {
                    float w[2];
#pragma unroll
                    for (int y = 0; y < 2; ++y) {
                        const int r = 4 * q + 2 * x + y;
                        const float p = ex2(s[r]);
                        l[r] += p;
                        w[y] = p * rows->lift[r0 + r] * vs;
                    }
                    two[x] = half2_bits(w[0], w[1]);
                }
#pragma unroll
                for (int k = 0; k < 4; ++k) {
                    if (k == 3) {                          // the last one rounded
                        two[0] += 0x00800080u;
                        two[1] += 0x00800080u;
                    }
                    piece[k][q] = __byte_perm(two[0], two[1], 0x7531);
                    if (k < 3) {
#pragma unroll
                        for (int x = 0; x < 2; ++x) two[x] = half2_times4(half2_sub(two[x], two[x] & 0xff00ff00u));
                    }
                }
            }
#pragma unroll
            for (int k = 0; k < 4; ++k)
                *reinterpret_cast<uint4*>(c.sm + kWeightsAt + tc::sw128(t, 2 * k + half)) =
                    make_uint4(piece[k][0], piece[k][1], piece[k][2], piece[k][3]);
            if (!by_all && half == 0)
                mend_values(c.sm + kRingAt + v_slot * kHalf, t, valid ? sight_of(tile, rt, at, 0, kRows) : 0);
            tc::fence_async_smem();
            tc::mbar_arrive(&c.bar->w_full);
        }

        // The end: the last sums, and the weights' sums over the tokens' threads.
        if (!dead) wait(&c.bar->pv_done, (tile_n - 1) & 1);
        tc::tc_fence_after();
        if (!dead && vote(bad, kBarSoftmax, kSoftmax)) dead = true;
        rows->part[quarter][r0 + (lane >> 1)] = reduce_rows(l, [](float x, float y) { return x + y; });
        tc::named_bar_sync(kBarSoftmax, kSoftmax);
        // What a row needs once, not 128 times: the factor that makes its sums outputs (with that worked out in every
        // thread, and the rows' places by divisions, 2,048 items of 4,096 tokens took 735 us instead of 688).
        const int rows_here = rows_of_tile(plan, rt);
        const int64_t place = ((int64_t)blockIdx.x * 2 + slot) * plan.stored;
        if (threadIdx.x < kRows) {
            const int r = threadIdx.x;
            const float L = dead ? NAN : (rows->part[0][r] + rows->part[1][r]) + (rows->part[2][r] + rows->part[3][r]);
            const uint32_t empty = __ballot_sync(0xffffffffu, L == 0.0f);
            if (r % kMine == 0) rows->empty[r / kMine] = empty >> r;
            rows->keep_o[r] = row_factor(rows->dm[r], L);
            if (r < rows_here) {
                if (!whole) plan.stats[place + r] = make_float4(rows->unset[r / kMine] >> r % kMine & 1 ? kLowest : rows->m[r], rows->dm[r], L, 0.0f);
                else if (a.lse) a.lse[output_row(a, plan, b, hk, rt, r)] = row_lse(rows->m[r], L);
            }
        }
        float o[16];
        read_sums(c.tmem + lanes + r0, n_tiles > kRun, o);
#pragma unroll
        for (int y = 0; y < 16; ++y) o[y] *= kToPlan;
        tc::named_bar_sync(kBarSoftmax, kSoftmax);
#pragma unroll
        for (int y = 0; y < 16; ++y)
            if (dead || (rows->nan[r0 + y][quarter] >> lane & 1)) o[y] = NAN;
        if (!whole) {
            float* to = plan.sums + (place + r0) * 128 + t;
#pragma unroll
            for (int y = 0; y < 16; ++y)
                if (r0 + y < rows_here) to[y * 128] = o[y];
        } else if (t < a.d) {
            const uint32_t empty = rows->empty[half];
            // row r's place in a query token's heads: after the last one, the next token's first
            int in_token = (rt * kRows + r0) % plan.group;
            __nv_bfloat16* to = static_cast<__nv_bfloat16*>(a.o) + output_row(a, plan, b, hk, rt, r0) * a.d + t;
#pragma unroll
            for (int y = 0; y < 16; ++y) {
                if (r0 + y < rows_here) *to = __float2bfloat16_rn(empty >> y & 1 ? 0.0f : o[y] * rows->keep_o[r0 + y]);
                to += a.d;
                if (++in_token == plan.group) {
                    in_token = 0;
                    to += (int64_t)(a.H_q - plan.group) * a.d;
                }
            }
        }
        tc::tc_fence_before();                             // the next piece's products may overwrite the sums
    }
};

template <bool WHOLE>
__global__ void __launch_bounds__(kThreads, kCtas) attention_tc_kernel(const CacheAttention a, const Plan plan) {
    extern __shared__ uint8_t smem_raw[];
    uint8_t* sm = smem_raw + ((1024u - (smem_u32(smem_raw) & 1023u)) & 1023u);
    Barriers* bar = reinterpret_cast<Barriers*>(sm + kBarriersAt);
    const int warp = threadIdx.x >> 5;
    after_the_kernel_before();
    if (threadIdx.x == 0) {
        for (int i = 0; i < kSlots; ++i) {
            tc::mbar_init(&bar->full[i], kLoaders);
            tc::mbar_init(&bar->empty[i], 1);
        }
        for (int i = 0; i < 2; ++i) {
            tc::mbar_init(&bar->s_full[i], 1);
            tc::mbar_init(&bar->s_free[i], kSoftmax);
        }
        tc::mbar_init(&bar->w_full, kSoftmax);
        tc::mbar_init(&bar->pv_done, 1);
        tc::mbar_init(&bar->q_full, kSoftmax);
        tc::mbar_init(&bar->drained, 1);
        tc::fence_mbar_init();
    }
    if (warp == kIssuerWarp) tc::tmem_alloc<kTmemCols>(&bar->tmem);
    tc::tc_fence_before();
    __syncthreads();
    tc::tc_fence_after();
    Share share = {};
    if (!WHOLE) share = find_share<kThreads>(a, plan);
    const Cta cta{a, plan, sm, bar, reinterpret_cast<Rows*>(sm + kRowsAt), bar->tmem};
    auto pieces = [&](auto f) {
        if constexpr (WHOLE) {
            const int pair = blockIdx.x / a.H_kv;
            const Tile tile = tile_of(a, plan, pair);
            f(pair, (int)(blockIdx.x % a.H_kv), tile, 0, tile.steps, 0, true);
        } else {
            const int4 join = for_each_piece(a, plan, share, f);
            if (threadIdx.x == 0) plan.joins[blockIdx.x] = join;
        }
    };
    if (warp < kSoftmax / 32) {
        asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(kSoftmaxRegs));
        Softmax role{cta};
        pieces([&](int pair, int hk, const Tile& tile, int from, int to, int slot, bool whole) {
            role.piece(pair, hk, tile, from, to, slot, whole);
        });
    } else {
        asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kOtherRegs));
        if (warp < kIssuerWarp) {
            Loader role{cta};
            pieces([&](int pair, int hk, const Tile& tile, int from, int to, int, bool) {
                if (role.dead) return;
                const int left = plan.stall.loads - role.next / 2, most = from + (left < 1 << 24 ? left : 1 << 24) * kTileSteps;
                role.piece(pair, hk, tile, from, to < most ? to : most);
                if (most < to) role.dead = true;
            });
            role.finish();
        } else if (threadIdx.x == 32 * kIssuerWarp) {
            Issuer role{cta};
            pieces([&](int, int, const Tile&, int from, int to, int, bool) {
                if (!role.dead) role.piece(from, to);
            });
            role.finish();
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

}  // namespace

// bf16 queries with heads of more than 64 channels and more rows a head than two tiles of 8: below, the products
// of kda_cache_attention.cu keep up with the memory.
bool attention_tc_takes(const CacheAttention& a, bool bf16) {
    return bf16 && a.d > 64 && (int64_t)a.T_q * (a.H_q / a.H_kv) > 16;
}

attn::Plan attention_tc_plan(const CacheAttention& a) {
    Plan plan = {};
    plan.group = a.H_q / a.H_kv;
    plan.rows = a.T_q * plan.group;
    plan.tile_rows = kRows;
    plan.row_tiles = (plan.rows + kRows - 1) / kRows;
    plan.stored = plan.rows < kRows ? plan.rows : kRows;
    plan.item_cost = 8 * kTileSteps;
    plan.cut = kTileSteps;
    return plan;
}

// A tile of 8 steps is the least that is cut, and a CTA's second start and end cost the time of a dozen.  Measured both ways:
// 16 tiles (2,048 tokens), 32 items 32 us whole and 23 cut, 128 items 32 and 37, 512 items 86 and 101, 2,048 items 294 and 343;
// 32 tiles, 256 items 76 and 86 us, lengths that differ 72 and 66.  Very few items are cut from 5 tiles on (8 items of 8
// tiles: 21 us whole, 17 cut).
int64_t attention_tc_grid(const CacheAttention& a, const attn::Plan& plan, int num_sms) {
    const int64_t cap = most_steps(a), items = (int64_t)a.B * plan.row_tiles * a.H_kv, most = (int64_t)num_sms * kCtas;
    const bool few = 10 * items < most;
    if (whole_items_pay(cap, items, most, 13 * kTileSteps, (few ? 4 : 32) * kTileSteps) ||
        (int64_t)a.B * plan.row_tiles > kMaxScan)
        return 0;
    const int64_t useful = (items * (cap + plan.item_cost) + kMinShare - 1) / kMinShare;
    return useful < most ? useful : most;
}

namespace {
thread_local Stall stall;
}

cudaError_t run_attention_tc(const CacheAttention& a, void* workspace, cudaStream_t stream, int num_sms) {
    Plan plan = attention_tc_plan(a);
    plan.stall = stall;
    const int64_t grid = attention_tc_grid(a, plan, num_sms);
    if (grid == 0) {
        const int64_t items = (int64_t)a.B * plan.row_tiles * a.H_kv;
        cudaError_t e = cudaFuncSetAttribute(attention_tc_kernel<true>, cudaFuncAttributeMaxDynamicSharedMemorySize, kSmem);
        if (e != cudaSuccess) return e;
        return launch_chained(attention_tc_kernel<true>, (unsigned)items, kThreads, kSmem, stream, a, plan);
    }
    set_attention_pieces(plan, workspace, grid);
    cudaError_t e = cudaFuncSetAttribute(attention_tc_kernel<false>, cudaFuncAttributeMaxDynamicSharedMemorySize, kSmem);
    if (e != cudaSuccess) return e;
    e = launch_chained(attention_tc_kernel<false>, (unsigned)grid, kThreads, kSmem, stream, a, plan);
    return e != cudaSuccess ? e : run_attention_join(a, plan, true, 128, grid, stream);
}

}  // namespace kda

extern "C" kda_status kda_selftest_attention_stall(int loads, int tiles, int wait_us) {
    if (wait_us == 0) {
        kda::stall = kda::attn::Stall{};
        return kda::report(KDA_OK, "%s", "");
    }
    if (loads < 0 || tiles < 0 || wait_us < 0 || wait_us > 2000000)
        return kda::report(KDA_ERR_INVALID_ARG, "bad arguments loads=%d tiles=%d wait_us=%d", loads, tiles, wait_us);
    kda::stall = kda::attn::Stall{loads, tiles, wait_us};
    return kda::report(KDA_OK, "%s", "");
}
