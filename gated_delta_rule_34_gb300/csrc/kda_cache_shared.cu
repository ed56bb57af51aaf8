// kda_cache_shared.cu -- attention over the paged 8-bit cache for groups of sequences that share a prefix.
//
// softmax over two sets of tokens is that over each, joined: with (m, l, x) a row's largest score, its sum of
// weights 2^(s - m) and its sum of weighted values over one set,
//
//   m = max(m1, m2),   l = l1 2^(m1 - m) + l2 2^(m2 - m),   x = x1 2^(m1 - m) + x2 2^(m2 - m),   o = x / l
//
// so a group's rows, all sequences' and all query tokens', meet its prefix once, as the rows of one product, and each
// sequence the rest of its tokens by itself.  The first leaves (m, l, x) for each row in the workspace, the
// second goes on from them where it writes its outputs.  The lengths are on the device, and so is the choice of what
// is shared: whole pages, where two sequences or more share them, for the sequences all of whose queries see all of them.
#include "kda_attention_common.cuh"

namespace kda {
namespace {

size_t up(size_t n) { return (n + 255) / 256 * 256; }
int padded(const CacheAttention& a) { return a.d <= 64 ? 64 : 128; }
size_t rows_of(const CacheAttention& a) { return (size_t)a.B * a.T_q * a.H_q; }
size_t carry_bytes(const CacheAttention& a) {
    return up(rows_of(a) * sizeof(float4)) + up(rows_of(a) * padded(a) * sizeof(float));
}

// Whether the prefixes are taken by themselves: that is two kernels and their start, and a trip of each row's sums through memory,
// against codes read, and rows of tiles filled up, again by each sequence.  By what the prefix table has room for: bf16 (each 32 rows
// of a sequence read the codes, from L2) from 96 MB of codes and the trip's bytes on; fp32 (bound by its products, of tiles of
// 8 to 64 rows, which sharing fills; eight rows count as the bytes of a tile's codes) from 96 MB and six times the trip on.
// Measured both ways, us, shared and each by itself, with 64 tokens of each sequence's own, 8 heads of 128 unless stated.  bf16:
// 256 sequences of 4 rows, 256 tokens (134 MB) 40 and 39, 1,024 48 and 93; 32 such, 2,048 tokens (130 MB) 30 and 31, 8,192 34 and 84;
// 40 of 260 rows, 128 tokens (92 MB and a trip of 85) 120 and 90, 256 127 and 123, 1,024 159 and 265; 40 of 32 rows, 512 tokens 40
// and 32, 1,024 (82 MB, 10) 42 and 46; 7 groups of two of 2 rows, 4,096 tokens (59 MB) 28 and 27, 16,384 59 and 86.  fp32: 81 of 66
// rows, 13 heads of 80, 256 tokens (528 MB and six trips of 71) 223 and 229, 1,024 449 and 622; 52 of 608 rows, 10 heads, 1,024 tokens
// (535 MB, 324) 1,750 and 1,564; 256 of 4 rows, 512 tokens (200 MB, 8) 69 and 63, 1,024 79 and 103; 8 of 64 rows (0 MB), 8,192 tokens
// 125 and 111.
bool sharing_pays(const CacheAttention& a, bool bf16) {
    if (a.n_groups == 0) return false;
    const int64_t rows = (int64_t)a.T_q * (a.H_q / a.H_kv), tokens = (int64_t)a.prefix_pages << a.page_shift;
    const int64_t tile = rows <= 8 ? 10 : rows <= 16 ? 16 : rows <= 32 ? 32 : (rows + 63) / 64 * 64;   // (10: 8 wait for the codes)
    const double reads = bf16 ? (double)((rows + 31) / 32) : (double)(tile - rows) / 8.0;
    const double saved = reads * (double)(a.B - a.n_groups) * a.H_kv * tokens * 2 * padded(a);
    const double trip = (double)rows_of(a) * 2 * sizeof(float) * padded(a);
    return saved >= (double)(96 << 20) + (bf16 ? 1.0 : 6.0) * trip;
}

// Whether a group's prefix goes to the tensor cores' kernel, whose products have 128 rows: bf16 groups of more than 16 rows of 128
// channels, or 32 of 64, where groups are alike.  Measured both ways, us, that kernel and the one for few rows, prefixes of 65,536
// tokens: 8 heads of 128, 7 groups of 4 rows 335 and 171, of 16 rows 332 and 226, of 32 rows 340 and 430, one group of 32 rows 73 and
// 85; 2 heads of 64, 7 groups of 16 rows 91 and 59, of 32 rows 92 and 72, of 64 rows 92 and 121.
bool prefix_has_many_rows(const CacheAttention& a, bool bf16) {
    const int64_t rows = (int64_t)((a.B + a.n_groups - 1) / a.n_groups) * a.T_q * (a.H_q / a.H_kv);
    return bf16 && rows * padded(a) > 16 * 128;
}

size_t most(size_t x, size_t y) { return x > y ? x : y; }

// The rest of more rows a head than 16: the tensor cores' kernel from 1,024 tokens on that the tables have room for behind a prefix.
// Its start and end take longer than a short rest.  Measured both ways with the prefix of 512 tokens (us, this and the few-row kernel,
// 8 heads of 128 channels): 40 sequences of 32 rows a head 63 and 42 (128 tokens), 82 and 74 (1,024), 129 and 139 (4,096); of
// 256 rows 247 and 141, 335 and 286, 425 and 452 (2,048), 611 and 808 (4,096); 4 of 256 rows 47 and 40, 59 and 65, 107 and 112.
bool rest_is_long(const CacheAttention& a, bool bf16) { return attention_tc_takes(a, bf16) && attn::rest_steps(a) > 1024 / attn::kStep; }

}  // namespace

size_t cache_attention_shared_workspace_bytes(const CacheAttention& a, int num_sms) {
    // (whatever the type of query; and a pool without pages holds nothing to share)
    CacheAttention alone = a;
    alone.prefix_pages = 0;
    const size_t by_itself = most(cache_attention_workspace_bytes(alone, num_sms), attention_rest_rows_workspace_bytes(alone, num_sms));
    if (!sharing_pays(a, true) && !sharing_pays(a, false)) return by_itself;
    // the two passes' pieces follow one another in the same place
    size_t pieces = most(attention_prefix_rows_workspace_bytes(a, num_sms), attention_rest_rows_workspace_bytes(a, num_sms));
    if (prefix_has_many_rows(a, true)) pieces = most(pieces, attention_prefix_tc_workspace_bytes(a, num_sms));
    if (rest_is_long(a, true)) {
        const attn::Plan plan = attention_tc_plan(a);
        pieces = most(pieces, attention_piece_bytes(attention_tc_grid(a, plan, num_sms, attn::kRest), plan.stored, 128));
    }
    return most(carry_bytes(a) + pieces, by_itself);
}

cudaError_t run_cache_attention_shared(CacheAttention a, bool bf16, void* workspace, cudaStream_t stream, int num_sms) {
    if (!sharing_pays(a, bf16) || a.n_pages == 0) {
        // Each sequence by itself: many rows of few tokens as the rest of more, with nothing carried (40 of 260 rows, 96 tokens:
        // 64 us, on the tensor cores' kernel 133; 576 tokens 183 and 198).
        a.prefix_pages = 0;
        if (attention_tc_takes(a, bf16) && !rest_is_long(a, bf16)) return run_attention_rest_rows(a, bf16, workspace, stream, num_sms);
        return run_cache_attention(a, bf16, workspace, stream, num_sms);
    }
    uint8_t* at = static_cast<uint8_t*>(workspace);
    a.carry_stats = reinterpret_cast<float4*>(at);
    a.carry_sums = reinterpret_cast<float*>(at + up(rows_of(a) * sizeof(float4)));
    void* pieces = at + carry_bytes(a);
    cudaError_t e = prefix_has_many_rows(a, bf16) ? run_attention_prefix_tc(a, pieces, stream, num_sms)
                                                  : run_attention_prefix_rows(a, bf16, pieces, stream, num_sms);
    if (e != cudaSuccess) return e;
    if (rest_is_long(a, bf16)) return run_attention_tc_rest(a, pieces, stream, num_sms);
    return run_attention_rest_rows(a, bf16, pieces, stream, num_sms);
}

}  // namespace kda
