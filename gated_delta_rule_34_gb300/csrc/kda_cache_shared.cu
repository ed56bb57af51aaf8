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
// against codes read again by each sequence (each 32 rows of one), which come from L2 and count for padded heads. By what the
// tables have room for, 96 MB of such codes are where the two are even.  Measured both ways with 64 tokens of each sequence's own, us,
// shared and each by itself: 256 sequences of 4 rows, 8 heads of 128, 256 tokens (134 MB) 40 and 39, 1,024 tokens 48 and 93; 32
// such, 1,024 tokens (65 MB) 30 and 21, 2,048 30 and 31, 8,192 34 and 84; 4 such, 8,192 tokens (50 MB) 30 and 21; 40 of 32 rows,
// 1,024 tokens (82 MB) 42 and 46; 2 of 260 rows, 2,048 tokens (38 MB) 40 and 33, 4,096 49 and 57; fp32: 32 of one row, 16 heads
// of 64, 1,024 tokens (65 MB) 23 and 28; 256 of 4 rows, 8 heads of 128, 256 tokens 49 and 43, 1,024 78 and 103.
bool sharing_pays(const CacheAttention& a) {
    const int64_t rows = (int64_t)a.T_q * (a.H_q / a.H_kv), tokens = (int64_t)a.prefix_pages << a.page_shift;
    const double bytes = (double)(a.B - a.n_groups) * a.H_kv * ((rows + 31) / 32) * tokens * 2 * padded(a);
    return a.n_groups > 0 && bytes >= (double)(96 << 20);
}

size_t most(size_t x, size_t y) { return x > y ? x : y; }

// The rest of more rows a head than 16: the tensor cores' kernel from 1,024 tokens on that the tables have room for behind a prefix.
// Its start and end take longer than a short rest.  Measured both ways with the prefix of 512 tokens (us, this and the few-row kernel,
// 8 heads of 128 channels): 40 sequences of 32 rows a head 63 and 42 (128 tokens), 82 and 74 (1,024), 129 and 139 (4,096); of
// 256 rows 247 and 141, 335 and 286, 425 and 452 (2,048), 611 and 808 (4,096); 4 of 256 rows 47 and 40, 59 and 65, 107 and 112.
bool rest_is_long(const CacheAttention& a, bool bf16) { return attention_tc_takes(a, bf16) && attn::rest_steps(a) > 1024 / attn::kStep; }

}  // namespace

size_t cache_attention_shared_workspace_bytes(const CacheAttention& a, int num_sms) {
    if (!sharing_pays(a)) return cache_attention_workspace_bytes(a, num_sms);
    // the two passes' pieces follow one another in the same place
    size_t pieces = most(attention_prefix_rows_workspace_bytes(a, num_sms), attention_prefix_tc_workspace_bytes(a, num_sms));
    pieces = most(pieces, attention_rest_rows_workspace_bytes(a, num_sms));
    if (rest_is_long(a, true)) {
        const attn::Plan plan = attention_tc_plan(a);
        pieces = most(pieces, attention_piece_bytes(attention_tc_grid(a, plan, num_sms, attn::kRest), plan.stored, 128));
    }
    // (a pool without pages holds nothing to share)
    return most(carry_bytes(a) + pieces, cache_attention_workspace_bytes(a, num_sms));
}

cudaError_t run_cache_attention_shared(CacheAttention a, bool bf16, void* workspace, cudaStream_t stream, int num_sms) {
    if (!sharing_pays(a) || a.n_pages == 0) return run_cache_attention(a, bf16, workspace, stream, num_sms);
    uint8_t* at = static_cast<uint8_t*>(workspace);
    a.carry_stats = reinterpret_cast<float4*>(at);
    a.carry_sums = reinterpret_cast<float*>(at + up(rows_of(a) * sizeof(float4)));
    void* pieces = at + carry_bytes(a);
    cudaError_t e = bf16 ? run_attention_prefix_tc(a, pieces, stream, num_sms) : run_attention_prefix_rows(a, pieces, stream, num_sms);
    if (e != cudaSuccess) return e;
    if (rest_is_long(a, bf16)) return run_attention_tc_rest(a, pieces, stream, num_sms);
    return run_attention_rest_rows(a, bf16, pieces, stream, num_sms);
}

}  // namespace kda
