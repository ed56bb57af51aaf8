// kda_cache_internal.h -- launch functions of the global-attention operators.  Apart from kda_internal.h, which the
// recurrent layer's kernels are built from, so that their recorded counters (profiles/traffic.json) stay theirs.
#pragma once

#include "kda_internal.h"

namespace kda {

// Rotary positions on q and k (k: H_k == 0 for none); strides in elements between tokens.
cudaError_t run_rotary(const void* q, int64_t q_stride, void* q_out, int64_t q_out_stride, int H_q,
                       const void* k, int64_t k_stride, void* k_out, int64_t k_out_stride, int H_k,
                       const int32_t* positions, const double* freq, float amplitude,
                       int64_t n_tokens, int d, int rot, bool half_layout, bool bf16,
                       cudaStream_t stream, int num_sms);

// The tokens that a cache write brings or a cache read asks for: n_seqs runs of
// T tokens each, or of lengths that only the device knows, `rows` in all.
struct CacheSpan {
    int64_t rows;
    int64_t T;              // fixed length; 0 if packed
    int64_t slots_per_seq;  // pages that a run of T tokens can touch
    int64_t n_pages;
    int64_t table_pages;    // columns of the block table
    int n_seqs;
    int H;
    int d;
    int page_shift;
};
// (page, sequence) slots that the write and read kernels deal out.
int64_t cache_slots(const CacheSpan& w, bool packed);
cudaError_t run_cache_write(const CacheSpan& w, const void* k, int64_t k_stride, const void* v,
                            int64_t v_stride, void* k_codes, void* v_codes, float* k_scale,
                            float* v_scale, const int32_t* table, const int32_t* start,
                            const int32_t* cu, bool bf16, cudaStream_t stream);
cudaError_t run_cache_read(const CacheSpan& w, const void* k_codes, const void* v_codes,
                           const float* k_scale, const float* v_scale, const int32_t* table,
                           const int32_t* start, const int32_t* cu, void* k, void* v, bool bf16,
                           cudaStream_t stream);

// Attention over the paged cache.
struct CacheAttention {
    const void* q;
    const uint8_t* k_codes;
    const uint8_t* v_codes;
    const float* k_scale;
    const float* v_scale;
    const int32_t* table;      // [B][table_pages]
    const int32_t* lengths;    // [B]
    void* o;                   // [B][T_q][H_q][d]
    float* lse;                // [B][T_q][H_q], or null
    int64_t q_stride;          // elements between tokens
    int64_t n_pages;
    int64_t window;            // 0: none
    int table_pages;
    int B, T_q, H_q, H_kv, d;
    int page_shift;
    int sinks;
    float scale;               // of the scores
};
size_t cache_attention_workspace_bytes(const CacheAttention& a, int num_sms);
cudaError_t run_cache_attention(const CacheAttention& a, bool bf16, void* workspace,
                                cudaStream_t stream, int num_sms);

}  // namespace kda
