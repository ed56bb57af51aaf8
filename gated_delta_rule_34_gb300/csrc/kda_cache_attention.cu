// kda_cache_attention.cu -- attention over a sequence's whole cache, few rows a head (kda_cache_attention_rows.cuh).
#include "kda_cache_attention_rows.cuh"

namespace kda {

size_t attention_piece_bytes(int64_t grid, int stored, int D) {
    return (size_t)grid * (sizeof(int4) + 2 * (size_t)stored * (sizeof(float4) + D * sizeof(float)));
}

void set_attention_pieces(attn::Plan& plan, void* workspace, int64_t grid) {
    plan.joins = static_cast<int4*>(workspace);
    plan.stats = reinterpret_cast<float4*>(plan.joins + grid);
    plan.sums = reinterpret_cast<float*>(plan.stats + grid * 2 * plan.stored);
}

cudaError_t run_attention_join(const CacheAttention& a, const attn::Plan& plan, bool bf16, int D, int64_t grid,
                               cudaStream_t stream) {
    return run_join<kAll>(a, plan, bf16, D, grid, stream);
}

size_t attention_rows_workspace_bytes(const CacheAttention& a, int num_sms) { return rows_workspace_bytes<kAll>(a, num_sms); }

cudaError_t run_attention_rows(const CacheAttention& a, bool bf16, void* workspace, cudaStream_t stream, int num_sms) {
    return run_rows<kAll>(a, bf16, workspace, stream, num_sms);
}

size_t cache_attention_workspace_bytes(const CacheAttention& a, int num_sms) {
    size_t most = attention_rows_workspace_bytes(a, num_sms);
    if (attention_tc_takes(a, true)) {
        const Plan plan = attention_tc_plan(a);
        const size_t need = attention_piece_bytes(attention_tc_grid(a, plan, num_sms), plan.stored, 128);
        most = need > most ? need : most;
    }
    return most;
}

cudaError_t run_cache_attention(const CacheAttention& a, bool bf16, void* workspace, cudaStream_t stream,
                                int num_sms) {
    if (attention_tc_takes(a, bf16)) return run_attention_tc(a, workspace, stream, num_sms);
    return run_attention_rows(a, bf16, workspace, stream, num_sms);
}

}  // namespace kda
