// kda_cache_attention_rest.cu -- attention over what follows a shared prefix in each sequence, few rows a head
// (kda_cache_attention_rows.cuh).
#include "kda_cache_attention_rows.cuh"

namespace kda {

cudaError_t run_attention_join_rest(const CacheAttention& a, const attn::Plan& plan, bool bf16, int D, int64_t grid,
                                    cudaStream_t stream) {
    return run_join<kRest>(a, plan, bf16, D, grid, stream);
}
size_t attention_rest_rows_workspace_bytes(const CacheAttention& a, int num_sms) {
    return rows_workspace_bytes<kRest>(a, num_sms);
}
cudaError_t run_attention_rest_rows(const CacheAttention& a, bool bf16, void* workspace, cudaStream_t stream, int num_sms) {
    return run_rows<kRest>(a, bf16, workspace, stream, num_sms);
}

}  // namespace kda
