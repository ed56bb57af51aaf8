// kda_cache_attention_prefix.cu -- attention of a group's rows over the prefix that its sequences share, few rows a
// head or fp32 (kda_cache_attention_rows.cuh).
#include "kda_cache_attention_rows.cuh"

namespace kda {

size_t attention_prefix_rows_workspace_bytes(const CacheAttention& a, int num_sms) {
    return rows_workspace_bytes<kPrefix>(a, num_sms);
}
cudaError_t run_attention_prefix_rows(const CacheAttention& a, bool bf16, void* workspace, cudaStream_t stream, int num_sms) {
    return run_rows<kPrefix>(a, bf16, workspace, stream, num_sms);
}

}  // namespace kda
