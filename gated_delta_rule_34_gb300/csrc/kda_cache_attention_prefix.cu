// kda_cache_attention_prefix.cu -- attention of a group's fp32 rows over the prefix that its sequences share, by the kernels
// for few rows (kda_cache_attention_rows.cuh); bf16 rows are kda_cache_prefix_tc.cu's.
#include "kda_cache_attention_rows.cuh"

namespace kda {

size_t attention_prefix_rows_workspace_bytes(const CacheAttention& a, int num_sms) {
    return rows_workspace_bytes<kPrefix>(a, num_sms);
}
cudaError_t run_attention_prefix_rows(const CacheAttention& a, void* workspace, cudaStream_t stream, int num_sms) {
    return run_rows<kPrefix>(a, false, workspace, stream, num_sms);
}

}  // namespace kda
