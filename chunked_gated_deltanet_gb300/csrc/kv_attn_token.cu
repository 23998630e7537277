// Attention of few query rows over whole contexts (bf16 inputs): kv_attn_token.cuh.
#include "kv_attn_token.cuh"

cudaError_t gdn_launch_kv_attn_token(const gdn::KvAttn &a, int d, int n_units, int rows_max, cudaStream_t st) {
    return gdn::launch_token_part<gdn::kKvWhole>(a, d, n_units, rows_max, st);
}
