// Attention of many query rows over whole contexts (bf16 inputs): kv_attn_prompt.cuh.
#include "kv_attn_prompt.cuh"

cudaError_t gdn_launch_kv_attn_prompt(const gdn::KvAttn &a, int d, int n_units, cudaStream_t st) {
    return gdn::launch_prompt_part<gdn::kKvWhole>(a, d, n_units, st);
}
