// Attention of many query rows over whole contexts (bf16 inputs): kv_attn_prompt.cuh.
#include "kv_attn_prompt.cuh"

cudaError_t gdn_launch_kv_attn_prompt(const gdn::KvAttn &a, int d, int n_units, cudaStream_t st) {
    if (d == 64) return gdn::launch_prompt<64>(a, n_units, st);
    if (d == 128) return gdn::launch_prompt<128>(a, n_units, st);
    return gdn::launch_prompt<256>(a, n_units, st);
}
