// ggq_k_prompt_64.cu -- instances of the prompt attention kernel for heads of 64 channels.
#include "ggq_attn_prompt.cuh"

namespace ggq {

cudaError_t launch_attn_prompt_64(const AttnParams& p, cudaStream_t s) { return launch_attn_prompt_dim<64>(p, s); }

}  // namespace ggq
