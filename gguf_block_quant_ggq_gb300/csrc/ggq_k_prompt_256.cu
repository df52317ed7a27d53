// ggq_k_prompt_256.cu -- instances of the prompt attention kernel for heads of 256 channels.
#include "ggq_attn_prompt.cuh"

namespace ggq {

cudaError_t launch_attn_prompt_256(const AttnParams& p, cudaStream_t s) { return launch_attn_prompt_dim<256>(p, s); }

}  // namespace ggq
