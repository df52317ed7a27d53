// ggq_k_prompt_128.cu -- instances of the prompt attention kernel for heads of 128 channels.
#include "ggq_attn_prompt.cuh"

namespace ggq {

cudaError_t launch_attn_prompt_128(const AttnParams& p, cudaStream_t s) { return launch_attn_prompt_dim<128>(p, s); }

}  // namespace ggq
