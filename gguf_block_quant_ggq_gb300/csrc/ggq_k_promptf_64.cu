// ggq_k_promptf_64.cu -- instances of the fp32 prompt attention kernel for heads of 64 channels.
#include "ggq_attn_promptf.cuh"

namespace ggq {

cudaError_t launch_attn_promptf_64(const AttnParams& p, cudaStream_t s) { return launch_attn_promptf_dim<64>(p, s); }

}  // namespace ggq
