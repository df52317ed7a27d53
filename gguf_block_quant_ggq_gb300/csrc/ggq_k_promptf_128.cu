// ggq_k_promptf_128.cu -- instances of the fp32 prompt attention kernel for heads of 128 channels.
#include "ggq_attn_promptf.cuh"

namespace ggq {

cudaError_t launch_attn_promptf_128(const AttnParams& p, cudaStream_t s) { return launch_attn_promptf_dim<128>(p, s); }

}  // namespace ggq
