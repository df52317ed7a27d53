// ggq_k_rows_64.cu -- instances of the fp32 prompt attention kernel for heads of 64 channels.
#include "ggq_attn_rows.cuh"

namespace ggq {

cudaError_t launch_attn_rows_64(const AttnParams& p, cudaStream_t s) { return launch_attn_rows_dim<64>(p, s); }

}  // namespace ggq
