// ggq_k_rows_128.cu -- instances of the fp32 prompt attention kernel for heads of 128 channels.
#include "ggq_attn_rows.cuh"

namespace ggq {

cudaError_t launch_attn_rows_128(const AttnParams& p, cudaStream_t s) { return launch_attn_rows_dim<128>(p, s); }

}  // namespace ggq
