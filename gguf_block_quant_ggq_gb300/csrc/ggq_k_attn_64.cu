// ggq_k_attn_64.cu -- instances of the streaming attention kernel for heads of 64 channels.
#include "ggq_attn_stream.cuh"

namespace ggq {

cudaError_t launch_attn_stream_64(const AttnParams& p, int nsm, cudaStream_t s) {
    if (p.k_q4) return p.v_q4 ? launch_attn_stream_mode<true, true, 64>(p, nsm, s) : launch_attn_stream_mode<true, false, 64>(p, nsm, s);
    return p.v_q4 ? launch_attn_stream_mode<false, true, 64>(p, nsm, s) : launch_attn_stream_mode<false, false, 64>(p, nsm, s);
}

}  // namespace ggq
