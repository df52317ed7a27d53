// ggq_attn.cu -- which kernel an attention call over the packed cache takes.
#include "ggq_attn.cuh"
#include "ggq_internal.h"

namespace ggq {

cudaError_t launch_attention(const AttnParams& p, int nsm, cudaStream_t s) {
    if (p.D == 64) return launch_attn_stream_64(p, nsm, s);
    if (p.D == 128) return launch_attn_stream_128(p, nsm, s);
    return launch_attn_stream_256(p, nsm, s);
}

}  // namespace ggq
