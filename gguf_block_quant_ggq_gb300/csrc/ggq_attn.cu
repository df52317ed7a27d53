// ggq_attn.cu -- which kernel an attention call over the packed cache takes.
#include "ggq_attn.cuh"
#include "ggq_internal.h"

namespace ggq {

// Query rows of a sequence and kv head from which a call takes the tcgen05 kernel.
constexpr int64_t kPromptRows = 64;

cudaError_t launch_attention(const AttnParams& p, int nsm, cudaStream_t s) {
    const int64_t rows = static_cast<int64_t>(p.max_q) * p.G;
    if (p.dtype != 0 && rows >= kPromptRows && rows <= 128ll * 65535) {
        if (p.D == 64) return launch_attn_prompt_64(p, s);
        if (p.D == 128) return launch_attn_prompt_128(p, s);
        return launch_attn_prompt_256(p, s);
    }
    if (p.dtype == 0 && rows >= kPromptRows && rows <= 64ll * 65535) {
        if (p.D == 64) return launch_attn_promptf_64(p, s);
        if (p.D == 128) return launch_attn_promptf_128(p, s);
        return launch_attn_rows_256(p, s);
    }
    if (p.D == 64) return launch_attn_stream_64(p, nsm, s);
    if (p.D == 128) return launch_attn_stream_128(p, nsm, s);
    return launch_attn_stream_256(p, nsm, s);
}

}  // namespace ggq
