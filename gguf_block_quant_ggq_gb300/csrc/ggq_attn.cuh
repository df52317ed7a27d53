// ggq_attn.cuh -- parameters of the attention kernels over the packed cache.
#pragma once
#include <cuda_runtime.h>
#include <stdint.h>

#include "ggq_attn_plan.h"
#include "ggq_kv.cuh"

namespace ggq {

struct AttnParams {
    const void* q;
    void* out;
    int64_t q_token, q_head, out_token, out_head;  // strides in elements
    const uint8_t* k;
    const uint8_t* v;
    const int32_t* table;
    const int32_t* lens;
    const int32_t* q_start;  // null: row b belongs to sequence b
    const float* slopes;
    int64_t table_stride;
    int64_t n_pages;
    int64_t n_tokens, n_seqs;
    int dtype;               // 0 f32, 1 f16, 2 bf16
    int H, Hkv, G, D, page;
    uint32_t page_magic;     // 2^32 / (page / 16) + 1
    int k_q4, v_q4;
    int max_q, max_len, window;
    float scale, cap;
    int min_share;           // units (one or two 16-token groups) below which a CTA's share is not cut
    float* parts;            // partial results [2 * kAttnMaxCtas][attn_part_floats(D)]
    int* pieces;             // arrival counters [kAttnCounters], zero between calls
    int* err;
};

// Bounds of a call: a sequence's tokens and the call's rows.  Positions are 32-bit: a key
// behind a sequence's last tile, and a position (at least -rows) minus a window (less than the
// longest sequence), stay in range.
constexpr int64_t kAttnMaxRows = 1 << 24, kAttnMaxLen = (1ll << 31) - (1 << 25);

// The kernels of 16-bit rows form cap * tanh(z) as cap - 2 cap / (1 + exp(2 z)), whose error is
// a few 2^-23 cap.  Beyond this cap that would show beside the scores' own roundings: such
// calls take the streaming kernel of fp32 rows, which has tanhf, at its times for fp32 (32
// heads on 8 of 128 channels, bf16, caps 50 / 2000: one token of 64 sequences of 4096 119 /
// 143 us, a prompt of 4096 274 / 4160 us).
constexpr float kWideCap = 1024.0f;

// A partial result: reference maxima [16], sums [16], values [16][D]; CTAs an SM at most for
// heads of 256 channels.
__host__ __device__ constexpr int attn_part_floats(int D) { return 32 + 16 * D; }
constexpr int kAttnWideCtas = 2;

cudaError_t launch_attention(const AttnParams& p, int nsm, cudaStream_t s);
cudaError_t launch_attn_stream_64(const AttnParams& p, int nsm, cudaStream_t s);
cudaError_t launch_attn_stream_128(const AttnParams& p, int nsm, cudaStream_t s);
cudaError_t launch_attn_stream_256(const AttnParams& p, int nsm, cudaStream_t s);
cudaError_t launch_attn_rows_256(const AttnParams& p, cudaStream_t s);
cudaError_t launch_attn_promptf_64(const AttnParams& p, cudaStream_t s);
cudaError_t launch_attn_promptf_128(const AttnParams& p, cudaStream_t s);
cudaError_t launch_attn_prompt_64(const AttnParams& p, cudaStream_t s);
cudaError_t launch_attn_prompt_128(const AttnParams& p, cudaStream_t s);
cudaError_t launch_attn_prompt_256(const AttnParams& p, cudaStream_t s);

}  // namespace ggq
