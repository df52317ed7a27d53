// ggq_norm.cuh -- parameters of the norms around a block (ggq_norm.cu).
#pragma once
#include <cuda_runtime.h>
#include <stdint.h>

namespace ggq {

constexpr int kNormMaxWidth = 32768;
enum NormPacked : int { NORM_ROWS = 0, NORM_Q8_K = 1, NORM_Q8_1 = 2, NORM_Q8_0 = 3 };

struct NormParams {
    const void* x;
    const void* residual;   // or null
    const void* gate;       // or null
    void* total;            // or null
    void* out;              // or null
    uint8_t* packed;        // or null
    const float* after_w;   // or null: none
    const float* before_w;  // or null: none
    int64_t x_token, residual_token, gate_token, total_token, out_token;  // strides in elements
    int64_t T;
    int H;
    int gate_channel;  // 0: one gate a token
    int sigmoid;
    int after, before;
    int form;          // NormPacked of `packed`
    float scale, eps, offset, inv_width;
};

// Rows of whole aligned groups of eight channels: 16-byte loads, and what packed outputs need.
bool norm_whole(const NormParams& p, int dtype);
cudaError_t launch_norm(const NormParams& p, int dtype, cudaStream_t s);

}  // namespace ggq
