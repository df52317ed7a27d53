// ggq_logprobs.cuh -- parameters of the log probabilities of given tokens (ggq_logprobs.cu).
#pragma once
#include <cuda_runtime.h>
#include <stdint.h>

namespace ggq {

constexpr int kLogprobsMaxTop = 32;

struct LogprobsParams {
    const void* logits;
    int64_t row;  // stride in elements
    int64_t T;
    int V;
    const int32_t* tokens;  // [T][given]
    int given;
    float* logprobs;  // [T][given]
    float* entropy;   // [T] or null
    int top;
    int32_t* ids;     // [T][top]
    float* best;      // [T][top]
    float scale;      // of the logits
    int* err;
};

cudaError_t launch_logprobs(const LogprobsParams& p, int dtype, cudaStream_t s);

}  // namespace ggq
