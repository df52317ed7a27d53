// ggq_adapt.cuh -- parameters of the low-rank adapters beside a projection (ggq_adapt.cu).
#pragma once
#include <cuda_runtime.h>
#include <stdint.h>

namespace ggq {

constexpr int kAdaptMaxRank = 256;

struct AdaptParams {
    const void* a;  // [n][R][K]
    const void* b;  // [n][N][R]
    const int32_t* ranks;  // [n] or null
    const float* scales;   // [n] or null
    int64_t n;
    int R, K;
    int64_t N;
    const void* x;
    const void* y;
    void* out;
    int64_t x_token, y_token, out_token;  // strides in elements
    const int32_t* ids;      // [seqs]
    const int32_t* q_start;  // [seqs + 1] or null: a row a sequence
    int64_t T, seqs;
    int bank;   // 1 f16, 2 bf16
    int x_whole, y_whole, out_whole;  // rows start at 16 bytes (y, out: 2; 1: at four elements) (set by the launch)
    int stages1, stages2;            // blocks of the two products' rings (set by the launch)
    int* err;
};

cudaError_t launch_adapt(const AdaptParams& p, int dtype, cudaStream_t s);

}  // namespace ggq
