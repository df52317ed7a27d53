// ggq_route.cuh -- parameters of the expert router (ggq_route.cu).
#pragma once
#include <cuda_runtime.h>
#include <stdint.h>

namespace ggq {

constexpr int kRouteMaxExperts = 4096, kRouteMaxTopK = 32, kRouteMaxGroups = 32;

struct RouteParams {
    const void* logits;
    const float* bias;
    int64_t T;
    int E, k, n_groups, top_groups, group_best;
    int sigmoid, normalize;
    int quads;  // rows of whole aligned quads (set by the launch)
    float scale;
    int32_t* ids;
    float* weights;
};

cudaError_t launch_route(const RouteParams& p, int dtype, cudaStream_t s);

}  // namespace ggq
