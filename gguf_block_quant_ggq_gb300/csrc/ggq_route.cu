// ggq_route.cu -- the expert router: scores, choice, groups, top-k, weights.
//
// Mathematics: score = softmax(l) or sigmoid(l); choice = score + bias (softmax
// without bias: the logits, whose order is the scores'); only the best groups'
// experts stay; the top_k choices in order, ties to the lower id; weights are
// the chosen scores, renormalised and scaled.  Reads each logit once; at a few
// thousand tokens bound by the k dependent rounds of the selection, not by
// bytes.
//
// One warp a token: lane l holds experts l, l + 32, ... as order-preserving
// 32-bit keys, in registers.  A round is a maximum over the lane's keys, one
// redux for the warp's largest key and one for the lowest expert that has it.
#include "ggq_device.cuh"
#include "ggq_internal.h"
#include "ggq_kv.cuh"
#include "ggq_route.cuh"

namespace ggq {

namespace {

constexpr uint32_t kFull = 0xffffffffu;
constexpr uint32_t kTaken = 0u, kNaN = 1u;  // below the key of every number

// Larger key = larger value; -0 counts as +0, a NaN is below -inf.
__device__ __forceinline__ uint32_t key_of(float x) {
    const uint32_t b = __float_as_uint(__fadd_rn(x, 0.0f));
    return x != x ? kNaN : (b & 0x80000000u) ? ~b : b | 0x80000000u;
}
__device__ __forceinline__ float value_of(uint32_t key) {
    return key <= kNaN ? -INFINITY : __uint_as_float(key & 0x80000000u ? key & 0x7fffffffu : ~key);
}

// score of logit x; m: the row's maximum (softmax numerators).  A NaN scores 0.
__device__ __forceinline__ float score_of(float x, bool sigmoid, float m) {
    if (x != x) return 0.0f;
    if (sigmoid) return __fdiv_rn(1.0f, __fadd_rn(1.0f, expf(-x)));
    return x == m ? 1.0f : expf(__fsub_rn(x, m));
}

// NV: keys a lane holds in registers (E <= 32 NV).
template <int NV, typename T>
__global__ void __launch_bounds__(128) k_route(const __grid_constant__ RouteParams p) {
    pdl_launch_dependents();
    pdl_wait();
    const int lane = threadIdx.x & 31;
    const int64_t t = (static_cast<int64_t>(blockIdx.x) * blockDim.x + threadIdx.x) >> 5;
    if (t >= p.T) return;
    const T* const row = static_cast<const T*>(p.logits) + t * p.E;
    const bool sigmoid = p.sigmoid != 0;
    float x[NV];
#pragma unroll
    for (int i = 0; i < NV; ++i) x[i] = lane + 32 * i < p.E ? ld1(row + lane + 32 * i) : -INFINITY;
    float m = 0.0f, inv = 1.0f;
    if (!sigmoid) {
        m = -INFINITY;
#pragma unroll
        for (int i = 0; i < NV; ++i) m = fmaxf(m, x[i]);
        m = warp_max(m);
        if (m == -INFINITY) m = 0.0f;  // a row of -inf: every score 0
        if (p.bias || !p.normalize) {  // the scores themselves are needed, not only their ratios
            float s = 0.0f;
#pragma unroll
            for (int i = 0; i < NV; ++i) s += score_of(x[i], false, m);
#pragma unroll
            for (int d = 16; d >= 1; d >>= 1) s += __shfl_xor_sync(kFull, s, d);
            inv = s > 0.0f ? __fdiv_rn(1.0f, s) : 0.0f;
        }
    }
    uint32_t key[NV];
#pragma unroll
    for (int i = 0; i < NV; ++i) {
        const int e = lane + 32 * i;
        float c = x[i];
        if (c == c && (p.bias || sigmoid)) {
            c = __fmul_rn(score_of(c, sigmoid, m), inv);
            if (p.bias) c = __fadd_rn(c, e < p.E ? p.bias[e] : 0.0f);
        }
        key[i] = e < p.E ? key_of(c) : kTaken;
    }
    if (p.n_groups > 1) {
        const int per = p.E / p.n_groups;
        uint32_t mine = kTaken;  // lane g: group g's score
        for (int g = 0; g < p.n_groups; ++g) {
            uint32_t a = kTaken, b = kTaken;  // this lane's two largest keys of the group
#pragma unroll
            for (int i = 0; i < NV; ++i) {
                const int e = lane + 32 * i;
                if (e >= g * per && e < (g + 1) * per) {
                    b = max(b, min(a, key[i]));
                    a = max(a, key[i]);
                }
            }
            const uint32_t first = __reduce_max_sync(kFull, a);
            float s = value_of(first);
            if (p.group_best == 2) {
                const uint32_t who = __ballot_sync(kFull, a == first);
                if (lane == __ffs(who) - 1) a = b;
                s = __fadd_rn(s, value_of(__reduce_max_sync(kFull, a)));
            }
            if (lane == g) mine = key_of(s);
        }
        uint32_t open = 0u;
        for (int j = 0; j < p.top_groups; ++j) {
            const uint32_t best = __reduce_max_sync(kFull, mine);
            const int g = __ffs(__ballot_sync(kFull, mine == best && lane < p.n_groups && !((open >> lane) & 1u))) - 1;
            open |= 1u << g;
            if (lane == g) mine = kTaken;
        }
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            const int e = lane + 32 * i;
            if (e < p.E && !((open >> (e / per)) & 1u)) key[i] = kTaken;
        }
    }
    int id = 0;  // lane j: the j-th choice
    for (int j = 0; j < p.k; ++j) {
        uint32_t a = kTaken;
#pragma unroll
        for (int i = 0; i < NV; ++i) a = max(a, key[i]);
        const uint32_t best = __reduce_max_sync(kFull, a);
        int e = 0x7fffffff;
#pragma unroll
        for (int i = NV - 1; i >= 0; --i)
            if (key[i] == best) e = lane + 32 * i;
        e = __reduce_min_sync(kFull, e);
#pragma unroll
        for (int i = 0; i < NV; ++i)
            if (lane + 32 * i == e) key[i] = kTaken;
        if (lane == j) id = e;
    }
    const float w = lane < p.k ? __fmul_rn(score_of(ld1(row + id), sigmoid, m), inv) : 0.0f;
    float sum = w;
#pragma unroll
    for (int d = 16; d >= 1; d >>= 1) sum += __shfl_xor_sync(kFull, sum, d);
    if (lane < p.k) {
        p.ids[t * p.k + lane] = id;
        p.weights[t * p.k + lane] = (p.normalize ? (sum > 0.0f ? __fdiv_rn(w, sum) : 0.0f) : w) * p.scale;
    }
}

template <typename T>
cudaError_t launch(const RouteParams& p, cudaStream_t s) {
    const dim3 grid(static_cast<unsigned>((p.T + 3) / 4));
    if (p.E <= 128) return launch_pdl(k_route<4, T>, grid, dim3(128), 0, s, p);
    if (p.E <= 256) return launch_pdl(k_route<8, T>, grid, dim3(128), 0, s, p);
    if (p.E <= 512) return launch_pdl(k_route<16, T>, grid, dim3(128), 0, s, p);
    return launch_pdl(k_route<128, T>, grid, dim3(128), 0, s, p);
}

}  // namespace

cudaError_t launch_route(const RouteParams& p, int dtype, cudaStream_t s) {
    if (p.T == 0) return cudaSuccess;
    if (dtype == 0) return launch<float>(p, s);
    if (dtype == 1) return launch<__half>(p, s);
    return launch<__nv_bfloat16>(p, s);
}

}  // namespace ggq
