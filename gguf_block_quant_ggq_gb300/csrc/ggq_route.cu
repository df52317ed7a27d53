// ggq_route.cu -- the expert router: scores, choice, groups, top-k, weights.
//
// Mathematics: score = softmax(l) or sigmoid(l); choice = score + bias (softmax
// without bias: the logits, whose order is the scores'; sums of a group's two best
// are of scores always); only the best groups' experts stay; the top_k choices in
// order, ties to the lower id; weights are the chosen scores, renormalised and scaled.  Reads each logit once; at a few
// thousand tokens bound by the k dependent rounds of the selection, not by
// bytes.
//
// One warp a token: lane l holds experts NV l .. NV l + NV - 1 as order-preserving
// 32-bit keys, in registers, so that lanes and places in them follow the experts'
// order.  A round of the choice is one redux for the warp's largest key, one ballot
// for the first lane that has it, and that lane's own search; groups of whole lanes
// are scored by butterflies over all groups at once.  Bound by its instructions at
// many tokens (4096 tokens of 256 experts in 8 groups: 11 us, 1250 instructions a
// token, where the logits' 4 MB take under 1 us; with the experts interleaved over the
// lanes and groups scored one after another 16 us and 2000), by the launch at few (4 us).
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
    const float e = expf(sigmoid ? -x : __fsub_rn(x, m));
    const float s = sigmoid ? __frcp_rn(__fadd_rn(1.0f, e)) : x == m ? 1.0f : e;
    return x != x ? 0.0f : s;
}

// A group's score as a key: the value of its largest key, or the sum of its two largest
// ones' (of one where the group has no second).  Keys of logits (softmax without bias) stand in the order of the scores, but
// their sums do not: the scores are added then.
struct GroupScore {
    bool two, logits;
    float m, inv;
    __device__ __forceinline__ float value(uint32_t key) const {
        const float x = value_of(key);
        return logits && key > kNaN ? __fmul_rn(score_of(x, false, m), inv) : x;
    }
    __device__ __forceinline__ uint32_t key(uint32_t a, uint32_t b) const {
        return key_of(!two ? value_of(a) : b == kTaken ? value(a) : __fadd_rn(value(a), value(b)));
    }
};

// NV: keys a lane holds in registers (E <= 32 NV).
template <int NV, typename T>
__global__ void __launch_bounds__(128) k_route(const __grid_constant__ RouteParams p) {
    pdl_launch_dependents();
    pdl_wait();
    __shared__ uint32_t s_keys[NV <= 16 ? 4 * 32 * NV : 1];  // groups that are not whole lanes
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int64_t t = static_cast<int64_t>(blockIdx.x) * 4 + warp;
    if (t >= p.T) return;
    const T* const row = static_cast<const T*>(p.logits) + t * p.E;
    const bool sigmoid = p.sigmoid != 0;
    const int e0 = lane * NV;
    float x[NV];
    if (p.quads) {
#pragma unroll
        for (int i = 0; i < NV; i += 4) {
            const float4 v = e0 + i < p.E ? ld4(row + e0 + i) : make_float4(-INFINITY, -INFINITY, -INFINITY, -INFINITY);
            x[i] = v.x, x[i + 1] = v.y, x[i + 2] = v.z, x[i + 3] = v.w;
        }
    } else {
#pragma unroll
        for (int i = 0; i < NV; ++i) x[i] = e0 + i < p.E ? ld1(row + e0 + i) : -INFINITY;
    }
    float m = 0.0f, inv = 1.0f;
    if (!sigmoid) {
        m = -INFINITY;
#pragma unroll
        for (int i = 0; i < NV; ++i) m = fmaxf(m, x[i]);
        m = warp_max(m);
        if (m == -INFINITY) m = 0.0f;  // a row of -inf: every score 0
        // the scores themselves are needed, not only their ratios (the sums of two: the same with a bias of 0)
        if (p.bias || !p.normalize || (p.n_groups > 1 && p.group_best == 2)) {
            float s = 0.0f;
#pragma unroll
            for (int i = 0; i < NV; ++i) s += score_of(x[i], false, m);
#pragma unroll
            for (int d = 16; d >= 1; d >>= 1) s += __shfl_xor_sync(kFull, s, d);
            inv = s > 0.0f ? __fdiv_rn(1.0f, s) : 0.0f;
        }
    }
    uint32_t key[NV], best = kTaken;
#pragma unroll
    for (int i = 0; i < NV; ++i) {
        float c = x[i];
        if (p.bias || sigmoid) {
            c = __fmul_rn(score_of(c, sigmoid, m), inv);
            if (p.bias) c = __fadd_rn(c, e0 + i < p.E ? p.bias[e0 + i] : 0.0f);
            if (x[i] != x[i]) c = x[i];
        }
        key[i] = e0 + i < p.E ? key_of(c) : kTaken;
    }
    if (p.n_groups > 1) {
        const int per = p.E / p.n_groups, lanes = per / NV;  // lanes of a group
        const GroupScore score{p.group_best == 2, !sigmoid && !p.bias, m, inv};
        const bool whole = lanes * NV == per && (lanes & (lanes - 1)) == 0;
        uint32_t mine = kTaken;  // this lane's group's score; lanes that are not a group's first one: none
        if (whole) {
            uint32_t a = kTaken, b = kTaken;  // the two largest keys
#pragma unroll
            for (int i = 0; i < NV; ++i) {
                b = max(b, min(a, key[i]));
                a = max(a, key[i]);
            }
            for (int d = 1; d < lanes; d <<= 1) {
                const uint32_t oa = __shfl_xor_sync(kFull, a, d), ob = __shfl_xor_sync(kFull, b, d);
                b = max(max(b, ob), min(a, oa));
                a = max(a, oa);
            }
            if ((lane & (lanes - 1)) == 0 && e0 < p.E) mine = score.key(a, b);
        } else if constexpr (NV <= 16) {
            uint32_t* const keys = s_keys + warp * 32 * NV;
#pragma unroll
            for (int i = 0; i < NV; ++i) keys[e0 + i] = key[i];
            __syncwarp();
            if (lane < p.n_groups) {
                uint32_t a = kTaken, b = kTaken;
                for (int i = 0; i < per; ++i) {
                    const uint32_t k = keys[lane * per + i];
                    b = max(b, min(a, k));
                    a = max(a, k);
                }
                mine = score.key(a, b);
            }
        } else {
            for (int g = 0; g < p.n_groups; ++g) {
                uint32_t a = kTaken, b = kTaken;
#pragma unroll
                for (int i = 0; i < NV; ++i)
                    if (e0 + i >= g * per && e0 + i < (g + 1) * per) {
                        b = max(b, min(a, key[i]));
                        a = max(a, key[i]);
                    }
                const uint32_t first = __reduce_max_sync(kFull, a);
                if (lane == __ffs(__ballot_sync(kFull, a == first)) - 1) a = b;
                const uint32_t second = __reduce_max_sync(kFull, a);
                if (lane == g) mine = score.key(first, second);
            }
        }
        uint32_t open = 0u;  // bit l: the group that lane l scored stays open
        for (int j = 0; j < p.top_groups; ++j) {
            const uint32_t top = __reduce_max_sync(kFull, mine);
            const int l = __ffs(__ballot_sync(kFull, mine == top)) - 1;
            open |= 1u << l;
            if (lane == l) mine = kTaken;
        }
        if (whole) {
            if (!((open >> (lane & ~(lanes - 1))) & 1u))
#pragma unroll
                for (int i = 0; i < NV; ++i) key[i] = kTaken;
        } else {
#pragma unroll
            for (int i = 0; i < NV; ++i)
                if (e0 + i < p.E && !((open >> ((e0 + i) / per)) & 1u)) key[i] = kTaken;
        }
    }
#pragma unroll
    for (int i = 0; i < NV; ++i) best = max(best, key[i]);
    int id = 0;  // lane j: the j-th choice
    for (int j = 0; j < p.k; ++j) {
        const uint32_t top = __reduce_max_sync(kFull, best);
        const int l = __ffs(__ballot_sync(kFull, best == top)) - 1;
        int at = 0;
        if (lane == l) {  // its first key of that size is taken
            best = kTaken;
#pragma unroll
            for (int i = NV - 1; i >= 0; --i) at = key[i] == top ? i : at;
#pragma unroll
            for (int i = 0; i < NV; ++i) {
                if (i == at) key[i] = kTaken;
                best = max(best, key[i]);
            }
        }
        at = __shfl_sync(kFull, at, l);
        if (lane == j) id = l * NV + at;
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
cudaError_t launch(RouteParams p, cudaStream_t s) {
    p.quads = p.E % 4 == 0 && reinterpret_cast<uintptr_t>(p.logits) % (4 * sizeof(T)) == 0;
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
