// ggq_norm.cu -- the norms before and after a block with its gate, scale and residual.
//
// Mathematics: t = residual + scale * act(gate) * N(x; after), out = N(t; before), with
// N(v; w) = v / sqrt(mean v^2 + eps) * (w + offset); either norm, the gate and the residual
// may be missing.  Statistics and everything between input and output are fp32; t is rounded
// to the rows' type when it is stored, the second norm takes it unrounded.
//
// Each value is read once and stays in registers between the two sums, so the bound is memory
// at many rows and the chain launch - load - sum - sum - store at few (one row of 4096: 2.8 us).  A row of up to 256
// channels is one warp's, wider ones a CTA's with eight channels a thread: the widest loads
// there are for 16-bit rows, and the eight that a packed block of 32 or 256 channels gives a
// lane, so that the packed forms are quantized from registers.  4096 rows of 4096 with a residual take 23.6 us as bf16
// rows (floor 19.8) and 28.7 to 29.7 as blocks (17.5), of fp32 52.0 (39.5) and 49.9 to 54.0 (32.4).
//
// Rows beyond 8192 channels, and odd or unaligned ones, are read without a row ahead, the latter value by value: 1024 of 16384
// 32.9 us (bf16, floor 19.8) and 53.0 (fp32, 39.5), 4096 of 4095 67.3 and 62.2.
#include <algorithm>

#include "ggq_device.cuh"
#include "ggq_internal.h"
#include "ggq_kv.cuh"
#include "ggq_norm.cuh"

namespace ggq {

namespace {

// Eight channels as they come from memory: asked for a row ahead
template <typename T>
struct Raw {
    uint4 u[sizeof(T) / 2];
    __device__ __forceinline__ void load(const T* p) {
#pragma unroll
        for (int i = 0; i < static_cast<int>(sizeof(T) / 2); ++i) u[i] = reinterpret_cast<const uint4*>(p)[i];
    }
    __device__ __forceinline__ void zero() {
#pragma unroll
        for (int i = 0; i < static_cast<int>(sizeof(T) / 2); ++i) u[i] = make_uint4(0, 0, 0, 0);
    }
    __device__ __forceinline__ void to(float (&x)[8]) const { ld8(reinterpret_cast<const T*>(u), x); }
};

// Eight consecutive channels of a row as four of a block of 32 (the quantizers of ggq_quantize_act).
// All lanes take part; `there`: this one writes.
template <bool SUMS>
__device__ __forceinline__ void quant32_regs(const float (&x)[8], uint8_t* block, bool there) {
    float m = 0.0f;
#pragma unroll
    for (int i = 0; i < 8; ++i) m = fmaxf(m, fabsf(x[i]));
    m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, 1));
    m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, 2));
    float id;
    const float d = quant_scale(m, &id);
    int q[8], s = 0;
#pragma unroll
    for (int i = 0; i < 8; ++i) s += q[i] = quant_one(x[i], id);
    s += __shfl_xor_sync(0xffffffffu, s, 1);
    s += __shfl_xor_sync(0xffffffffu, s, 2);
    if (!there) return;
    const int at = 8 * (threadIdx.x & 3);
    uint16_t* const to = reinterpret_cast<uint16_t*>(block + (SUMS ? 4 : 2) + at);
#pragma unroll
    for (int i = 0; i < 4; ++i) to[i] = static_cast<uint16_t>((q[2 * i] & 0xFF) | (q[2 * i + 1] & 0xFF) << 8);
    if (at == 0) {
        reinterpret_cast<__half*>(block)[0] = __float2half_rn(d);
        if (SUMS) reinterpret_cast<__half*>(block)[1] = __float2half_rn(__fmul_rn(d, static_cast<float>(s)));
    }
}

// The sum of v over the row's threads.  `part`: a slot for each warp, not in use by another sum.
template <bool WARP>
__device__ __forceinline__ float row_sum(float v, float* part) {
#pragma unroll
    for (int d = 16; d >= 1; d >>= 1) v += __shfl_xor_sync(0xffffffffu, v, d);
    if constexpr (!WARP) {
        const int warps = static_cast<int>(blockDim.x) >> 5, lane = threadIdx.x & 31;
        if (lane == 0) part[threadIdx.x >> 5] = v;
        __syncthreads();
        v = lane < warps ? part[lane] : 0.0f;
#pragma unroll
        for (int d = 16; d >= 1; d >>= 1) v += __shfl_xor_sync(0xffffffffu, v, d);
    }
    return v;
}

// Words of a weight in shared memory: a group of eight as two quads, so that neighbouring lanes' quads are neighbours.
__device__ __forceinline__ int weight_at(int group, int half, int threads) { return 4 * (half * threads + group); }

// NU: groups of eight channels a thread holds.  THREADS: at most so many a CTA; a row is a CTA's, with 128 a
// warp's.  VEC: rows of whole aligned groups; otherwise a thread's channels lie a row's threads apart and are
// loaded one by one.  With one group a thread (AHEAD: rows of up to 8192 channels) a CTA keeps the weights in
// shared memory, goes through rows and asks for everything that the next one needs before it sums (4096 rows of 4096
// bf16 channels, two norms, gate and residual: 28.5 us; 42.4 with a CTA a row, 34.4 with the weights in registers).
template <typename T, int NU, int THREADS, bool VEC>
__global__ void __launch_bounds__(THREADS, THREADS == 1024 ? 1 : 1024 / THREADS) k_norm(const __grid_constant__ NormParams p) {
    constexpr bool WARP = THREADS == 128, AHEAD = VEC && NU == 1;
    pdl_launch_dependents();
    pdl_wait();
    extern __shared__ __align__(16) float weights[];  // AHEAD: of the two norms, two quads a thread
    __shared__ float part[4][32];
    const int threads = WARP ? 32 : static_cast<int>(blockDim.x), at = WARP ? threadIdx.x & 31 : threadIdx.x;
    const int64_t step = WARP ? static_cast<int64_t>(gridDim.x) * 4 : gridDim.x;
    int64_t t = WARP ? static_cast<int64_t>(blockIdx.x) * 4 + (threadIdx.x >> 5) : blockIdx.x;
    const auto first = [&](int u) { return VEC ? (u * threads + at) * 8 : u * 8 * threads + at; };
    const auto channel = [&](int u, int i) { return first(u) + (VEC ? i : i * threads); };
    // channels behind the row's end are zeros
    const auto load = [&](const auto* row, int u, float (&x)[8]) {
#pragma unroll
        for (int i = 0; i < 8; ++i) x[i] = 0.0f;
        if constexpr (VEC) {
            if (first(u) < p.H) ld8(row + first(u), x);
        } else {
#pragma unroll
            for (int i = 0; i < 8; ++i)
                if (channel(u, i) < p.H) x[i] = ld1(row + channel(u, i));
        }
    };
    const auto store = [&](T* row, int u, const float (&x)[8]) {
        if constexpr (VEC) {
            if (first(u) < p.H) st8(row + first(u), x);
        } else {
#pragma unroll
            for (int i = 0; i < 8; ++i)
                if (channel(u, i) < p.H) st1(row + channel(u, i), x[i]);
        }
    };
    const T* const xs = static_cast<const T*>(p.x);
    const T* const rs = static_cast<const T*>(p.residual);
    const T* const gs = static_cast<const T*>(p.gate);
    const bool gates = p.gate && p.gate_channel;
    // a row's groups as they come from memory
    Raw<T> next_x, next_r, next_g;
    if constexpr (AHEAD) next_x.zero(), next_r.zero(), next_g.zero();
    const auto ask = [&](int64_t row) {
        if (first(0) >= p.H) return;
        next_x.load(xs + row * p.x_token + first(0));
        if (p.residual) next_r.load(rs + row * p.residual_token + first(0));
        if (gates) next_g.load(gs + row * p.gate_token + first(0));
    };
    const auto act = [&](float x) { return p.sigmoid ? __frcp_rn(1.0f + expf(-x)) : x; };
    if constexpr (AHEAD)
        if (t < p.T) ask(t);
    float* const mine = weights + 8 * threads * (WARP ? 2 * (threadIdx.x >> 5) : 0);
    if constexpr (AHEAD) {
#pragma unroll
        for (int k = 0; k < 2; ++k) {
            const float* const w = k ? p.before_w : p.after_w;
            if (!w) continue;
            float x[8];
            load(w, 0, x);
#pragma unroll
            for (int i = 0; i < 8; ++i) x[i] = __fadd_rn(x[i], p.offset);
            // (read by this thread alone)
            float* const to = mine + k * 8 * threads;
            st4(to + weight_at(at, 0, threads), make_float4(x[0], x[1], x[2], x[3]));
            st4(to + weight_at(at, 1, threads), make_float4(x[4], x[5], x[6], x[7]));
        }
    }
    // w + offset of group u; k: 0 of the norm of x, 1 of the total's
    const auto weight = [&](const float* w, int k, int u, float (&x)[8]) {
        if constexpr (AHEAD) {
            const float* const from = mine + k * 8 * threads;
            const float4 a = ld4(from + weight_at(at, 0, threads)), b = ld4(from + weight_at(at, 1, threads));
            x[0] = a.x, x[1] = a.y, x[2] = a.z, x[3] = a.w, x[4] = b.x, x[5] = b.y, x[6] = b.z, x[7] = b.w;
        } else {
            load(w, u, x);
#pragma unroll
            for (int i = 0; i < 8; ++i) x[i] = __fadd_rn(x[i], p.offset);
        }
    };
    for (int turn = 0; t < p.T; t += step, turn ^= 2) {
        float v[NU][8];
        const Raw<T> r = next_r, g = next_g;
        if constexpr (AHEAD) {
            next_x.to(v[0]);
        } else {
#pragma unroll
            for (int u = 0; u < NU; ++u) load(xs + t * p.x_token, u, v[u]);
        }
        float g1 = p.gate && !p.gate_channel ? ld1(gs + t * p.gate_token) : 1.0f;
        if constexpr (AHEAD)
            if (t + step < p.T) ask(t + step);
        const auto inverse = [&](float* parts) {
            float s = 0.0f;
#pragma unroll
            for (int u = 0; u < NU; ++u)
#pragma unroll
                for (int i = 0; i < 8; ++i) s = fmaf(v[u][i], v[u][i], s);
            return rsqrtf(fmaf(row_sum<WARP>(s, parts), p.inv_width, p.eps));
        };
        const float inv_after = p.after ? inverse(part[turn]) : 1.0f;
        if (p.gate && !p.gate_channel) g1 = act(g1);
#pragma unroll
        for (int u = 0; u < NU; ++u) {
            float x[8];
            if (p.after_w) {
                weight(p.after_w, 0, u, x);
#pragma unroll
                for (int i = 0; i < 8; ++i) v[u][i] = v[u][i] * inv_after * x[i];
            } else if (p.after) {
#pragma unroll
                for (int i = 0; i < 8; ++i) v[u][i] *= inv_after;
            }
            if (gates) {
                if constexpr (AHEAD) g.to(x);
                else load(gs + t * p.gate_token, u, x);
#pragma unroll
                for (int i = 0; i < 8; ++i) v[u][i] *= act(x[i]);
            } else {
#pragma unroll
                for (int i = 0; i < 8; ++i) v[u][i] *= g1;
            }
            if constexpr (AHEAD) {
                r.to(x);
            } else {
                if (p.residual) load(rs + t * p.residual_token, u, x);
                else
#pragma unroll
                    for (int i = 0; i < 8; ++i) x[i] = 0.0f;
            }
#pragma unroll
            for (int i = 0; i < 8; ++i) v[u][i] = fmaf(v[u][i], p.scale, x[i]);
            if (p.total) store(static_cast<T*>(p.total) + t * p.total_token, u, v[u]);
        }
        if (!p.before) continue;
        const float inv = inverse(part[turn + 1]);
#pragma unroll
        for (int u = 0; u < NU; ++u) {
            float x[8];
            if (p.before_w) {
                weight(p.before_w, 1, u, x);
#pragma unroll
                for (int i = 0; i < 8; ++i) v[u][i] = v[u][i] * inv * x[i];
            } else {
#pragma unroll
                for (int i = 0; i < 8; ++i) v[u][i] *= inv;
            }
            if (p.out) store(static_cast<T*>(p.out) + t * p.out_token, u, v[u]);
            if constexpr (VEC) {
                if (p.packed) {
                    const int c = first(u);
                    const int64_t row = t * p.H;
                    if (p.form == NORM_Q8_K) {  // whole warps: the width is a multiple of 256
                        if (c < p.H) warp_quant_q8k_regs(v[u], p.packed + ((row + c) >> 8) * 292, threadIdx.x & 31);
                    } else if (p.form == NORM_Q8_1) {
                        quant32_regs<true>(v[u], p.packed + ((row + c) >> 5) * 36, c < p.H);
                    } else {
                        quant32_regs<false>(v[u], p.packed + ((row + c) >> 5) * 34, c < p.H);
                    }
                }
            }
        }
    }
}

template <typename T, int NU, int THREADS, bool VEC>
cudaError_t launch_rows(const NormParams& p, cudaStream_t s) {
    constexpr bool WARP = THREADS == 128;
    const int threads = WARP ? 128 : (p.H + 256 * NU - 1) / (256 * NU) * 32;
    const int64_t ctas = WARP ? (p.T + 3) / 4 : p.T;
    // as many CTAs as the SMs hold at once go through the rows
    const dim3 grid(static_cast<unsigned>(std::min<int64_t>(ctas, 152 * (1024 / threads))));
    const size_t smem = VEC && NU == 1 ? static_cast<size_t>(threads) * 64 : 0;
    if (smem > 48 * 1024) {
        static thread_local bool done[kMaxDevices] = {};
        int dev = 0;
        cudaError_t e = cudaGetDevice(&dev);
        if (e == cudaSuccess && (dev >= kMaxDevices || !done[dev])) {
            e = cudaFuncSetAttribute(k_norm<T, NU, THREADS, VEC>, cudaFuncAttributeMaxDynamicSharedMemorySize, 1024 * 64);
            if (e == cudaSuccess && dev < kMaxDevices) done[dev] = true;
        }
        if (e != cudaSuccess) return e;
    }
    return launch_pdl(k_norm<T, NU, THREADS, VEC>, grid, dim3(static_cast<unsigned>(threads)), smem, s, p);
}

template <typename T, bool VEC>
cudaError_t launch(const NormParams& p, cudaStream_t s) {
    if (p.H <= 256) return launch_rows<T, 1, 128, VEC>(p, s);
    if (p.H <= 4096) return launch_rows<T, 1, 512, VEC>(p, s);
    if (p.H <= 8192) return launch_rows<T, 1, 1024, VEC>(p, s);
    if (p.H <= 16384) return launch_rows<T, 2, 1024, VEC>(p, s);
    return launch_rows<T, 4, 1024, VEC>(p, s);
}

template <typename T>
cudaError_t launch_type(const NormParams& p, bool whole, cudaStream_t s) {
    return whole ? launch<T, true>(p, s) : launch<T, false>(p, s);
}

}  // namespace

bool norm_whole(const NormParams& p, int dtype) {
    const int size = dtype == 0 ? 4 : 2;
    const auto whole = [&](const void* at, int64_t stride) { return aligned_to(at, 16) && (!at || p.T < 2 || stride * size % 16 == 0); };
    return p.H % 8 == 0 && whole(p.x, p.x_token) && whole(p.residual, p.residual_token) &&
           (!p.gate || !p.gate_channel || whole(p.gate, p.gate_token)) && whole(p.total, p.total_token) && whole(p.out, p.out_token) &&
           aligned_to(p.after_w, 16) && aligned_to(p.before_w, 16);
}

cudaError_t launch_norm(const NormParams& p, int dtype, cudaStream_t s) {
    if (p.T == 0) return cudaSuccess;
    const bool whole = norm_whole(p, dtype);
    if (dtype == 0) return launch_type<float>(p, whole, s);
    if (dtype == 1) return launch_type<__half>(p, whole, s);
    return launch_type<__nv_bfloat16>(p, whole, s);
}

}  // namespace ggq
