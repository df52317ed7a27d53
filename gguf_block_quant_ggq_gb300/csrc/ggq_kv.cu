// ggq_kv.cu -- quantizing keys and values into the paged cache and reading them back.
//
// Mathematics: per token and 32 channels, Q8_0 d = amax * (1/127), q = round(x / d);
// Q4_0 d = m / -8 with m the first value of the largest magnitude, q = floor(x /
// d + 8.5) in 0..15.  Bound by memory: each value is read once and stands in the
// cache for 17/16 (Q8_0) or 9/16 (Q4_0) bytes.
//
// A CTA takes 16 consecutive rows of one head's keys or values.  Rows whose
// slots fill an aligned group of 16 (the tokens of a prompt) are quantized as a
// group: a warp holds what one 512-byte line of the blob needs, reduces the
// blocks' extremes inside itself and writes the line whole.  Other rows (one
// token of each sequence) go row by row, four channels a lane: a word of a K
// blob, four bytes of a V blob.
#include "ggq_device.cuh"
#include "ggq_internal.h"
#include "ggq_kv.cuh"

namespace ggq {

namespace {

constexpr int kKvThreads = 128;
constexpr int kKvRows = 16;

// The extreme of a Q4_0 block while it is reduced: the value of the largest
// magnitude, the first one (smallest channel) on a tie.
struct Extreme {
    float v;
    int at;
};
__device__ __forceinline__ void take(Extreme& a, float v, int at) {
    const float x = fabsf(v), y = fabsf(a.v);
    if (x > y || (x == y && at < a.at)) {
        a.v = v;
        a.at = at;
    }
}
__device__ __forceinline__ void merge(Extreme& a, int mask) {
    const float v = __shfl_xor_sync(0xffffffffu, a.v, mask);
    const int at = __shfl_xor_sync(0xffffffffu, a.at, mask);
    take(a, v, at);
}

__device__ __forceinline__ float q4_scale(float m, float* id) {
    const float d = __fdiv_rn(m, -8.0f);
    *id = d != 0.0f ? __fdiv_rn(1.0f, d) : 0.0f;
    return d;
}
__device__ __forceinline__ uint32_t q4_one(float x, float id) {
    const float r = floorf(__fadd_rn(__fmul_rn(x, id), 8.5f));
    return static_cast<uint32_t>(static_cast<int>(fminf(fmaxf(r, 0.0f), 15.0f)));
}
__device__ __forceinline__ uint32_t q8_one(float x, float id) { return static_cast<uint32_t>(quant_one(x, id) + 128); }

__device__ __forceinline__ float q8_scale(float amax, float* id) {
    const float d = __fmul_rn(amax, 1.0f / 127.0f);
    *id = d != 0.0f ? __fdiv_rn(1.0f, d) : 0.0f;
    return d;
}

// A block's scale from its reduced extreme (Q8_0: the magnitude) and its inverse.
template <bool Q4>
__device__ __forceinline__ float block_scale(const Extreme& m, float* id) {
    return Q4 ? q4_scale(m.v, id) : q8_scale(m.v, id);
}
template <bool Q4>
__device__ __forceinline__ void extreme_of(Extreme& m, float x, int at) {
    if (Q4) take(m, x, at); else m.v = fmaxf(m.v, fabsf(x));
}
template <bool Q4>
__device__ __forceinline__ void extreme_merge(Extreme& m, int mask) {
    if (Q4) merge(m, mask); else m.v = fmaxf(m.v, __shfl_xor_sync(0xffffffffu, m.v, mask));
}
template <bool Q4>
__device__ __forceinline__ uint32_t quant(float x, float id) { return Q4 ? q4_one(x, id) : q8_one(x, id); }
// quant -> value
template <bool Q4>
__device__ __forceinline__ float value(uint32_t q, float d) {
    return d * static_cast<float>(static_cast<int>(q) - (Q4 ? 8 : 128));
}

// ---- the group form: 16 rows -> one blob (or back), one 512-byte line of quants a warp and step

// K: word f of lane (g, t) holds channels of token 8 o + g.
template <bool Q4, typename T>
__device__ __forceinline__ void store_group_k(const T* src, int64_t st, uint8_t* blob, int D, int warp, int lane) {
    const int g = lane >> 2, t = lane & 3, nb = D >> 5;
    __half* const sc = reinterpret_cast<__half*>(blob + kv_quant_bytes(Q4, D));
    const int per = Q4 ? nb : D >> 4;  // words of an octet
    for (int v = warp; v < per / 2; v += kKvThreads / 32) {
        uint32_t w[4];
        if constexpr (Q4) {
            float4 x[4][2];
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const int f = 4 * v + i, o = f >= per, b = f - o * per;
                const T* const row = src + (8 * o + g) * st + 32 * b + 4 * t;
                x[i][0] = ld4(row);
                x[i][1] = ld4(row + 16);
            }
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const int f = 4 * v + i, o = f >= per, b = f - o * per;
                const float e[8] = {x[i][0].x, x[i][0].y, x[i][0].z, x[i][0].w, x[i][1].x, x[i][1].y, x[i][1].z, x[i][1].w};
                Extreme m{0.0f, 64};
#pragma unroll
                for (int c = 0; c < 8; ++c) take(m, e[c], 16 * (c >> 2) + 4 * t + (c & 3));
                merge(m, 1);
                merge(m, 2);
                float id;
                const float d = q4_scale(m.v, &id);
                w[i] = 0;
#pragma unroll
                for (int c = 0; c < 8; ++c) w[i] |= q4_one(e[c], id) << (4 * (4 * (c & 1) + 2 * (c >> 2) + ((c >> 1) & 1)));
                if (t == 0) sc[(8 * o + g) * nb + b] = __float2half_rn(d);
            }
        } else {
            const int o = 4 * v >= per, j = 4 * v - o * per;  // four words: two blocks of one token
            const T* const row = src + (8 * o + g) * st + 16 * j + 4 * t;
            float4 x[4];
#pragma unroll
            for (int i = 0; i < 4; ++i) x[i] = ld4(row + 16 * i);
#pragma unroll
            for (int b = 0; b < 2; ++b) {
                float m = 0.0f;
#pragma unroll
                for (int i = 2 * b; i < 2 * b + 2; ++i)
                    m = fmaxf(m, fmaxf(fmaxf(fabsf(x[i].x), fabsf(x[i].y)), fmaxf(fabsf(x[i].z), fabsf(x[i].w))));
                m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, 1));
                m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, 2));
                float id;
                const float d = q8_scale(m, &id);
#pragma unroll
                for (int i = 2 * b; i < 2 * b + 2; ++i)
                    w[i] = q8_one(x[i].x, id) | q8_one(x[i].y, id) << 8 | q8_one(x[i].z, id) << 16 | q8_one(x[i].w, id) << 24;
                if (t == 0) sc[(8 * o + g) * nb + (j >> 1) + b] = __float2half_rn(d);
            }
        }
        *reinterpret_cast<uint4*>(blob + (v * 32 + lane) * 16) = make_uint4(w[0], w[1], w[2], w[3]);
    }
}

// V: word f of lane (g, t) holds tokens 2t, 2t+1, 2t+8, 2t+9 of channels 8 n + g.
template <bool Q4, typename T>
__device__ __forceinline__ void store_group_v(const T* src, int64_t st, uint8_t* blob, int D, int warp, int lane) {
    const int g = lane >> 2, t = lane & 3, nb = D >> 5;
    __half* const sc = reinterpret_cast<__half*>(blob + kv_quant_bytes(Q4, D));
    constexpr int kBlocks = Q4 ? 2 : 1;  // blocks of 32 channels of a line
    for (int v = warp; v < nb / kBlocks; v += kKvThreads / 32) {
        uint32_t w[4] = {0u, 0u, 0u, 0u};
#pragma unroll
        for (int r = 0; r < 4; ++r) {  // token 8 o + 2 t + e
            const int o = r >> 1, e = r & 1, token = 8 * o + 2 * t + e;
#pragma unroll
            for (int b = 0; b < kBlocks; ++b) {
                const T* const row = src + token * st + 32 * (kBlocks * v + b) + g;
                float x[4];
                Extreme m{0.0f, 64};
#pragma unroll
                for (int n = 0; n < 4; ++n) x[n] = ld1(row + 8 * n);
#pragma unroll
                for (int n = 0; n < 4; ++n) extreme_of<Q4>(m, x[n], 8 * n + g);
                extreme_merge<Q4>(m, 4);
                extreme_merge<Q4>(m, 8);
                extreme_merge<Q4>(m, 16);
                float id;
                const float d = block_scale<Q4>(m, &id);
#pragma unroll
                for (int n = 0; n < 4; ++n) {
                    const uint32_t q = quant<Q4>(x[n], id);
                    if (Q4) w[2 * b + (n >> 1)] |= q << (4 * (4 * e + 2 * o + (n & 1)));
                    else w[n] |= q << (8 * (2 * o + e));
                }
                if (g == 0) sc[token * nb + kBlocks * v + b] = __float2half_rn(d);
            }
        }
        *reinterpret_cast<uint4*>(blob + (v * 32 + lane) * 16) = make_uint4(w[0], w[1], w[2], w[3]);
    }
}

template <bool Q4, typename T>
__device__ __forceinline__ void load_group_k(T* dst, int64_t st, const uint8_t* blob, int D, int warp, int lane) {
    const int g = lane >> 2, t = lane & 3, nb = D >> 5;
    const __half* const sc = reinterpret_cast<const __half*>(blob + kv_quant_bytes(Q4, D));
    const int per = Q4 ? nb : D >> 4;
    for (int v = warp; v < per / 2; v += kKvThreads / 32) {
        const uint4 q = *reinterpret_cast<const uint4*>(blob + (v * 32 + lane) * 16);
        const uint32_t w[4] = {q.x, q.y, q.z, q.w};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const int f = 4 * v + i, o = f >= per, j = f - o * per;
            const float d = __half2float(sc[(8 * o + g) * nb + (Q4 ? j : j >> 1)]);
            T* const row = dst + (8 * o + g) * st + (Q4 ? 32 : 16) * j + 4 * t;
            if constexpr (Q4) {
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                    const uint32_t u = w[i] >> (8 * h);  // nibbles 4 (c & 1) + (c >> 1) of this half
                    st4(row + 16 * h, make_float4(value<true>(u & 15u, d), value<true>((u >> 16) & 15u, d),
                                                  value<true>((u >> 4) & 15u, d), value<true>((u >> 20) & 15u, d)));
                }
            } else {
                st4(row, make_float4(value<false>(w[i] & 255u, d), value<false>((w[i] >> 8) & 255u, d),
                                     value<false>((w[i] >> 16) & 255u, d), value<false>(w[i] >> 24, d)));
            }
        }
    }
}

template <bool Q4, typename T>
__device__ __forceinline__ void load_group_v(T* dst, int64_t st, const uint8_t* blob, int D, int warp, int lane) {
    const int g = lane >> 2, t = lane & 3, nb = D >> 5;
    const __half* const sc = reinterpret_cast<const __half*>(blob + kv_quant_bytes(Q4, D));
    constexpr int kBlocks = Q4 ? 2 : 1;
    for (int v = warp; v < nb / kBlocks; v += kKvThreads / 32) {
        const uint4 q = *reinterpret_cast<const uint4*>(blob + (v * 32 + lane) * 16);
        const uint32_t w[4] = {q.x, q.y, q.z, q.w};
#pragma unroll
        for (int r = 0; r < 4; ++r) {
            const int o = r >> 1, e = r & 1, token = 8 * o + 2 * t + e;
#pragma unroll
            for (int b = 0; b < kBlocks; ++b) {
                const float d = __half2float(sc[token * nb + kBlocks * v + b]);
                T* const row = dst + token * st + 32 * (kBlocks * v + b) + g;
#pragma unroll
                for (int n = 0; n < 4; ++n) {
                    const uint32_t u = Q4 ? (w[2 * b + (n >> 1)] >> (4 * (4 * e + 2 * o + (n & 1)))) & 15u
                                          : (w[n] >> (8 * (2 * o + e))) & 255u;
                    st1(row + 8 * n, value<Q4>(u, d));
                }
            }
        }
    }
}

// ---- the row form: 8 lanes a block, four channels each, r the token's place in its blob

template <bool Q4, bool V, typename T>
__device__ __forceinline__ void store_row(const T* row, uint8_t* blob, int r, int D, int c) {
    // c: first of this lane's four channels; every lane of the warp takes part
    const int nb = D >> 5, l8 = (threadIdx.x & 7);
    const float4 x4 = ld4(row + c);
    const float x[4] = {x4.x, x4.y, x4.z, x4.w};
    Extreme m{0.0f, 64};
#pragma unroll
    for (int i = 0; i < 4; ++i) extreme_of<Q4>(m, x[i], 4 * l8 + i);
    extreme_merge<Q4>(m, 1);
    extreme_merge<Q4>(m, 2);
    extreme_merge<Q4>(m, 4);
    float id;
    const float d = block_scale<Q4>(m, &id);
    if (l8 == 0) reinterpret_cast<__half*>(blob + kv_quant_bytes(Q4, D))[r * nb + (c >> 5)] = __float2half_rn(d);
    uint32_t q[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) q[i] = quant<Q4>(x[i], id);
    if constexpr (!V) {
        const int o = r >> 3, lane = 4 * (r & 7) + ((c & 15) >> 2), j = c >> 4;
        if constexpr (Q4) {
            uint32_t w = (q[0] | q[1] << 16 | q[2] << 4 | q[3] << 20) << (8 * (j & 1));
            w |= __shfl_xor_sync(0xffffffffu, w, 4);
            if (!(j & 1)) *reinterpret_cast<uint32_t*>(blob + kv_word(o * nb + (j >> 1), lane)) = w;
        } else {
            *reinterpret_cast<uint32_t*>(blob + kv_word(o * (D >> 4) + j, lane)) = q[0] | q[1] << 8 | q[2] << 16 | q[3] << 24;
        }
    } else {
        const int o = r >> 3, t = (r & 7) >> 1, e = r & 1, n = c >> 3;
        if constexpr (Q4) {
            // channels d and d + 8 (n even, odd) share a byte: lanes c and c + 8
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const uint32_t other = __shfl_xor_sync(0xffffffffu, q[i], 2);
                if (!(n & 1))
                    blob[kv_word(n >> 1, 4 * ((c & 7) + i) + t) + 2 * e + o] = static_cast<uint8_t>(q[i] | other << 4);
            }
        } else {
#pragma unroll
            for (int i = 0; i < 4; ++i) blob[kv_word(n, 4 * ((c & 7) + i) + t) + 2 * o + e] = static_cast<uint8_t>(q[i]);
        }
    }
}

template <bool Q4, bool V, typename T>
__device__ __forceinline__ void load_row(T* row, const uint8_t* blob, int r, int D, int c) {
    const int nb = D >> 5;
    const float d = __half2float(reinterpret_cast<const __half*>(blob + kv_quant_bytes(Q4, D))[r * nb + (c >> 5)]);
    float x[4];
    if constexpr (!V) {
        const int o = r >> 3, lane = 4 * (r & 7) + ((c & 15) >> 2), j = c >> 4;
        const uint32_t w = *reinterpret_cast<const uint32_t*>(blob + kv_word(Q4 ? o * nb + (j >> 1) : o * (D >> 4) + j, lane));
#pragma unroll
        for (int i = 0; i < 4; ++i)
            x[i] = value<Q4>(Q4 ? (w >> (4 * (4 * (i & 1) + 2 * (j & 1) + (i >> 1)))) & 15u : (w >> (8 * i)) & 255u, d);
    } else {
        const int o = r >> 3, t = (r & 7) >> 1, e = r & 1, n = c >> 3;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const uint8_t* const w = blob + kv_word(Q4 ? n >> 1 : n, 4 * ((c & 7) + i) + t);
            x[i] = value<Q4>(Q4 ? (w[2 * e + o] >> (4 * (n & 1))) & 15u : w[2 * o + e], d);
        }
    }
    st4(row + c, make_float4(x[0], x[1], x[2], x[3]));
}

template <bool STORE, bool Q4, bool V, typename T>
__device__ __forceinline__ void kv_rows(const KvParams& p, T* rows, int64_t st, uint8_t* pool, int h, int64_t row0,
                                        const int64_t* s_slot, int start, uint32_t singles) {
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int blob = kv_blob_bytes(Q4, p.D), groups = p.page / kBlobTokens;
    const auto at = [&](int64_t slot) {
        const int64_t pg = slot / p.page, in = slot - pg * p.page;
        return pool + ((pg * p.H + h) * groups + (in >> 4)) * static_cast<int64_t>(blob);
    };
    if (start >= 0) {
        uint8_t* const b = at(s_slot[kKvRows - 1 + start]);
        T* const x = rows + (row0 + start) * st;
        if constexpr (STORE) {
            if (V) store_group_v<Q4, T>(x, st, b, p.D, warp, lane);
            else store_group_k<Q4, T>(x, st, b, p.D, warp, lane);
        } else {
            if (V) load_group_v<Q4, T>(x, st, b, p.D, warp, lane);
            else load_group_k<Q4, T>(x, st, b, p.D, warp, lane);
        }
    }
    // 32 lanes take 128 channels: one row of 128, half a row of 256, two rows of 64
    const int lanes = p.D >> 2;  // lanes a row
    const int total = __popc(singles) * lanes;
    for (int i = threadIdx.x; i < (total + 31) / 32 * 32; i += kKvThreads) {
        const bool there = i < total;
        const int k = there ? i / lanes : 0, c = there ? 4 * (i - k * lanes) : 4 * (threadIdx.x & 7);
        const int row = __fns(singles, 0, k + 1);
        const int64_t slot = s_slot[kKvRows - 1 + row];
        T* const x = rows + (row0 + row) * st;
        if constexpr (STORE) {
            // lanes past the end repeat the first row's first block, which they may write again
            store_row<Q4, V, T>(x, at(slot), static_cast<int>(slot & 15), p.D, c);
        } else if (there) {
            load_row<Q4, V, T>(x, at(slot), static_cast<int>(slot & 15), p.D, c);
        }
    }
}

// Grid: (windows of 16 rows, 2 * heads); blockIdx.y < H: keys.
template <bool STORE, typename T>
__global__ void __launch_bounds__(kKvThreads) k_kv(const __grid_constant__ KvParams p) {
    pdl_launch_dependents();
    pdl_wait();
    __shared__ int64_t s_slot[3 * kKvRows];  // rows row0 - 15 .. row0 + 30
    __shared__ int s_start;
    __shared__ uint32_t s_singles, s_zeros;
    const int tid = threadIdx.x;
    const int64_t row0 = static_cast<int64_t>(blockIdx.x) * kKvRows;
    if (tid < 3 * kKvRows) {
        const int64_t r = row0 - (kKvRows - 1) + tid;
        s_slot[tid] = r >= 0 && r < p.n ? p.slots[r] : -1;
    }
    __syncthreads();
    if (tid < 32) {
        // a group: 16 consecutive slots from a multiple of 16, inside the cache
        bool ok = tid < 2 * kKvRows - 1;
        if (ok) {
            const int64_t s = s_slot[tid];
            ok = s >= 0 && (s & 15) == 0 && s + 15 < p.n_slots;
            for (int i = 1; ok && i < 16; ++i) ok = s_slot[tid + i] == s + i;
        }
        const uint32_t starts = __ballot_sync(0xffffffffu, ok);  // bit i: one starts at row row0 - 15 + i
        bool single = false, zero = false;
        if (tid < kKvRows && row0 + tid < p.n) {
            const int64_t s = s_slot[kKvRows - 1 + tid];
            if (s >= p.n_slots) set_error(p.err, DEV_ERR_BAD_PLACE);
            zero = s < 0 || s >= p.n_slots;
            // in a group: it started at one of the 16 rows up to this one
            single = !zero && !((starts >> tid) & 0xFFFFu);
        }
        const uint32_t singles = __ballot_sync(0xffffffffu, single), zeros = __ballot_sync(0xffffffffu, zero);
        if (tid == 0) {
            const uint32_t mine = starts >> (kKvRows - 1);
            s_start = mine ? __ffs(mine) - 1 : -1;
            s_singles = singles;
            s_zeros = zeros;
        }
    }
    __syncthreads();
    const bool is_v = blockIdx.y >= static_cast<unsigned>(p.H);
    const int h = static_cast<int>(blockIdx.y) - (is_v ? p.H : 0);
    T* const rows = static_cast<T*>(const_cast<void*>(is_v ? p.vs : p.ks)) + h * (is_v ? p.v_head : p.k_head);
    const int64_t st = is_v ? p.v_token : p.k_token;
    if (is_v) {
        if (p.v.q4) kv_rows<STORE, true, true, T>(p, rows, st, p.v.p, h, row0, s_slot, s_start, s_singles);
        else kv_rows<STORE, false, true, T>(p, rows, st, p.v.p, h, row0, s_slot, s_start, s_singles);
    } else {
        if (p.k.q4) kv_rows<STORE, true, false, T>(p, rows, st, p.k.p, h, row0, s_slot, s_start, s_singles);
        else kv_rows<STORE, false, false, T>(p, rows, st, p.k.p, h, row0, s_slot, s_start, s_singles);
    }
    if constexpr (!STORE) {  // places outside the cache read as zeros
        const uint32_t zeros = s_zeros;
        const int lanes = p.D >> 2, total = __popc(zeros) * lanes;
        for (int i = tid; i < total; i += kKvThreads) {
            const int row = __fns(zeros, 0, i / lanes + 1);
            st4(rows + (row0 + row) * st + 4 * (i % lanes), make_float4(0.0f, 0.0f, 0.0f, 0.0f));
        }
    }
}

template <bool STORE>
cudaError_t launch_kv(const KvParams& p, int dtype, cudaStream_t s) {
    if (p.n == 0) return cudaSuccess;
    const dim3 grid(static_cast<unsigned>((p.n + kKvRows - 1) / kKvRows), static_cast<unsigned>(2 * p.H));
    if (dtype == 0) return launch_pdl(k_kv<STORE, float>, grid, dim3(kKvThreads), 0, s, p);
    if (dtype == 1) return launch_pdl(k_kv<STORE, __half>, grid, dim3(kKvThreads), 0, s, p);
    return launch_pdl(k_kv<STORE, __nv_bfloat16>, grid, dim3(kKvThreads), 0, s, p);
}

}  // namespace

cudaError_t launch_kv_store(const KvParams& p, int dtype, cudaStream_t s) { return launch_kv<true>(p, dtype, s); }
cudaError_t launch_kv_load(const KvParams& p, int dtype, cudaStream_t s) { return launch_kv<false>(p, dtype, s); }

}  // namespace ggq
