// ggq_attn_exact.cuh -- one row of attention over the packed cache by one warp, in fp32.
//
// The prompt kernel of 16-bit activations forms quant times scale in fp16 (keys; values of
// fp16 rows too).  Keys and values whose products may pass fp16's range count as 0 in its
// tiles, and the rows that see one are computed here instead.  Such places are rare
// (|key| > 65504 or an fp16 value at the type's very end), so this is written for the
// result, not for speed: 32 keys at a time, a lane a key for the scores, a lane a channel
// of each block of 32 for the outputs.
#pragma once
#include "ggq_attn.cuh"
#include "ggq_device.cuh"

namespace ggq {

// Largest scales (fp16 bits) whose products with every quant stay in fp16: 128 * 511.75 and
// 8 * 8188 are 65504.
template <bool Q4>
__host__ __device__ constexpr uint32_t attn_half_limit() { return Q4 ? 0x6FFFu : 0x5FFFu; }

// Whether scales may be past a limit, or not finite, given the bits of all of them OR'ed
// together: 512 and above have bits 13 and 14.  May be true of harmless ones (2 beside 1).
__device__ __forceinline__ bool attn_maybe_wide(uint32_t any) { return (any & (any << 1) & 0x40004000u) != 0u; }

// The blob of a key's group.
template <bool Q4, int D>
__device__ __forceinline__ const uint8_t* exact_blob(const AttnParams& p, const uint8_t* pool, int b, int hk, int key) {
    const int gpp = p.page >> 4, g = key >> 4;
    int pg = p.table[b * p.table_stride + g / gpp];
    if (pg < 0 || pg >= p.n_pages) pg = 0;
    return pool + ((static_cast<int64_t>(pg) * p.Hkv + hk) * gpp + g % gpp) * kv_blob_bytes(Q4, D);
}
template <bool Q4, int D>
__device__ __forceinline__ uint32_t exact_scale(const uint8_t* blob, int r, int blk) {
    return __ldg(reinterpret_cast<const uint16_t*>(blob + kv_quant_bytes(Q4, D)) + r * (D / 32) + blk);
}
// Stored quant of channel c of the token at place r of a key blob, and of a value blob.
template <bool Q4, int D>
__device__ __forceinline__ float exact_key(const uint8_t* blob, int r, int c) {
    const int o = r >> 3, j = c >> 4, i = c & 3, lane = 4 * (r & 7) + ((c & 15) >> 2);
    if constexpr (Q4) {
        const int nibble = 4 * (i & 1) + 2 * (j & 1) + (i >> 1);
        const int u = __ldg(blob + kv_word(o * (D / 32) + (j >> 1), lane) + (nibble >> 1));
        return static_cast<float>(((u >> (4 * (nibble & 1))) & 15) - 8);
    }
    return static_cast<float>(static_cast<int>(__ldg(blob + kv_word(o * (D / 16) + j, lane) + i)) - 128);
}
template <bool Q4, int D>
__device__ __forceinline__ float exact_value(const uint8_t* blob, int r, int c) {
    const int o = r >> 3, e = r & 1, n = c >> 3, lane = 4 * (c & 7) + ((r & 7) >> 1);
    if constexpr (Q4) {
        const int u = __ldg(blob + kv_word(n >> 1, lane) + 2 * e + o);
        return static_cast<float>(((u >> (4 * (n & 1))) & 15) - 8);
    }
    return static_cast<float>(static_cast<int>(__ldg(blob + kv_word(n, lane) + 2 * o + e)) - 128);
}

// A finite scale past that limit.
template <bool Q4>
__device__ __forceinline__ bool attn_wide(uint32_t bits) {
    return (bits & 0x7FFFu) > attn_half_limit<Q4>() && (bits & 0x7FFFu) < 0x7C00u;
}

// Row `token` of query head h over the keys first_key .. pos of sequence b, by a whole
// warp, if a scale of those keys is past its limit (WIDE_V: of the values too); else the
// row's output stays what it is.
template <bool K4, bool V4, int D, typename T, bool WIDE_V>
__device__ __noinline__ void attn_exact_row(const AttnParams& p, int b, int hk, int h, int64_t token, int first_key, int pos) {
    constexpr int NB = D / 32;
    const int lane = threadIdx.x & 31;
    if (first_key < 0) first_key = 0;
    bool wide = false;
    for (int key = first_key + lane; key <= pos; key += 32) {
        const uint8_t* const kb = exact_blob<K4, D>(p, p.k, b, hk, key);
        for (int blk = 0; blk < NB; ++blk) wide |= attn_wide<K4>(exact_scale<K4, D>(kb, key & 15, blk));
        if constexpr (WIDE_V) {
            const uint8_t* const vb = exact_blob<V4, D>(p, p.v, b, hk, key);
            for (int blk = 0; blk < NB; ++blk) wide |= attn_wide<V4>(exact_scale<V4, D>(vb, key & 15, blk));
        }
    }
    if (!__any_sync(0xffffffffu, wide)) return;
    const T* const q = static_cast<const T*>(p.q) + token * p.q_token + h * p.q_head;
    const float slope = p.slopes ? p.slopes[h] : 0.0f;
    float m = -INFINITY, l = 0.0f, out[NB];
#pragma unroll
    for (int i = 0; i < NB; ++i) out[i] = 0.0f;
#pragma unroll 1
    for (int k0 = first_key; k0 <= pos; k0 += 32) {
        const int key = k0 + lane;
        float s = -INFINITY;
        if (key <= pos) {
            const uint8_t* const kb = exact_blob<K4, D>(p, p.k, b, hk, key);
            s = 0.0f;
#pragma unroll 1
            for (int blk = 0; blk < NB; ++blk) {
                float dot = 0.0f;
#pragma unroll 4
                for (int i = 0; i < 32; ++i) dot = fmaf(ld1(q + 32 * blk + i), exact_key<K4, D>(kb, key & 15, 32 * blk + i), dot);
                s = fmaf(dot, half_lo(exact_scale<K4, D>(kb, key & 15, blk)), s);
            }
            s *= p.scale;
            if (p.cap > 0.0f) s = p.cap * tanhf(s / p.cap);
            if (p.slopes) s = fmaf(slope, static_cast<float>(key - pos), s);
        }
        const float top = fmaxf(m, warp_max(s));
        const float a = m == top ? 1.0f : expf(m - top), w = key <= pos ? expf(s - top) : 0.0f;
        m = top;
        l = fmaf(l, a, w);
#pragma unroll
        for (int i = 0; i < NB; ++i) out[i] *= a;
#pragma unroll 1
        for (int k = 0; k < 32 && k0 + k <= pos; ++k) {
            const float pk = __shfl_sync(0xffffffffu, w, k);
            const uint8_t* const vb = exact_blob<V4, D>(p, p.v, b, hk, k0 + k);
#pragma unroll
            for (int i = 0; i < NB; ++i)
                out[i] = fmaf(pk, half_lo(exact_scale<V4, D>(vb, (k0 + k) & 15, i)) * exact_value<V4, D>(vb, (k0 + k) & 15, 32 * i + lane), out[i]);
        }
    }
#pragma unroll
    for (int d = 16; d >= 1; d >>= 1) l += __shfl_xor_sync(0xffffffffu, l, d);
    T* const to = static_cast<T*>(p.out) + token * p.out_token + h * p.out_head;
#pragma unroll
    for (int i = 0; i < NB; ++i) st1(to + 32 * i + lane, out[i] / l);
}

}  // namespace ggq
