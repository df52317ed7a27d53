// ggq_kv.cuh -- the key/value cache's byte layout and the activation types of
// the calls around it.
//
// A blob holds 16 tokens of one kv head: the quants in the order in which an
// mma.m16n8k16 takes them as its second operand, then the fp16 scales
// [16][D/32].  For scores the operand is 16 channels x 8 keys, for the values
// 16 keys x 8 channels; lane 4 g + t of a warp holds four of its elements, so
// with the words of a lane stored four by four a warp reads 512 consecutive
// bytes at once and no transposition is left to the readers.
#pragma once
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <stdint.h>

namespace ggq {

constexpr int kBlobTokens = 16;

inline bool aligned_to(const void* p, size_t bytes) { return reinterpret_cast<uintptr_t>(p) % bytes == 0; }

__host__ __device__ constexpr int kv_quant_bytes(bool q4, int D) { return q4 ? 8 * D : 16 * D; }
__host__ __device__ constexpr int kv_blob_bytes(bool q4, int D) { return kv_quant_bytes(q4, D) + D; }

struct KvPool {
    uint8_t* p;
    int q4;        // 1: Q4_0, 0: Q8_0
};

struct KvParams {
    KvPool k, v;
    int H, D, page;
    uint32_t page_magic;         // 2^32 / (page / 16) + 1
    int heads_at_once;           // heads of a CTA
    int64_t n_slots;             // pages * page_size
    const int64_t* slots;
    int64_t n;
    const void* ks;              // keys and values outside the cache (read by the store, written by the load)
    const void* vs;
    int64_t k_token, k_head, v_token, v_head;  // strides in elements
    int* err;
};

// Four consecutive elements of a row, and one.
__device__ __forceinline__ float4 ld4(const float* p) { return *reinterpret_cast<const float4*>(p); }
__device__ __forceinline__ float4 ld4(const __half* p) {
    const uint2 u = *reinterpret_cast<const uint2*>(p);
    const float2 a = __half22float2(*reinterpret_cast<const __half2*>(&u.x));
    const float2 b = __half22float2(*reinterpret_cast<const __half2*>(&u.y));
    return make_float4(a.x, a.y, b.x, b.y);
}
__device__ __forceinline__ float4 ld4(const __nv_bfloat16* p) {
    const uint2 u = *reinterpret_cast<const uint2*>(p);
    return make_float4(__uint_as_float(u.x << 16), __uint_as_float(u.x & 0xFFFF0000u), __uint_as_float(u.y << 16),
                       __uint_as_float(u.y & 0xFFFF0000u));
}
__device__ __forceinline__ float ld1(const float* p) { return *p; }
__device__ __forceinline__ float ld1(const __half* p) { return __half2float(*p); }
__device__ __forceinline__ float ld1(const __nv_bfloat16* p) { return __bfloat162float(*p); }
__device__ __forceinline__ void st1(float* p, float v) { *p = v; }
__device__ __forceinline__ void st1(__half* p, float v) { *p = __float2half_rn(v); }
__device__ __forceinline__ void st1(__nv_bfloat16* p, float v) { *p = __float2bfloat16_rn(v); }
__device__ __forceinline__ void st4(float* p, float4 v) { *reinterpret_cast<float4*>(p) = v; }
__device__ __forceinline__ void st4(__half* p, float4 v) {
    const __half2 a = __floats2half2_rn(v.x, v.y), b = __floats2half2_rn(v.z, v.w);
    *reinterpret_cast<uint2*>(p) = make_uint2(*reinterpret_cast<const uint32_t*>(&a), *reinterpret_cast<const uint32_t*>(&b));
}
__device__ __forceinline__ void st4(__nv_bfloat16* p, float4 v) {
    const __nv_bfloat162 a = __floats2bfloat162_rn(v.x, v.y), b = __floats2bfloat162_rn(v.z, v.w);
    *reinterpret_cast<uint2*>(p) = make_uint2(*reinterpret_cast<const uint32_t*>(&a), *reinterpret_cast<const uint32_t*>(&b));
}

// Eight consecutive elements of a row (16-bit ones: 16 aligned bytes).
__device__ __forceinline__ void ld8(const float* p, float (&x)[8]) {
    const float4 a = reinterpret_cast<const float4*>(p)[0], b = reinterpret_cast<const float4*>(p)[1];
    x[0] = a.x, x[1] = a.y, x[2] = a.z, x[3] = a.w, x[4] = b.x, x[5] = b.y, x[6] = b.z, x[7] = b.w;
}
__device__ __forceinline__ void ld8(const __half* p, float (&x)[8]) {
    const uint4 u = *reinterpret_cast<const uint4*>(p);
    const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&w[i]));
        x[2 * i] = f.x, x[2 * i + 1] = f.y;
    }
}
__device__ __forceinline__ void ld8(const __nv_bfloat16* p, float (&x)[8]) {
    const uint4 u = *reinterpret_cast<const uint4*>(p);
    const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) x[2 * i] = __uint_as_float(w[i] << 16), x[2 * i + 1] = __uint_as_float(w[i] & 0xFFFF0000u);
}
__device__ __forceinline__ void st8(float* p, const float (&x)[8]) {
    st4(p, make_float4(x[0], x[1], x[2], x[3]));
    st4(p + 4, make_float4(x[4], x[5], x[6], x[7]));
}
template <typename T2, typename F>
__device__ __forceinline__ void st8_pairs(void* p, const float (&x)[8], F pack) {
    uint32_t w[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const T2 h = pack(x[2 * i], x[2 * i + 1]);
        w[i] = *reinterpret_cast<const uint32_t*>(&h);
    }
    *static_cast<uint4*>(p) = make_uint4(w[0], w[1], w[2], w[3]);
}
__device__ __forceinline__ void st8(__half* p, const float (&x)[8]) {
    st8_pairs<__half2>(p, x, [](float a, float b) { return __floats2half2_rn(a, b); });
}
__device__ __forceinline__ void st8(__nv_bfloat16* p, const float (&x)[8]) {
    st8_pairs<__nv_bfloat162>(p, x, [](float a, float b) { return __floats2bfloat162_rn(a, b); });
}

// Byte offset of word f of lane l in a blob's quants.
__device__ __forceinline__ int kv_word(int f, int l) { return ((f >> 2) * 32 + l) * 16 + (f & 3) * 4; }

cudaError_t launch_kv_store(const KvParams& p, int dtype, cudaStream_t s);
cudaError_t launch_kv_load(const KvParams& p, int dtype, cudaStream_t s);

}  // namespace ggq
