// ggq_attn_prompt.cuh -- attention of many query rows (prompts) over the packed
// cache on tcgen05, for 16-bit activations.
//
// Mathematics: S = Q K^T and O = P V per kv head, the rows being the head
// group's query heads of consecutive tokens, with the softmax's running maximum
// and sum.  4 D operations per (row, key); the packed cache is a small part.  Measured:
// the last 4096 of 8192 causal bf16 rows, 32 heads on 8 of 128 channels: 427 us, 966
// TFLOP/s, half the rate of a plain 16-bit product; the tensor pipe is busy 39% of the
// time, the issue slots 65%: bound by the instructions of the softmax and of unpacking
// the blobs (done once for 256 rows) and the waits between them.
//
// A CTA takes one kv head of one sequence and one or two tiles of 128 rows that
// share its steps of keys (heads of 256 channels: one tile, whose O fills half of
// tensor memory).  Roles:
//   * warps 0-3 and 4-7: the softmax of a tile, one thread a row.  Scores come
//     from tensor memory; probabilities go back over them as the first operand of
//     P V (tensor memory holds it, so only V is read from shared memory), in the
//     channels' key order of the V tile;
//   * warps 8-15: the packed blobs, read straight from the cache, to fp16 (V with
//     bf16 activations: bf16) tiles in the K-major 128-byte-swizzled layout, two
//     buffers each for K and V;
//   * warps 16, 17 and 18, 19: one thread each issues a tile's S = Q K^T and O +=
//     P V, 64 keys a turn; two score buffers a tile let the next turn's scores be
//     computed while the softmax works on this one's.
// The running maximum is raised (and O rescaled in tensor memory) only when a row
// passes it by 2^8.  fp16 queries are exact; bf16 ones too (rows are scaled by a
// power of two).  K is rounded to fp16 (2^-11 of each value at most); V and P to the
// activations' type: with bf16 2^-8 of each at most, as much as the output's own rounding,
// but no probability is lost for being small (fp16 would lose those below 2^-31 of the
// largest, which are all of an output whose channel the large ones leave at 0) and no value
// for being large; with fp16 2^-11, P being kept at 2^7 times its value.  Each row's sum is fp32.  Keys, and values of fp16
// rows, that leave fp16's range count as 0 here, and the rows that see them are computed
// again in fp32 (ggq_attn_exact.cuh).
#pragma once
#include <atomic>
#include <type_traits>

#include "ggq_attn.cuh"
#include "ggq_attn_exact.cuh"
#include "ggq_device.cuh"
#include "ggq_internal.h"
#include "ggq_tcgen05.cuh"

namespace ggq {

constexpr int kSoftmaxWarps = 8, kDecodeWarps = 8, kMmaWarps = 4;
constexpr int kFirstMma = kSoftmaxWarps + kDecodeWarps;
constexpr int kPromptThreads = (kSoftmaxWarps + kDecodeWarps + kMmaWarps) * 32;

// Registers a thread: 640 threads launch with 96 each; the decoding and MMA warps
// give some back (setmaxnreg.dec, never above 96), the softmax warps take them.
constexpr int kLaunchRegs = 96, kSoftmaxRegs = 128, kDecodeRegs = 88, kMmaRegs = 48;
static_assert(kSoftmaxRegs >= kLaunchRegs && kDecodeRegs <= kLaunchRegs && kMmaRegs <= kLaunchRegs &&
                  kSoftmaxRegs % 8 == 0 && kDecodeRegs % 8 == 0 && kMmaRegs % 8 == 0 &&
                  32 * (kSoftmaxWarps * kSoftmaxRegs + kDecodeWarps * kDecodeRegs + kMmaWarps * kMmaRegs) <=
                      kPromptThreads * kLaunchRegs &&
                  kPromptThreads * kLaunchRegs <= 65536,
              "register split");

template <int D>
struct PromptShape {
    static constexpr int kTiles = D <= 128 ? 2 : 1;
    static constexpr int kKeys = D <= 128 ? 128 : 64;  // of a step
    static constexpr int kRows = 128 * kTiles;
    static constexpr int kQ = 128 * D * 2;             // bytes of a tile's queries
    static constexpr int kK = kKeys * D * 2, kV = kK;  // bytes of a step's keys, values
    static constexpr int oK = kTiles * kQ, oV = oK + 2 * kK, oBar = oV + 2 * kV;
    static constexpr int oScale = oBar + 384;          // of the rows
    static constexpr int kTotal = oScale + kRows * 4 + 1024;  // + alignment of the tiles
    // tensor-memory columns: two 64-key score buffers of each tile (probabilities over
    // them), then the outputs
    static constexpr uint32_t cS = 128, cO = kTiles * cS;
    static_assert(cO + kTiles * D <= 512, "tensor memory");
};

__host__ __device__ constexpr uint32_t prompt_idesc(uint32_t n, bool bf16) {
    return (1u << 4) | (bf16 ? (1u << 7) | (1u << 10) : 0u) | ((n >> 3) << 17) | (8u << 24);
}
// D[tensor memory] (+)= A[tensor memory] * B[shared memory]
__device__ __forceinline__ void tc_mma_ts(uint32_t d, uint32_t a, uint64_t b, uint32_t idesc, uint32_t accumulate) {
    asm volatile(
        "{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %4, 0;\n\t"
        "tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n\t}" ::"r"(d),
        "r"(a), "l"(b), "r"(idesc), "r"(accumulate)
        : "memory");
}
// 32 columns, to be used after prompt_wait_ld on the same registers
__device__ __forceinline__ void prompt_ld32(uint32_t taddr, float* v) {
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x32.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,"
        "%16,%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31}, [%32];"
        : "=f"(v[0]), "=f"(v[1]), "=f"(v[2]), "=f"(v[3]), "=f"(v[4]), "=f"(v[5]), "=f"(v[6]), "=f"(v[7]), "=f"(v[8]),
          "=f"(v[9]), "=f"(v[10]), "=f"(v[11]), "=f"(v[12]), "=f"(v[13]), "=f"(v[14]), "=f"(v[15]), "=f"(v[16]),
          "=f"(v[17]), "=f"(v[18]), "=f"(v[19]), "=f"(v[20]), "=f"(v[21]), "=f"(v[22]), "=f"(v[23]), "=f"(v[24]),
          "=f"(v[25]), "=f"(v[26]), "=f"(v[27]), "=f"(v[28]), "=f"(v[29]), "=f"(v[30]), "=f"(v[31])
        : "r"(taddr));
}
__device__ __forceinline__ void prompt_ld16(uint32_t taddr, float (&v)[16]) {
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x16.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15}, [%16];\n\t"
        "tcgen05.wait::ld.sync.aligned;"
        : "=f"(v[0]), "=f"(v[1]), "=f"(v[2]), "=f"(v[3]), "=f"(v[4]), "=f"(v[5]), "=f"(v[6]), "=f"(v[7]), "=f"(v[8]),
          "=f"(v[9]), "=f"(v[10]), "=f"(v[11]), "=f"(v[12]), "=f"(v[13]), "=f"(v[14]), "=f"(v[15])
        : "r"(taddr)
        : "memory");
}
__device__ __forceinline__ void prompt_st16(uint32_t taddr, const float (&v)[16]) {
    asm volatile(
        "tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16};\n\t"
        "tcgen05.wait::st.sync.aligned;" ::"r"(taddr),
        "f"(v[0]), "f"(v[1]), "f"(v[2]), "f"(v[3]), "f"(v[4]), "f"(v[5]), "f"(v[6]), "f"(v[7]), "f"(v[8]), "f"(v[9]),
        "f"(v[10]), "f"(v[11]), "f"(v[12]), "f"(v[13]), "f"(v[14]), "f"(v[15])
        : "memory");
}
__device__ __forceinline__ void prompt_wait_ld() { asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory"); }
// keeps uses of v behind the wait
__device__ __forceinline__ void prompt_tie32(float* v) {
    asm volatile(""
                 : "+f"(v[0]), "+f"(v[1]), "+f"(v[2]), "+f"(v[3]), "+f"(v[4]), "+f"(v[5]), "+f"(v[6]), "+f"(v[7]),
                   "+f"(v[8]), "+f"(v[9]), "+f"(v[10]), "+f"(v[11]), "+f"(v[12]), "+f"(v[13]), "+f"(v[14]), "+f"(v[15]),
                   "+f"(v[16]), "+f"(v[17]), "+f"(v[18]), "+f"(v[19]), "+f"(v[20]), "+f"(v[21]), "+f"(v[22]),
                   "+f"(v[23]), "+f"(v[24]), "+f"(v[25]), "+f"(v[26]), "+f"(v[27]), "+f"(v[28]), "+f"(v[29]),
                   "+f"(v[30]), "+f"(v[31]));
}
__device__ __forceinline__ void prompt_st32(uint32_t taddr, const uint32_t (&v)[32]) {
    asm volatile(
        "tcgen05.st.sync.aligned.32x32b.x32.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16,"
        "%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31,%32};" ::"r"(taddr),
        "r"(v[0]), "r"(v[1]), "r"(v[2]), "r"(v[3]), "r"(v[4]), "r"(v[5]), "r"(v[6]), "r"(v[7]), "r"(v[8]), "r"(v[9]),
        "r"(v[10]), "r"(v[11]), "r"(v[12]), "r"(v[13]), "r"(v[14]), "r"(v[15]), "r"(v[16]), "r"(v[17]), "r"(v[18]),
        "r"(v[19]), "r"(v[20]), "r"(v[21]), "r"(v[22]), "r"(v[23]), "r"(v[24]), "r"(v[25]), "r"(v[26]), "r"(v[27]),
        "r"(v[28]), "r"(v[29]), "r"(v[30]), "r"(v[31])
        : "memory");
}
// packed fp32: (a0, a1) * b + (c0, c1), (a0, a1) + (b0, b1), (a0, a1) * (b0, b1)
__device__ __forceinline__ void add2(float& d0, float& d1, float a0, float a1, float b0, float b1) {
    asm("{\n\t.reg .b64 x, y;\n\tmov.b64 x, {%2, %3};\n\tmov.b64 y, {%4, %5};\n\tadd.rn.f32x2 x, x, y;\n\t"
        "mov.b64 {%0, %1}, x;\n\t}"
        : "=f"(d0), "=f"(d1)
        : "f"(a0), "f"(a1), "f"(b0), "f"(b1));
}
__device__ __forceinline__ void mul2(float& d0, float& d1, float a0, float a1, float b0, float b1) {
    asm("{\n\t.reg .b64 x, y;\n\tmov.b64 x, {%2, %3};\n\tmov.b64 y, {%4, %5};\n\tmul.rn.f32x2 x, x, y;\n\t"
        "mov.b64 {%0, %1}, x;\n\t}"
        : "=f"(d0), "=f"(d1)
        : "f"(a0), "f"(a1), "f"(b0), "f"(b1));
}
__device__ __forceinline__ void tmem_wait_st() { asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory"); }

__device__ __forceinline__ float prompt_ex2(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}
template <bool BF>
__device__ __forceinline__ uint32_t prompt_pack(float lo, float hi) {
    uint32_t r;
    if (BF) asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
    else asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
    return r;
}
__device__ __forceinline__ uint32_t prompt_sub2(uint32_t a, uint32_t b) {
    const __half2 r = __hsub2(*reinterpret_cast<const __half2*>(&a), *reinterpret_cast<const __half2*>(&b));
    return *reinterpret_cast<const uint32_t*>(&r);
}
__device__ __forceinline__ uint32_t prompt_mul2(uint32_t a, uint32_t b) {
    const __half2 r = __hmul2(*reinterpret_cast<const __half2*>(&a), *reinterpret_cast<const __half2*>(&b));
    return *reinterpret_cast<const uint32_t*>(&r);
}
__device__ __forceinline__ uint32_t prompt_fma2(uint32_t a, uint32_t b, uint32_t c) {
    const __half2 r = __hfma2(*reinterpret_cast<const __half2*>(&a), *reinterpret_cast<const __half2*>(&b),
                              *reinterpret_cast<const __half2*>(&c));
    return *reinterpret_cast<const uint32_t*>(&r);
}
// Quants of a word as pairs of exact fp16 integers: bytes (0, 1) and (2, 3); nibbles
// (0, 4), (1, 5), (2, 6), (3, 7).
__device__ __forceinline__ void prompt_ints8(uint32_t w, uint32_t (&h)[2]) {
    h[0] = prompt_sub2(prmt(w, 0x64646464u, 0x4140u), 0x64806480u);
    h[1] = prompt_sub2(prmt(w, 0x64646464u, 0x4342u), 0x64806480u);
}
__device__ __forceinline__ void prompt_ints4(uint32_t w, uint32_t (&h)[4]) {
    const uint32_t y = w >> 8;
    h[0] = prompt_sub2((w & 0x000F000Fu) | 0x64006400u, 0x64086408u);                          // 1024 + q - 1032
    h[1] = prompt_fma2((w & 0x00F000F0u) | 0x64006400u, 0x2C002C00u, 0xD480D480u);             // (1024 + 16 q) / 16 - 72
    h[2] = prompt_sub2((y & 0x000F000Fu) | 0x64006400u, 0x64086408u);
    h[3] = prompt_fma2((y & 0x00F000F0u) | 0x64006400u, 0x2C002C00u, 0xD480D480u);
}

// The two key pairs of a V word (bytes 0, 1 and 2, 3) times the keys' scales, in
// the operand's type (bf16: one rounding of the fp32 product, whose integer comes
// out of 2^23 + u).
template <bool BF>
__device__ __forceinline__ void prompt_v8(uint32_t w, const float (&df)[4], uint32_t d01, uint32_t d23, uint32_t (&o)[2]) {
    if constexpr (BF) {
        float x[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) x[i] = __uint_as_float(prmt(w, 0x4B000000u, 0x7440u + i));
#pragma unroll
        for (int i = 0; i < 4; i += 2) {
            add2(x[i], x[i + 1], x[i], x[i + 1], -8388736.0f, -8388736.0f);
            mul2(x[i], x[i + 1], x[i], x[i + 1], df[i], df[i + 1]);
            o[i >> 1] = prompt_pack<true>(x[i], x[i + 1]);
        }
    } else {
        uint32_t h[2];
        prompt_ints8(w, h);
        o[0] = prompt_mul2(h[0], d01), o[1] = prompt_mul2(h[1], d23);
    }
}
template <bool BF>
__device__ __forceinline__ uint32_t prompt_v4(uint32_t h, float d0, float d1, uint32_t d2) {
    if constexpr (BF) {
        const float2 a = __half22float2(*reinterpret_cast<const __half2*>(&h));
        float x, y;
        mul2(x, y, a.x, a.y, d0, d1);
        return prompt_pack<true>(x, y);
    }
    return prompt_mul2(h, d2);
}

// Whether a value scale of block blk is not finite among the keys first_key .. pos.  The
// tile kernels keep the first and last such key that they meet; a row whose window lies
// between the two looks for itself.
template <bool V4, int D>
__device__ __noinline__ bool prompt_bad_value(const AttnParams& p, int b, int hk, int blk, int first_key, int pos) {
    const int gpp = p.page >> 4;
    const uint16_t* scales = nullptr;
    for (int key = first_key; key <= pos; ++key) {
        if (scales == nullptr || (key & 15) == 0) {
            const int g = key >> 4;
            int pg = p.table[b * p.table_stride + g / gpp];
            if (pg < 0 || pg >= p.n_pages) pg = 0;
            const int64_t at = (static_cast<int64_t>(pg) * p.Hkv + hk) * gpp + g % gpp;
            scales = reinterpret_cast<const uint16_t*>(p.v + at * kv_blob_bytes(V4, D) + kv_quant_bytes(V4, D)) + blk;
        }
        if ((__ldg(scales + (key & 15) * (D / 32)) & 0x7C00u) == 0x7C00u) return true;
    }
    return false;
}
// A row sees a value scale of block blk that is not finite; s_bad: the first and last key of those.
template <bool V4, int D>
__device__ __forceinline__ bool prompt_spoilt(const AttnParams& p, const int* s_bad, int b, int hk, int blk, int first_key, int pos) {
    const int lo = s_bad[2 * blk], hi = s_bad[2 * blk + 1];
    if (lo > pos || hi < first_key || hi < 0) return false;
    if (lo >= first_key || hi <= pos) return true;
    return prompt_bad_value<V4, D>(p, b, hk, blk, first_key, pos);
}

template <bool REGS_UP, int N>
__device__ __forceinline__ void prompt_regs() {
    if (REGS_UP) asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(N));
    else asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(N));
}

template <bool K4, bool V4, int D, bool BF>
__global__ void __launch_bounds__(kPromptThreads, 1) k_attn_prompt(const __grid_constant__ AttnParams p) {
    using SH = PromptShape<D>;
    constexpr int TILES = SH::kTiles, KT = SH::kKeys, NB = D / 32, KG = KT / 16;
    extern __shared__ __align__(1024) uint8_t smem_raw[];
    uint8_t* const smem = smem_raw + ((1024 - (smem_addr(smem_raw) & 1023)) & 1023);
    const int tid = threadIdx.x, warp = __shfl_sync(0xffffffffu, tid >> 5, 0), lane = tid & 31;  // warp: uniform
    uint64_t* const bars = reinterpret_cast<uint64_t*>(smem + SH::oBar);
    uint64_t *const kfull = bars, *const kempty = bars + 2, *const vfull = bars + 4, *const vempty = bars + 6;
    // per tile and score buffer: scores there, probabilities there, P V done; per MMA thread: all done
    uint64_t *const sfull = bars + 8, *const pfull = bars + 12, *const pdone = bars + 16, *const done = bars + 20;
    uint32_t* const tslot = reinterpret_cast<uint32_t*>(bars + 24);
    volatile int* const abort = reinterpret_cast<volatile int*>(tslot + 1);
    int* const s_bad = reinterpret_cast<int*>(tslot + 2);  // [NB][2] first and last key whose value scale is not finite
    int* const s_wide = s_bad + 2 * NB;                    // first and last key that fp16 tiles cannot hold
    int* const s_odd = s_wide + 2;                         // 1: there is one of either kind

    pdl_launch_dependents();
    pdl_wait();
    // ---- the item: heaviest (last) rows first
    const int b = static_cast<int>(blockIdx.x / static_cast<unsigned>(p.Hkv));
    const int hk = static_cast<int>(blockIdx.x) - b * p.Hkv;
    const int tile = static_cast<int>(gridDim.y - 1 - blockIdx.y);
    int len = p.lens[b], first = b, end = b + 1;
    if (p.q_start) first = p.q_start[b], end = p.q_start[b + 1];
    bool bad = false;
    if (first < 0 || end > p.n_tokens || first > end) first = end = 0, bad = true;
    const int n = end - first, shown = min(n, p.max_q);
    if (n > p.max_q) bad = true;
    if (len < 0 || len > p.max_len) len = len < 0 ? 0 : p.max_len, bad = true;
    if (bad && tid == 0) set_error(p.err, DEV_ERR_BAD_PLACE);
    const int R = shown * p.G, r_begin = tile * SH::kRows;
    if (r_begin >= R) return;
    const int r_end = min(R, r_begin + SH::kRows);
    const int from = len - n;  // position of the first row
    const int ntiles = r_end - r_begin > 128 ? TILES : 1;
    const int pos_last = from + (r_end - 1) / p.G, pos_first = from + r_begin / p.G;
    const int glo = p.window > 0 && pos_first - p.window + 1 > 0 ? (pos_first - p.window + 1) >> 4 : 0;
    const int ghi = pos_last < 0 ? glo : (pos_last >> 4) + 1;
    const int steps = ghi > glo ? (ghi - glo + KG - 1) / KG : 0;   // K and V tiles
    const int turns = ghi > glo ? (ghi - glo + 3) / 4 : 0;         // of 64 keys
    constexpr int kTurns = KT / 64;                                // of a step

    if (tid == 0) {
        for (int i = 0; i < 2; ++i) {
            mbar_init(kfull + i, kDecodeWarps * 32);
            mbar_init(vfull + i, kDecodeWarps * 32);
            mbar_init(kempty + i, static_cast<uint32_t>(ntiles));
            mbar_init(vempty + i, static_cast<uint32_t>(ntiles));
        }
        for (int i = 0; i < 4; ++i) {
            mbar_init(sfull + i, 1);
            mbar_init(pfull + i, 128);
            mbar_init(pdone + i, 1);
            mbar_init(done + i, 1);
        }
        *abort = *s_odd = 0;
        for (int i = 0; i <= NB; ++i) s_bad[2 * i] = 0x7fffffff, s_bad[2 * i + 1] = -1;  // and s_wide
        fence_barrier_init();
    }
    if (warp == kFirstMma) {
        asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_addr(tslot)), "r"(512u)
                     : "memory");
        asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
    }
    // ---- queries: whole rows at a time, 8 channels a lane, as fp16 with the row's largest element in [2^13, 2^14)
    float* const s_scale = reinterpret_cast<float*>(smem + SH::oScale);
    if (warp < 4 * TILES && (warp >> 2) < ntiles) {
        constexpr int LR = D / 8, RL = 32 / LR;  // lanes of a row, rows of a load
        const int d = 8 * (lane % LR);
        // the K tile's channel order: 16 t + 4 j + i holds 16 j + 4 t + i of 64
        uint8_t* const to = smem + (warp >> 2) * SH::kQ + (d >> 6) * (128 * 128) + 8 * ((d >> 4) & 1);
        const int chunk = 2 * ((d >> 2) & 3) + ((d >> 5) & 1);
#pragma unroll 1
        for (int k0 = 0; k0 < 32; k0 += 8 * RL) {
            float4 x[8][2];
#pragma unroll
            for (int k = 0; k < 8; ++k) {
                const int r = min(r_begin + 32 * warp + k0 + k * RL + lane / LR, r_end - 1), i = r / p.G;
                const int64_t at = (first + i) * p.q_token + (hk * p.G + r - i * p.G) * p.q_head + d;
#pragma unroll
                for (int z = 0; z < 2; ++z)
                    x[k][z] = BF ? ld4(static_cast<const __nv_bfloat16*>(p.q) + at + 4 * z)
                                 : ld4(static_cast<const __half*>(p.q) + at + 4 * z);
            }
#pragma unroll
            for (int k = 0; k < 8; ++k) {
                const int row = 32 * warp + k0 + k * RL + lane / LR, rr = row & 127;
                float amax = 0.0f;
#pragma unroll
                for (int z = 0; z < 2; ++z)
                    amax = fmaxf(amax, fmaxf(fmaxf(fabsf(x[k][z].x), fabsf(x[k][z].y)), fmaxf(fabsf(x[k][z].z), fabsf(x[k][z].w))));
#pragma unroll
                for (int m = 1; m < LR; m <<= 1) amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, m));
                const int ex = static_cast<int>(__float_as_uint(amax) >> 23) - 127;
                const int sh = ex == 128 ? 0 : min(13 - ex, 100);
                const float up = copysignf(__uint_as_float(static_cast<uint32_t>(sh + 127) << 23), p.scale);
#pragma unroll
                for (int z = 0; z < 2; ++z)
                    *reinterpret_cast<uint2*>(to + rr * 128 + (((chunk + 2 * z) ^ (rr & 7)) << 4)) =
                        make_uint2(prompt_pack<false>(x[k][z].x * up, x[k][z].y * up), prompt_pack<false>(x[k][z].z * up, x[k][z].w * up));
                // not negative: the largest product is the largest logit
                if (lane % LR == 0) s_scale[row] = fabsf(p.scale) * scalbnf(1.0f, -sh);
            }
        }
        fence_proxy_async_smem();
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = __shfl_sync(0xffffffffu, *tslot, 0);

    const auto wait1 = [&](uint64_t* bar, uint32_t parity) {
        const bool ok = !*abort && mbar_wait(bar, parity);
        if (!ok) {
            *abort = 1;
            set_error(p.err, DEV_ERR_TIMEOUT);
        }
        return ok;
    };
    const auto wait = [&](uint64_t* bar, uint32_t parity) {
        bool ok = !*abort && mbar_wait(bar, parity);
        ok = __all_sync(0xffffffffu, ok);
        if (!ok) {
            *abort = 1;
            set_error(p.err, DEV_ERR_TIMEOUT);
        }
        return ok;
    };

    if (warp >= kFirstMma) {
        // ================================================================ MMA: one thread a tile
        prompt_regs<false, kMmaRegs>();
        const int t = (warp - kFirstMma) & 1;
        const bool scores = warp < kFirstMma + 2;
        if (t < ntiles && elect_one() && turns > 0) {
            const uint32_t cs = tmem + t * SH::cS, co = tmem + SH::cO + t * D;
            if (scores) {
                const uint64_t qd = umma_desc_sw128(smem_addr(smem + t * SH::kQ));
                constexpr uint32_t id = prompt_idesc(64, false);
                for (int i = 0; i < turns; ++i) {
                    const int j = i / kTurns, h = i % kTurns, buf = j & 1, sb = i & 1;
                    if (h == 0 && !wait1(kfull + buf, (j >> 1) & 1)) break;
                    if (i >= 2 && !wait1(pdone + 2 * t + sb, ((i >> 1) - 1) & 1)) break;
                    tc_fence_after();
                    const uint64_t kd = umma_desc_sw128(smem_addr(smem + SH::oK + buf * SH::kK + h * (64 * 128)));
#pragma unroll
                    for (int k = 0; k < D / 16; ++k)  // 32 bytes a step inside a 64-channel atom
                        tc_mma(cs + 64 * sb, qd + (k >> 2) * (128 * 128 / 16) + 2 * (k & 3),
                               kd + (k >> 2) * (KT * 128 / 16) + 2 * (k & 3), id, k > 0);
                    tc_commit(sfull + 2 * t + sb);
                    if (h == kTurns - 1) tc_commit(kempty + buf);
                }
            } else {
                constexpr uint32_t id = prompt_idesc(D, BF);
                for (int i = 0; i < turns; ++i) {
                    const int j = i / kTurns, h = i % kTurns, buf = j & 1, sb = i & 1;
                    if (h == 0 && !wait1(vfull + buf, (j >> 1) & 1)) break;
                    if (!wait1(pfull + 2 * t + sb, (i >> 1) & 1)) break;
                    tc_fence_after();
                    const uint64_t vd = umma_desc_sw128(smem_addr(smem + SH::oV + buf * SH::kV + h * (D * 128)));
#pragma unroll
                    for (int k = 0; k < 4; ++k)
                        tc_mma_ts(co, cs + 64 * sb + 8 * k, vd + 2 * k, id, (i > 0 || k > 0) ? 1u : 0u);
                    tc_commit(pdone + 2 * t + sb);
                    if (h == kTurns - 1) tc_commit(vempty + buf);
                }
            }
            tc_commit(done + warp - kFirstMma);
            mbar_wait(done + warp - kFirstMma, 0);  // every MMA has ended before tensor memory goes
        }
    } else if (warp >= kSoftmaxWarps) {
        // ================================================================ packed blobs -> operand tiles
        prompt_regs<false, kDecodeRegs>();
        const int cw = warp - kSoftmaxWarps, g8 = lane >> 2, t4 = lane & 3, gpp = p.page >> 4;
        constexpr int kKB = kv_blob_bytes(K4, D), kVB = kv_blob_bytes(V4, D);
        // keys: a warp takes one group of the step (64-key steps: one octet of it)
        constexpr int KP = kDecodeWarps / KG, KO = 2 / KP;        // parts of a group, octets of a part
        constexpr int KL = (K4 ? D / 64 : D / 32) / KP;           // 16-byte words of a lane
        const int k_group = cw % KG, k_part = cw / KG;
        // values: two neighbouring groups, some of the blocks of 32 channels
        constexpr int VP = KG / 2, VB = NB / (kDecodeWarps / VP); // pairs of groups; blocks of a warp: 1 or 2
        const int pair = cw % VP, b0 = (cw / VP) * VB;
        const uint32_t v_sel = (VB == 1 && (b0 & 1)) ? 0x7632u : 0x5410u;
        // blobs of the step's groups, one a lane
        const auto locate = [&](int j) {
            const int g = glo + j * KG + (lane & (KG - 1));
            int64_t at = -1;
            if (j < steps && g < ghi) {
                int pg = p.table[b * p.table_stride + g / gpp];
                if (pg < 0 || pg >= p.n_pages) {
                    set_error(p.err, DEV_ERR_BAD_PLACE);
                    pg = 0;
                }
                at = (static_cast<int64_t>(pg) * p.Hkv + hk) * gpp + g % gpp;
            }
            return at;
        };
        uint4 kq[KL];
        uint32_t ks[KO][NB / 2];
        uint4 vq[2][VB];          // a block: four words of bytes, or two of nibbles
        uint32_t vsc[2][4];       // scales of the four keys of a word, blocks b0 and b0 + 1
        const auto load_k = [&](int64_t blobs) {
            const int64_t at = __shfl_sync(0xffffffffu, blobs, k_group);
            if (at < 0) return;  // past the last key: the tile keeps what it held, every row masks it
            const uint8_t* const src = p.k + at * kKB;
#pragma unroll
            for (int i = 0; i < KL; ++i)
                kq[i] = __ldg(reinterpret_cast<const uint4*>(src + ((k_part * KL + i) * 32 + lane) * 16));
#pragma unroll
            for (int o = 0; o < KO; ++o)
#pragma unroll
                for (int i = 0; i < NB / 2; ++i)
                    ks[o][i] = __ldg(reinterpret_cast<const uint32_t*>(src + kv_quant_bytes(K4, D) +
                                                                       (8 * (k_part + o) + g8) * NB * 2) + i);
        };
        const auto load_v = [&](int64_t blobs) {
#pragma unroll
            for (int c = 0; c < 2; ++c) {
                const int64_t at = __shfl_sync(0xffffffffu, blobs, 2 * pair + c);
                if (at < 0) {
#pragma unroll
                    for (int i = 0; i < VB; ++i) vq[c][i] = make_uint4(0u, 0u, 0u, 0u);
#pragma unroll
                    for (int r = 0; r < 4; ++r) vsc[c][r] = 0u;
                    continue;
                }
                const uint8_t* const src = p.v + at * kVB;
#pragma unroll
                for (int i = 0; i < VB; ++i) {
                    const int blk = b0 + i;
                    if constexpr (V4) {
                        const uint2 u = __ldg(reinterpret_cast<const uint2*>(src + ((blk >> 1) * 32 + lane) * 16 + (blk & 1) * 8));
                        vq[c][i].x = u.x, vq[c][i].y = u.y;
                    } else {
                        vq[c][i] = __ldg(reinterpret_cast<const uint4*>(src + (blk * 32 + lane) * 16));
                    }
                }
#pragma unroll
                for (int r = 0; r < 4; ++r)
                    vsc[c][r] = __ldg(reinterpret_cast<const uint32_t*>(src + kv_quant_bytes(V4, D) +
                                                                        (8 * (r >> 1) + 2 * t4 + (r & 1)) * NB * 2) + (b0 >> 1));
            }
        };
        int64_t blobs = locate(0), next = locate(1);
        if (steps > 0) {
            load_k(blobs);
            load_v(blobs);
        }
        for (int j = 0; j < steps; ++j) {
            const int buf = j & 1;
            blobs = next;
            next = locate(j + 2);
            // ---- keys: lane (g, t) writes 16 channels of a 64-channel atom as two chunks of its token's row
            if (j >= 2 && !wait(kempty + buf, ((j >> 1) - 1) & 1)) break;
            uint8_t* const kt = smem + SH::oK + buf * SH::kK + (k_group * 16 + 8 * k_part + g8) * 128;
            uint32_t any = 0u;
#pragma unroll
            for (int o = 0; o < KO; ++o)
#pragma unroll
                for (int q = 0; q < NB / 2; ++q) any |= ks[o][q];
            if (attn_maybe_wide(any)) {
                // scales whose products leave fp16: 0 here, and the rows that see them are told
#pragma unroll
                for (int o = 0; o < KO; ++o)
#pragma unroll
                    for (int q = 0; q < NB / 2; ++q) {
                        const int key = 16 * (glo + j * KG + k_group) + 8 * (k_part + o) + g8;
                        const bool lo = attn_wide<K4>(ks[o][q]), hi = attn_wide<K4>(ks[o][q] >> 16);
                        if ((lo || hi) && key < len) atomicMin(s_wide, key), atomicMax(s_wide + 1, key), *s_odd = 1;
                        ks[o][q] = (lo ? 0u : ks[o][q] & 0xFFFFu) | (hi ? 0u : ks[o][q] & 0xFFFF0000u);
                    }
            }
#pragma unroll
            for (int i = 0; i < KL; ++i) {
                const uint32_t w[4] = {kq[i].x, kq[i].y, kq[i].z, kq[i].w};
#pragma unroll
                for (int q = 0; q < 4; q += K4 ? 1 : 2) {  // a chunk: one word of 8 nibbles or two of 4 bytes
                    const int f = 4 * i + q, per = K4 ? NB : D / 16, o = f / per, jj = f % per;
                    const int blk = K4 ? jj : jj >> 1, chunk = 2 * t4 + (blk & 1);
                    const uint32_t d2 = prmt(ks[o][blk >> 1], 0u, (blk & 1) ? 0x3232u : 0x1010u);
                    uint32_t h[4];
                    if constexpr (K4) {
                        prompt_ints4(w[q], h);
                    } else {
                        uint32_t a[2], e[2];
                        prompt_ints8(w[q], a);
                        prompt_ints8(w[q + 1 < 4 ? q + 1 : 3], e);
                        h[0] = a[0], h[1] = a[1], h[2] = e[0], h[3] = e[1];
                    }
                    *reinterpret_cast<uint4*>(kt + o * (8 * 128) + (blk >> 1) * (KT * 128) + ((chunk ^ g8) << 4)) =
                        make_uint4(prompt_mul2(h[0], d2), prompt_mul2(h[1], d2), prompt_mul2(h[2], d2), prompt_mul2(h[3], d2));
                }
            }
            load_k(blobs);
            fence_proxy_async_smem();
            mbar_arrive(kfull + buf);
            // ---- values: whatever lies past the sequence's end counts as 0
            if (j >= 2 && !wait(vempty + buf, ((j >> 1) - 1) & 1)) break;
            const int key0 = 16 * (glo + j * KG + 2 * pair);
            any = 0u;
#pragma unroll
            for (int c = 0; c < 2; ++c)
#pragma unroll
                for (int r = 0; r < 4; ++r) {
                    if (key0 + 16 * c + 8 * (r >> 1) + 2 * t4 + (r & 1) >= len) vsc[c][r] = 0u;
                    any |= vsc[c][r];
                }
            if (attn_maybe_wide(any)) {
                // scales that are not finite, or (fp16 rows) whose products are not: 0 here, and the rows that
                // see them are told
                int* const bad = s_bad + 4 * (b0 >> 1);
#pragma unroll
                for (int c = 0; c < 2; ++c)
#pragma unroll
                    for (int r = 0; r < 4; ++r) {
                        const uint32_t u = vsc[c][r];
                        const int key = key0 + 16 * c + 8 * (r >> 1) + 2 * t4 + (r & 1);
                        bool lo = (u & 0x7C00u) == 0x7C00u, hi = (u & 0x7C000000u) == 0x7C000000u;
                        if (lo) atomicMin(bad, key), atomicMax(bad + 1, key);
                        if (hi) atomicMin(bad + 2, key), atomicMax(bad + 3, key);
                        if constexpr (!BF) {
                            const bool wide_lo = attn_wide<V4>(u), wide_hi = attn_wide<V4>(u >> 16);
                            if (wide_lo || wide_hi) atomicMin(s_wide, key), atomicMax(s_wide + 1, key);
                            lo |= wide_lo, hi |= wide_hi;
                        }
                        if (lo || hi) *s_odd = 1;
                        vsc[c][r] = (lo ? 0u : u & 0xFFFFu) | (hi ? 0u : u & 0xFFFF0000u);
                    }
            }
            // lane (g, t) writes 8 keys of both groups as one chunk of channel 8 n + g
            uint8_t* const vt = smem + SH::oV + buf * SH::kV + (pair >> 1) * (D * 128) + (4 * 8 * b0 + g8) * 128 +
                                (((2 * t4 + (pair & 1)) ^ g8) << 4);
#pragma unroll
            for (int i = 0; i < VB; ++i) {
                float df[2][4];
                uint32_t d2[2][2];
#pragma unroll
                for (int c = 0; c < 2; ++c) {
#pragma unroll
                    for (int k = 0; k < 2; ++k) d2[c][k] = prmt(vsc[c][2 * k], vsc[c][2 * k + 1], i ? 0x7632u : v_sel);
#pragma unroll
                    for (int k = 0; k < 4; ++k) df[c][k] = (k & 1) ? half_hi(d2[c][k >> 1]) : half_lo(d2[c][k >> 1]);
                }
                const uint32_t w0[4] = {vq[0][i].x, vq[0][i].y, vq[0][i].z, vq[0][i].w};
                const uint32_t w1[4] = {vq[1][i].x, vq[1][i].y, vq[1][i].z, vq[1][i].w};
#pragma unroll
                for (int q = 0; q < (V4 ? 2 : 4); ++q) {
                    if constexpr (V4) {
                        uint32_t h[2][4];
                        prompt_ints4(w0[q], h[0]);
                        prompt_ints4(w1[q], h[1]);
#pragma unroll
                        for (int k = 0; k < 2; ++k)  // even and odd eights of channels
                            *reinterpret_cast<uint4*>(vt + (4 * i + 2 * q + k) * (8 * 128)) =
                                make_uint4(prompt_v4<BF>(h[0][k], df[0][0], df[0][1], d2[0][0]),
                                           prompt_v4<BF>(h[0][2 + k], df[0][2], df[0][3], d2[0][1]),
                                           prompt_v4<BF>(h[1][k], df[1][0], df[1][1], d2[1][0]),
                                           prompt_v4<BF>(h[1][2 + k], df[1][2], df[1][3], d2[1][1]));
                    } else {
                        uint32_t x[2], y[2];
                        prompt_v8<BF>(w0[q], df[0], d2[0][0], d2[0][1], x);
                        prompt_v8<BF>(w1[q], df[1], d2[1][0], d2[1][1], y);
                        *reinterpret_cast<uint4*>(vt + (4 * i + q) * (8 * 128)) = make_uint4(x[0], x[1], y[0], y[1]);
                    }
                }
            }
            load_v(blobs);
            fence_proxy_async_smem();
            mbar_arrive(vfull + buf);
        }
    } else {
        prompt_regs<true, kSoftmaxRegs>();
        if ((warp >> 2) < ntiles) {
        // ================================================================ softmax: one thread a row
        const int t = warp >> 2, r = min(r_begin + tid, r_end - 1);
        const bool there = r_begin + tid < r_end;
        const uint32_t lanes = static_cast<uint32_t>((warp & 3) * 32) << 16;
        const uint32_t cs = tmem + t * SH::cS + lanes, co = tmem + SH::cO + t * D + lanes;
        const int i_row = r / p.G, h = hk * p.G + r - i_row * p.G, pos = from + i_row;
        const int first_key = p.window > 0 ? pos - p.window + 1 : 0;
        const float rscale = s_scale[tid];
        const bool plain = p.cap <= 0.0f && !p.slopes && rscale > 0.0f;
        constexpr float kLog2e = 1.44269504088896340736f;
        const float sx = p.cap > 0.0f ? rscale : rscale * kLog2e, slope = p.slopes ? p.slopes[h] * kLog2e : 0.0f;
        const float inv_cap = p.cap > 0.0f ? 2.0f * kLog2e / p.cap : 0.0f;
        // steps that every row of the tile sees whole
        const int t_first = from + (r_begin + 128 * t) / p.G, t_last = from + (min(r_end, r_begin + 128 * t + 128) - 1) / p.G;
        const int seen_from = p.window > 0 ? t_last - p.window + 1 : 0;
        float m = -1e30f, l = 0.0f;
        for (int i = 0; i < turns; ++i) {
            const int sb = i & 1;
            if (!wait(sfull + 2 * t + sb, (i >> 1) & 1)) break;
            tc_fence_after();
            const int key0 = 16 * glo + i * 64;
            const bool whole = key0 + 63 <= t_first && key0 >= seen_from;
            float x[64];
            prompt_ld32(cs + 64 * sb, x);
            prompt_ld32(cs + 64 * sb + 32, x + 32);
            prompt_wait_ld();
            prompt_tie32(x);
            prompt_tie32(x + 32);
            // logits in units of log2 (plain: still to be multiplied by sx)
            if (!plain) {
                const float rel = static_cast<float>(key0 - pos);
#pragma unroll
                for (int k = 0; k < 64; ++k) {
                    float y = x[k] * sx;
                    // tanh(z) = 1 - 2 / (1 + exp(2 z))
                    if (p.cap > 0.0f) {
                        const float z = y * inv_cap;
                        y = kLog2e * (p.cap - __fdividef(2.0f * p.cap, 1.0f + prompt_ex2(z > 120.0f ? 120.0f : z)));
                    }
                    x[k] = fmaf(slope, rel + static_cast<float>(k), y);
                }
            }
            if (!whole) {
#pragma unroll
                for (int k = 0; k < 64; ++k)
                    if (key0 + k > pos || key0 + k < first_key) x[k] = -INFINITY;
            }
            float tops[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
#pragma unroll
            for (int k = 0; k < 64; ++k) tops[k & 3] = fmaxf(tops[k & 3], x[k]);
            const float mul = plain ? sx : 1.0f;
            const float top = fmaxf(fmaxf(tops[0], tops[1]), fmaxf(tops[2], tops[3])) * mul;
            const bool raise = top > m + 8.0f;
            if (__any_sync(0xffffffffu, raise)) {
                const float mn = raise ? top : m, a = prompt_ex2(m - mn);
                m = mn;
                l *= a;
                if (i > 0) {
                    if (!wait(pdone + 2 * t + (sb ^ 1), ((i - 1) >> 1) & 1)) break;
                    tc_fence_after();
#pragma unroll 1
                    for (int c = 0; c < D / 16; ++c) {
                        float o[16];
                        prompt_ld16(co + 16 * c, o);
#pragma unroll
                        for (int k = 0; k < 16; ++k) o[k] *= a;
                        prompt_st16(co + 16 * c, o);
                    }
                }
            }
            // fp16: 2^7 times the probabilities, at most 2^15, so that fewer are subnormal
            const float ref = BF ? m : m - 7.0f;
            float sum[4] = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
            for (int k = 0; k < 64; k += 2) {
                ffma2(x[k], x[k + 1], x[k], x[k + 1], mul, -ref, -ref);
                x[k] = prompt_ex2(x[k]);
                x[k + 1] = prompt_ex2(x[k + 1]);
                add2(sum[k & 2], sum[(k & 2) + 1], sum[k & 2], sum[(k & 2) + 1], x[k], x[k + 1]);
            }
            // the V tile's key order in an atom of 64: word 8 t + 2 g holds keys 2 t, 2 t + 1 of group g,
            // the next one keys 8 + 2 t, 9 + 2 t
            uint32_t w[32];
#pragma unroll
            for (int q = 0; q < 4; ++q)
#pragma unroll
                for (int gq = 0; gq < 4; ++gq) {
                    const int k = 16 * gq + 2 * q;
                    w[8 * q + 2 * gq] = prompt_pack<BF>(x[k], x[k + 1]);
                    w[8 * q + 2 * gq + 1] = prompt_pack<BF>(x[k + 8], x[k + 9]);
                }
            prompt_st32(cs + 64 * sb, w);
            l += (sum[0] + sum[1]) + (sum[2] + sum[3]);
            tmem_wait_st();
            tc_fence_before();
            mbar_arrive(pfull + 2 * t + sb);
        }
        // ---- output rows
        if (turns > 0) wait(pdone + 2 * t + ((turns - 1) & 1), ((turns - 1) >> 1) & 1);
        tc_fence_after();
        const float inv = l > 0.0f || l != l ? 1.0f / l : 0.0f;
        const int64_t at = (first + i_row) * p.out_token + h * p.out_head;
        const bool odd = *s_odd != 0;
        bool spoilt = false;  // an infinite or NaN value of the block among those that the row sees
#pragma unroll 1
        for (int c = 0; c < D / 16; ++c) {
            float o[16];
            if (odd && (c & 1) == 0) {
                spoilt = prompt_spoilt<V4, D>(p, s_bad, b, hk, c >> 1, first_key, pos);
                __syncwarp();
            }
            if (steps > 0) prompt_ld16(co + 16 * c, o);
            if (there) {
#pragma unroll
                for (int k = 0; k < 16; k += 8) {
                    uint32_t w[4];
#pragma unroll
                    for (int q = 0; q < 4; ++q) {
                        const float a = steps > 0 && l != 0.0f ? o[k + 2 * q] * inv : 0.0f, b2 = steps > 0 && l != 0.0f ? o[k + 2 * q + 1] * inv : 0.0f;
                        w[q] = prompt_pack<BF>(spoilt ? NAN : a, spoilt ? NAN : b2);
                    }
                    uint2* const dst = reinterpret_cast<uint2*>(static_cast<uint16_t*>(p.out) + at + 16 * c + k);
                    dst[0] = make_uint2(w[0], w[1]);
                    dst[1] = make_uint2(w[2], w[3]);
                }
            }
        }
        // ---- rows that may see keys or values which the tiles left out
        __syncwarp();  // their outputs, written above by their own lanes, are written again by the warp
        uint32_t again = odd ? __ballot_sync(0xffffffffu, there && s_wide[0] <= pos && s_wide[1] >= first_key && s_wide[1] >= 0) : 0u;
        for (; again; again &= again - 1u) {
            const int from_lane = __ffs(again) - 1;
            attn_exact_row<K4, V4, D, std::conditional_t<BF, __nv_bfloat16, __half>, !BF>(
                p, b, hk, __shfl_sync(0xffffffffu, h, from_lane), first + __shfl_sync(0xffffffffu, i_row, from_lane),
                __shfl_sync(0xffffffffu, first_key, from_lane), __shfl_sync(0xffffffffu, pos, from_lane));
        }
        }
    }
    tc_fence_before();
    __syncthreads();
    if (warp == kFirstMma) {
        tc_fence_after();
        asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(512u) : "memory");
    }
}

template <bool K4, bool V4, int D, bool BF>
cudaError_t launch_attn_prompt_one(const AttnParams& p, cudaStream_t s) {
    using SH = PromptShape<D>;
    static_assert(SH::kTotal <= kSmemLimit, "shared memory");
    static std::atomic<bool> set[kMaxDevices] = {};
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    if (dev < 0 || dev >= kMaxDevices) return cudaErrorInvalidDevice;
    if (!set[dev].load(std::memory_order_acquire)) {
        cudaFuncAttributes at;
        e = cudaFuncGetAttributes(&at, k_attn_prompt<K4, V4, D, BF>);
        if (e != cudaSuccess) return e;
        if (at.numRegs != kLaunchRegs) return cudaErrorInvalidConfiguration;  // the split would not add up
        e = cudaFuncSetAttribute(k_attn_prompt<K4, V4, D, BF>, cudaFuncAttributeMaxDynamicSharedMemorySize, SH::kTotal);
        if (e != cudaSuccess) return e;
        set[dev].store(true, std::memory_order_release);
    }
    const int64_t tiles = (static_cast<int64_t>(p.max_q) * p.G + SH::kRows - 1) / SH::kRows;
    return launch_pdl(k_attn_prompt<K4, V4, D, BF>,
                      dim3(static_cast<unsigned>(p.n_seqs * p.Hkv), static_cast<unsigned>(tiles)), dim3(kPromptThreads),
                      SH::kTotal, s, p);
}

template <int D>
cudaError_t launch_attn_prompt_dim(const AttnParams& p, cudaStream_t s) {
    const bool bf = p.dtype == 2;
    if (p.k_q4) {
        if (p.v_q4) return bf ? launch_attn_prompt_one<true, true, D, true>(p, s) : launch_attn_prompt_one<true, true, D, false>(p, s);
        return bf ? launch_attn_prompt_one<true, false, D, true>(p, s) : launch_attn_prompt_one<true, false, D, false>(p, s);
    }
    if (p.v_q4) return bf ? launch_attn_prompt_one<false, true, D, true>(p, s) : launch_attn_prompt_one<false, true, D, false>(p, s);
    return bf ? launch_attn_prompt_one<false, false, D, true>(p, s) : launch_attn_prompt_one<false, false, D, false>(p, s);
}

}  // namespace ggq
