// ggq_attn_prompt.cuh -- attention of many query rows (prompts) over the packed
// cache on tcgen05, for 16-bit activations.
//
// Mathematics: S = Q K^T and O = P V per kv head, the rows being the head
// group's query heads of consecutive tokens, with the softmax's running maximum
// and sum.  Bound by the tensor cores: 4 D operations per (row, key), 2 kt D bytes
// of packed cache per 128-row tile and step of kt keys.
//
// A CTA takes one kv head of one sequence and one or two tiles of 128 rows that
// share its steps of keys (heads of 256 channels: one tile, whose O fills half of
// tensor memory).  Roles:
//   * warps 0-3 and 4-7: the softmax of a tile, one thread a row.  Scores come
//     from tensor memory; probabilities go back over them as the first operand of
//     P V (tensor memory holds it, so only V is read from shared memory), in the
//     channels' key order of the V tile;
//   * warps 8-11: the packed blobs, read straight from the cache, to fp16 (V with
//     bf16 activations: bf16) tiles in the K-major 128-byte-swizzled layout, two
//     buffers each for K and V;
//   * warps 12, 13: one thread each issues a tile's MMAs: S of step j when its K
//     tile is there, then O += P V when the softmax has written P.  The two tiles'
//     products and softmaxes take turns.
// The running maximum is raised (and O rescaled in tensor memory) only when a row
// passes it by 2^8.  fp16 queries are exact; bf16 ones too (rows are scaled by a
// power of two).  K is rounded to fp16; V and P to the activations' type, so that
// with bf16 no probability is lost for being small.
#pragma once
#include <atomic>

#include "ggq_attn.cuh"
#include "ggq_device.cuh"
#include "ggq_internal.h"
#include "ggq_tcgen05.cuh"

namespace ggq {

constexpr int kPromptThreads = 14 * 32;

template <int D>
struct PromptShape {
    static constexpr int kTiles = D <= 128 ? 2 : 1;
    static constexpr int kKeys = D <= 128 ? 128 : 64;  // of a step
    static constexpr int kRows = 128 * kTiles;
    static constexpr int kQ = 128 * D * 2;             // bytes of a tile's queries
    static constexpr int kK = kKeys * D * 2, kV = kK;  // bytes of a step's keys, values
    static constexpr int oK = kTiles * kQ, oV = oK + 2 * kK, oBar = oV + 2 * kV;
    static constexpr int kTotal = oBar + 256 + 1024;   // + alignment of the tiles
    // tensor-memory columns: scores of each tile (probabilities over them), then the outputs
    static constexpr uint32_t cS = kKeys, cO = kTiles * cS;
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
__device__ __forceinline__ void tmem_st16(uint32_t taddr, const uint32_t (&v)[16]) {
    asm volatile(
        "tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16};" ::"r"(taddr),
        "r"(v[0]), "r"(v[1]), "r"(v[2]), "r"(v[3]), "r"(v[4]), "r"(v[5]), "r"(v[6]), "r"(v[7]), "r"(v[8]), "r"(v[9]),
        "r"(v[10]), "r"(v[11]), "r"(v[12]), "r"(v[13]), "r"(v[14]), "r"(v[15])
        : "memory");
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
// A pair of exact fp16 integers times a pair of fp16 scales, in the operand's type
// (bf16: one rounding of the fp32 product).
template <bool BF>
__device__ __forceinline__ uint32_t prompt_scaled(uint32_t q, uint32_t d) {
    if constexpr (BF) {
        const float2 a = __half22float2(*reinterpret_cast<const __half2*>(&q));
        const float2 b = __half22float2(*reinterpret_cast<const __half2*>(&d));
        return prompt_pack<true>(a.x * b.x, a.y * b.y);
    }
    return prompt_mul2(q, d);
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

template <bool K4, bool V4, int D, bool BF>
__global__ void __launch_bounds__(kPromptThreads, 1) k_attn_prompt(const __grid_constant__ AttnParams p) {
    using SH = PromptShape<D>;
    constexpr int TILES = SH::kTiles, KT = SH::kKeys, NB = D / 32, KG = KT / 16;
    extern __shared__ __align__(1024) uint8_t smem_raw[];
    uint8_t* const smem = smem_raw + ((1024 - (smem_addr(smem_raw) & 1023)) & 1023);
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    uint64_t* const bars = reinterpret_cast<uint64_t*>(smem + SH::oBar);
    uint64_t *const kfull = bars, *const kempty = bars + 2, *const vfull = bars + 4, *const vempty = bars + 6;
    uint64_t *const sfull = bars + 8, *const pfull = bars + 10, *const ofull = bars + 12, *const done = bars + 14;
    uint32_t* const tslot = reinterpret_cast<uint32_t*>(bars + 16);
    volatile int* const abort = reinterpret_cast<volatile int*>(tslot + 1);
    int* const s_bad = reinterpret_cast<int*>(tslot + 2);  // [NB][2] first and last key whose value scale is not finite

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
    const int steps = ghi > glo ? (ghi - glo + KG - 1) / KG : 0;

    if (tid == 0) {
        for (int i = 0; i < 2; ++i) {
            mbar_init(kfull + i, 128);
            mbar_init(vfull + i, 128);
            mbar_init(kempty + i, static_cast<uint32_t>(ntiles));
            mbar_init(vempty + i, static_cast<uint32_t>(ntiles));
            mbar_init(sfull + i, 1);
            mbar_init(pfull + i, 128);
            mbar_init(ofull + i, 1);
            mbar_init(done + i, 1);
        }
        *abort = 0;
        for (int i = 0; i < NB; ++i) s_bad[2 * i] = 0x7fffffff, s_bad[2 * i + 1] = -1;
        fence_barrier_init();
    }
    if (warp == 12) {
        asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_addr(tslot)), "r"(512u)
                     : "memory");
        asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
    }
    // ---- queries: thread a row, fp16 with the row's largest element in [2^13, 2^14)
    float rscale = 0.0f;
    if (warp < 4 * TILES && (warp >> 2) < ntiles) {
        const int r = min(r_begin + tid, r_end - 1), i = r / p.G, h = hk * p.G + r - i * p.G;
        const int64_t at = (first + i) * p.q_token + h * p.q_head;
        const auto q4 = [&](int d) {
            return BF ? ld4(static_cast<const __nv_bfloat16*>(p.q) + at + d) : ld4(static_cast<const __half*>(p.q) + at + d);
        };
        float amax = 0.0f;
#pragma unroll 8
        for (int d = 0; d < D; d += 4) {
            const float4 x = q4(d);
            amax = fmaxf(fmaxf(amax, fmaxf(fabsf(x.x), fabsf(x.y))), fmaxf(fabsf(x.z), fabsf(x.w)));
        }
        const int ex = static_cast<int>(__float_as_uint(amax) >> 23) - 127;
        const int sh = ex == 128 ? 0 : min(13 - ex, 100);
        const float up = __uint_as_float(static_cast<uint32_t>(sh + 127) << 23);
        rscale = p.scale * scalbnf(1.0f, -sh);
        uint8_t* const row = smem + (tid >> 7) * SH::kQ + (tid & 127) * 128;
#pragma unroll 4
        for (int d = 0; d < D; d += 8) {
            const float4 x = q4(d), y = q4(d + 4);
            const uint4 u = make_uint4(prompt_pack<false>(x.x * up, x.y * up), prompt_pack<false>(x.z * up, x.w * up),
                                       prompt_pack<false>(y.x * up, y.y * up), prompt_pack<false>(y.z * up, y.w * up));
            *reinterpret_cast<uint4*>(row + (d >> 6) * (128 * 128) + ((((d & 63) >> 3) ^ (tid & 7)) << 4)) = u;
        }
        fence_proxy_async_smem();
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = *tslot;

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

    if (warp >= 12) {
        // ================================================================ MMA: one thread a tile
        const int t = warp - 12;
        if (t < ntiles && lane == 0 && steps > 0) {
            const uint32_t id_s = prompt_idesc(KT, false), id_o = prompt_idesc(D, BF);
            const uint32_t cs = tmem + t * SH::cS, co = tmem + SH::cO + t * D;
            const uint64_t qd = umma_desc_sw128(smem_addr(smem + t * SH::kQ));
            for (int j = 0; j < steps; ++j) {
                const int buf = j & 1;
                const uint32_t ph = (j >> 1) & 1;
                if (!wait1(kfull + buf, ph)) break;
                tc_fence_after();
                const uint64_t kd = umma_desc_sw128(smem_addr(smem + SH::oK + buf * SH::kK));
#pragma unroll
                for (int k = 0; k < D / 16; ++k)  // 32 bytes a step inside a 64-channel atom
                    tc_mma(cs, qd + (k >> 2) * (128 * 128 / 16) + 2 * (k & 3), kd + (k >> 2) * (KT * 128 / 16) + 2 * (k & 3),
                           id_s, k > 0);
                tc_commit(sfull + t);
                tc_commit(kempty + buf);
                if (!wait1(pfull + t, j & 1)) break;
                if (!wait1(vfull + buf, ph)) break;
                tc_fence_after();
                const uint64_t vd = umma_desc_sw128(smem_addr(smem + SH::oV + buf * SH::kV));
#pragma unroll
                for (int k = 0; k < KT / 16; ++k)
                    tc_mma_ts(co, cs + 8 * k, vd + (k >> 2) * (D * 128 / 16) + 2 * (k & 3), id_o, (j > 0 || k > 0) ? 1u : 0u);
                tc_commit(ofull + t);
                tc_commit(vempty + buf);
            }
            tc_commit(done + t);
            mbar_wait(done + t, 0);  // every MMA has ended before tensor memory goes
        }
    } else if (warp >= 8) {
        // ================================================================ packed blobs -> operand tiles
        const int cw = warp - 8, g8 = lane >> 2, t4 = lane & 3, gpp = p.page >> 4;
        constexpr int kKB = kv_blob_bytes(K4, D), kVB = kv_blob_bytes(V4, D);
        constexpr int kPer = KG / 4;  // groups of a step and warp: cw, cw + 4
        constexpr int KL = K4 ? D / 64 : D / 32, VL = V4 ? D / 64 : D / 32;  // 16-byte words of a lane and blob
        const auto page_at = [&](int s) {  // page of this warp's s-th group; 32 at a time, one a lane
            const int g = glo + (s / kPer) * KG + cw + 4 * (s % kPer);
            int pg = -1;
            if (g < ghi) {
                pg = p.table[b * p.table_stride + g / gpp];
                if (pg < 0 || pg >= p.n_pages) {
                    set_error(p.err, DEV_ERR_BAD_PLACE);
                    pg = 0;
                }
            }
            return pg;
        };
        const int total = steps * kPer;
        int pages = page_at(lane);
        uint4 kq[KL], vq[VL];
        uint32_t ks[2][NB / 2], vsc[4][NB / 2];
        int64_t blob = -1;
        const auto locate = [&](int s) {
            if ((s & 31) == 0 && s > 0) pages = page_at(s + lane);
            const int pg = __shfl_sync(0xffffffffu, pages, s & 31);
            const int g = glo + (s / kPer) * KG + cw + 4 * (s % kPer);
            return pg < 0 ? int64_t(-1) : (static_cast<int64_t>(pg) * p.Hkv + hk) * gpp + g % gpp;
        };
        const auto load_k = [&](int64_t at) {
            if (at < 0) return;
            const uint8_t* const src = p.k + at * kKB;
#pragma unroll
            for (int i = 0; i < KL; ++i) kq[i] = __ldg(reinterpret_cast<const uint4*>(src + (i * 32 + lane) * 16));
#pragma unroll
            for (int o = 0; o < 2; ++o)
#pragma unroll
                for (int i = 0; i < NB / 2; ++i)
                    ks[o][i] = __ldg(reinterpret_cast<const uint32_t*>(src + kv_quant_bytes(K4, D) + (8 * o + g8) * NB * 2) + i);
        };
        const auto load_v = [&](int64_t at) {
            if (at < 0) return;
            const uint8_t* const src = p.v + at * kVB;
#pragma unroll
            for (int i = 0; i < VL; ++i) vq[i] = __ldg(reinterpret_cast<const uint4*>(src + (i * 32 + lane) * 16));
#pragma unroll
            for (int r = 0; r < 4; ++r)
#pragma unroll
                for (int i = 0; i < NB / 2; ++i)
                    vsc[r][i] = __ldg(reinterpret_cast<const uint32_t*>(src + kv_quant_bytes(V4, D) +
                                                                        (8 * (r >> 1) + 2 * t4 + (r & 1)) * NB * 2) + i);
        };
        if (total > 0) {
            blob = locate(0);
            load_k(blob);
            load_v(blob);
        }
        bool ok = true;
        for (int s = 0; s < total && ok; ++s) {
            const int j = s / kPer, buf = j & 1, gi = cw + 4 * (s % kPer), g = glo + j * KG + gi;
            const int64_t now = blob;
            blob = s + 1 < total ? locate(s + 1) : -1;
            // keys
            if (s % kPer == 0 && j >= 2) ok = wait(kempty + buf, ((j >> 1) - 1) & 1);
            if (!ok) break;
            if (now >= 0) {
                uint8_t* const kt = smem + SH::oK + buf * SH::kK + (gi * 16 + g8) * 128 + 8 * (t4 & 1);
#pragma unroll
                for (int i = 0; i < KL; ++i) {
                    const uint32_t w[4] = {kq[i].x, kq[i].y, kq[i].z, kq[i].w};
#pragma unroll
                    for (int c = 0; c < 4; ++c) {
                        const int f = 4 * i + c, per = K4 ? NB : D / 16, o = f / per, jj = f % per;
                        const int blk = K4 ? jj : jj >> 1;
                        const uint32_t d2 = prmt(ks[o][blk >> 1], 0u, (blk & 1) ? 0x3232u : 0x1010u);
                        uint8_t* const row = kt + o * (8 * 128);
                        if constexpr (K4) {
                            uint32_t h[4];
                            prompt_ints4(w[c], h);
#pragma unroll
                            for (int k = 0; k < 2; ++k) {
                                const int ks16 = 2 * jj + k;  // 16-channel step
                                *reinterpret_cast<uint2*>(row + (ks16 >> 2) * (KT * 128) + (((2 * (ks16 & 3) + (t4 >> 1)) ^ g8) << 4)) =
                                    make_uint2(prompt_mul2(h[2 * k], d2), prompt_mul2(h[2 * k + 1], d2));
                            }
                        } else {
                            uint32_t h[2];
                            prompt_ints8(w[c], h);
                            *reinterpret_cast<uint2*>(row + (jj >> 2) * (KT * 128) + (((2 * (jj & 3) + (t4 >> 1)) ^ g8) << 4)) =
                                make_uint2(prompt_mul2(h[0], d2), prompt_mul2(h[1], d2));
                        }
                    }
                }
            }
            load_k(blob);
            if (s % kPer == kPer - 1) {
                fence_proxy_async_smem();
                mbar_arrive(kfull + buf);
            }
            // values: whatever lies past the sequence's end counts as 0
            if (s % kPer == 0 && j >= 2) ok = wait(vempty + buf, ((j >> 1) - 1) & 1);
            if (!ok) break;
            if (now < 0) {
#pragma unroll
                for (int r = 0; r < 4; ++r)
#pragma unroll
                    for (int i = 0; i < NB / 2; ++i) vsc[r][i] = 0u;
#pragma unroll
                for (int i = 0; i < VL; ++i) vq[i] = make_uint4(0u, 0u, 0u, 0u);
            } else if (16 * g + 16 > len) {
#pragma unroll
                for (int r = 0; r < 4; ++r)
                    if (16 * g + 8 * (r >> 1) + 2 * t4 + (r & 1) >= len)
#pragma unroll
                        for (int i = 0; i < NB / 2; ++i) vsc[r][i] = 0u;
            }
            // scales that are not finite: 0 here, and the rows that see them are told
#pragma unroll
            for (int r = 0; r < 4; ++r)
#pragma unroll
                for (int i = 0; i < NB / 2; ++i) {
                    const uint32_t u = vsc[r][i];
                    if ((u & 0x7C00u) == 0x7C00u || (u & 0x7C000000u) == 0x7C000000u) {
                        const int key = 16 * g + 8 * (r >> 1) + 2 * t4 + (r & 1);
                        if ((u & 0x7C00u) == 0x7C00u) atomicMin(s_bad + 4 * i, key), atomicMax(s_bad + 4 * i + 1, key);
                        if ((u & 0x7C000000u) == 0x7C000000u) atomicMin(s_bad + 4 * i + 2, key), atomicMax(s_bad + 4 * i + 3, key);
                        vsc[r][i] = ((u & 0x7C00u) == 0x7C00u ? 0u : u & 0xFFFFu) |
                                    ((u & 0x7C000000u) == 0x7C000000u ? 0u : u & 0xFFFF0000u);
                    }
                }
            uint8_t* const vt = smem + SH::oV + buf * SH::kV + (gi >> 2) * (D * 128) + g8 * 128 +
                                (((2 * (gi & 3) + (t4 >> 1)) ^ g8) << 4) + 8 * (t4 & 1);
#pragma unroll
            for (int i = 0; i < VL; ++i) {
                const uint32_t w[4] = {vq[i].x, vq[i].y, vq[i].z, vq[i].w};
#pragma unroll
                for (int c = 0; c < 4; ++c) {
                    const int blk = V4 ? (4 * i + c) >> 1 : i;
                    // scales of the key pairs (2t, 2t+1) and (8+2t, 9+2t) in this block
                    const uint32_t sel = (blk & 1) ? 0x7632u : 0x5410u;
                    const uint32_t d0 = prmt(vsc[0][blk >> 1], vsc[1][blk >> 1], sel);
                    const uint32_t d1 = prmt(vsc[2][blk >> 1], vsc[3][blk >> 1], sel);
                    if constexpr (V4) {
                        uint32_t h[4];
                        prompt_ints4(w[c], h);
                        const int n0 = 2 * (4 * i + c);
                        *reinterpret_cast<uint2*>(vt + n0 * (8 * 128)) = make_uint2(prompt_scaled<BF>(h[0], d0), prompt_scaled<BF>(h[2], d1));
                        *reinterpret_cast<uint2*>(vt + (n0 + 1) * (8 * 128)) = make_uint2(prompt_scaled<BF>(h[1], d0), prompt_scaled<BF>(h[3], d1));
                    } else {
                        uint32_t h[2];
                        prompt_ints8(w[c], h);
                        *reinterpret_cast<uint2*>(vt + (4 * i + c) * (8 * 128)) = make_uint2(prompt_scaled<BF>(h[0], d0), prompt_scaled<BF>(h[1], d1));
                    }
                }
            }
            load_v(blob);
            if (s % kPer == kPer - 1) {
                fence_proxy_async_smem();
                mbar_arrive(vfull + buf);
            }
        }
    } else if ((warp >> 2) < ntiles) {
        // ================================================================ softmax: one thread a row
        const int t = warp >> 2, r = min(r_begin + tid, r_end - 1);
        const bool there = r_begin + tid < r_end;
        const uint32_t lanes = static_cast<uint32_t>((warp & 3) * 32) << 16;
        const uint32_t cs = tmem + t * SH::cS + lanes, co = tmem + SH::cO + t * D + lanes;
        const int i_row = r / p.G, h = hk * p.G + r - i_row * p.G, pos = from + i_row;
        const int first_key = p.window > 0 ? pos - p.window + 1 : 0;
        const float slope = p.slopes ? p.slopes[h] : 0.0f;
        const bool plain = p.cap <= 0.0f && !p.slopes;
        constexpr float kLog2e = 1.44269504088896340736f;
        const float sx = plain ? rscale * kLog2e : rscale;
        const float inv_cap = p.cap > 0.0f ? 2.0f * kLog2e / p.cap : 0.0f;
        // steps that every row of the tile sees whole
        const int t_first = from + (r_begin + 128 * t) / p.G, t_last = from + (min(r_end, r_begin + 128 * t + 128) - 1) / p.G;
        const int seen_from = p.window > 0 ? t_last - p.window + 1 : 0;
        float m = -1e30f, l = 0.0f;
        for (int j = 0; j < steps; ++j) {
            if (!wait(sfull + t, j & 1)) break;
            tc_fence_after();
            const int key0 = 16 * glo + j * KT;
            const bool whole = key0 + KT - 1 <= t_first && key0 >= seen_from;
            // logits of 32 keys in units of log2
            const auto logits = [&](int c, float (&x)[32]) {
                tmem_ld32(cs + 32 * c, x);
                if (plain) {
#pragma unroll
                    for (int k = 0; k < 32; ++k) x[k] *= sx;
                } else {
#pragma unroll
                    for (int k = 0; k < 32; ++k) {
                        float y = x[k] * sx;
                        // tanh(z) = 1 - 2 / (1 + exp(2 z))
                        if (p.cap > 0.0f) {
                            const float z = y * inv_cap;
                            y = p.cap - __fdividef(2.0f * p.cap, 1.0f + prompt_ex2(z > 120.0f ? 120.0f : z));
                        }
                        x[k] = fmaf(slope, static_cast<float>(key0 + 32 * c + k - pos), y) * kLog2e;
                    }
                }
                if (!whole) {
#pragma unroll
                    for (int k = 0; k < 32; ++k) {
                        const int key = key0 + 32 * c + k;
                        if (key > pos || key < first_key) x[k] = -INFINITY;
                    }
                }
            };
            float top = -INFINITY;
#pragma unroll
            for (int c = 0; c < KT / 32; ++c) {
                float x[32];
                logits(c, x);
#pragma unroll
                for (int k = 0; k < 32; ++k) top = fmaxf(top, x[k]);
            }
            const bool raise = top > m + 8.0f;
            if (__any_sync(0xffffffffu, raise)) {
                const float mn = raise ? top : m, a = prompt_ex2(m - mn);
                m = mn;
                l *= a;
                if (j > 0) {
                    if (!wait(ofull + t, (j - 1) & 1)) break;
                    tc_fence_after();
#pragma unroll 1
                    for (int c = 0; c < D / 32; ++c) {
                        float o[32];
                        tmem_ld32(co + 32 * c, o);
#pragma unroll
                        for (int k = 0; k < 32; ++k) o[k] *= a;
                        tmem_st32(co + 32 * c, o);
                    }
                }
            }
#pragma unroll
            for (int c = 0; c < KT / 32; ++c) {
                float x[32];
                logits(c, x);
                float sum[4] = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
                for (int k = 0; k < 32; ++k) {
                    x[k] = prompt_ex2(x[k] - m);
                    sum[k & 3] += x[k];
                }
                l += (sum[0] + sum[1]) + (sum[2] + sum[3]);
                // the V tile's key order: 2t, 2t + 1, 8 + 2t, 9 + 2t inside a group of 16
                uint32_t w[16];
#pragma unroll
                for (int gq = 0; gq < 2; ++gq)
#pragma unroll
                    for (int q = 0; q < 4; ++q) {
                        w[8 * gq + 2 * q] = prompt_pack<BF>(x[16 * gq + 2 * q], x[16 * gq + 2 * q + 1]);
                        w[8 * gq + 2 * q + 1] = prompt_pack<BF>(x[16 * gq + 8 + 2 * q], x[16 * gq + 9 + 2 * q]);
                    }
                tmem_st16(cs + 16 * c, w);
            }
            tmem_wait_st();
            tc_fence_before();
            mbar_arrive(pfull + t);
        }
        // ---- output rows
        if (steps > 0) wait(ofull + t, (steps - 1) & 1);
        tc_fence_after();
        const float inv = l > 0.0f || l != l ? 1.0f / l : 0.0f;
        const int64_t at = (first + i_row) * p.out_token + h * p.out_head;
#pragma unroll 1
        for (int c = 0; c < D / 32; ++c) {
            float o[32];
            if (steps > 0) tmem_ld32(co + 32 * c, o);
            // an infinite or NaN value among those that the row sees
            const bool spoilt = s_bad[2 * c] <= pos && s_bad[2 * c + 1] >= first_key && s_bad[2 * c + 1] >= 0;
            if (there) {
#pragma unroll
                for (int k = 0; k < 32; k += 8) {
                    uint32_t w[4];
#pragma unroll
                    for (int q = 0; q < 4; ++q) {
                        const float a = steps > 0 && l != 0.0f ? o[k + 2 * q] * inv : 0.0f, b2 = steps > 0 && l != 0.0f ? o[k + 2 * q + 1] * inv : 0.0f;
                        w[q] = prompt_pack<BF>(spoilt ? NAN : a, spoilt ? NAN : b2);
                    }
                    uint2* const dst = reinterpret_cast<uint2*>(static_cast<uint16_t*>(p.out) + at + 32 * c + k);
                    dst[0] = make_uint2(w[0], w[1]);
                    dst[1] = make_uint2(w[2], w[3]);
                }
            }
        }
    }
    tc_fence_before();
    __syncthreads();
    if (warp == 12) {
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
