// ggq_attn_promptf.cuh -- attention of many fp32 query rows (prompts) over the packed
// cache on tcgen05, for heads of 64 and 128 channels.
//
// Mathematics: with q the stored integers and d the scales of 32-channel blocks b,
//   s[key] = sum_b d_k[key][b] (Q_b . q_k[key][b]),   O_b += (p[key] d_v[key][b]) q_v[key][b].
// The integers are exact operands; the scales are applied in fp32 to the scores
// (one accumulator a block) and to the probabilities (one operand a block).  What is
// rounded: Q, to two fp16 terms of a row scaled by a power of two (22 bits).  p d_v is
// cut into three bf16 terms (all 24 bits, and the type's range is fp32's: nothing is
// lost for being small; with two terms the outputs were 6 times further off).  Tensor memory sums 128 keys; the sums of those are added up
// in registers, in fp32 with rounding to nearest.
//
// Measured (28 heads on 4 of 128 channels, distance bias, 5 ragged prompts of up to 1000
// rows): 177 us, 103 TFLOP/s of the formula's operations (on mma.sync with the scales in
// the accumulators: 321 us); 4096 causal rows of 32 heads on 8: 744 us (1716).  A step of
// 32 keys takes 128 rows 1.5 us for 40 MMAs of 32 columns, some 70 cycles each whatever
// their width; issue slots 64% used, tensor pipe 11%.
//
// A CTA takes 128 rows of one kv head of one sequence.  Roles:
//   * warps 0-15: four threads a row, each a quarter of a step's keys and of the output's
//     channels; they agree on the row's maximum through shared memory;
//   * warps 16-23: the packed blobs to fp16 (keys) and bf16 (values) integers, K-major
//     128-byte-swizzled tiles of 128 keys, and their scales to fp32;
//   * warps 24, 25 and 26, 27: one thread each issues the scores' and the outputs' MMAs
//     of half the blocks (the instructions are small: one thread's issue would bound them).
// Keys lie in tiles, scores and probabilities in the order in which a V word's lanes
// hold them: key 16 c + 8 o + 2 t + e of 32 at place 8 t + 4 c + 2 o + e.
#pragma once
#include <atomic>

#include "ggq_attn_prompt.cuh"

namespace ggq {

// Four threads a row: 16 softmax warps, four a scheduler (measured together, 5 ragged prompts
// of up to 1000 rows with a distance bias: 175 us; two threads a row with 160 registers each:
// 191.  4096 causal rows without one: 737 and 727).
constexpr int kPfParts = 4, kPfSoftmaxWarps = 4 * kPfParts, kPfFirstMma = kPfSoftmaxWarps + kDecodeWarps;
constexpr int kPfThreads = (kPfFirstMma + kMmaWarps) * 32;
constexpr int kPfLaunchRegs = 72, kPfSoftmaxRegs = 88, kPfDecodeRegs = 56, kPfMmaRegs = 40;
static_assert(kPfSoftmaxRegs >= kPfLaunchRegs && kPfDecodeRegs <= kPfLaunchRegs && kPfMmaRegs <= kPfLaunchRegs &&
                  32 * (kPfSoftmaxWarps * kPfSoftmaxRegs + kDecodeWarps * kPfDecodeRegs + kMmaWarps * kPfMmaRegs) <=
                      kPfThreads * kPfLaunchRegs &&
                  kPfThreads * kPfLaunchRegs <= 65536,
              "register split");

template <int D>
struct PromptfShape {
    static constexpr int NB = D / 32;
    static constexpr int kTile = 128;             // keys of a tile
    static constexpr int kKeys = 128 / NB;        // keys of a step: its scores fill 128 columns
    static constexpr int kSteps = kTile / kKeys;  // steps of a tile; tensor memory sums over a tile
    static constexpr int kQ = 128 * D * 2, kK = kTile * D * 2, kV = kK, kS = kTile * NB * 4;
    static constexpr int oK = 2 * kQ, oV = oK + 2 * kK, oSK = oV + 2 * kV, oSV = oSK + 2 * kS, oTop = oSV + 2 * kS;
    static constexpr int oBar = oTop + 2 * kPfParts * 128 * 4, kTotal = oBar + 256 + 1024;
    static constexpr uint32_t cBuf = 192, cO = 2 * cBuf;  // columns: two buffers (scores 128, probabilities 192), then the output
    static_assert(cO + D <= 512, "tensor memory");
};

// A word's four bytes u as bf16 integers u - 128: 128 + (u & 127), minus 128 or 256.
__device__ __forceinline__ uint32_t pf_bf16_of(uint32_t a) {
    const uint32_t x = a & 0x437F437Fu, c = (a & 0x00800080u) ^ 0x43804380u;
    const __nv_bfloat162 r = __hsub2(*reinterpret_cast<const __nv_bfloat162*>(&x), *reinterpret_cast<const __nv_bfloat162*>(&c));
    return *reinterpret_cast<const uint32_t*>(&r);
}
__device__ __forceinline__ void pf_bytes(uint32_t w, uint32_t (&h)[2]) {
    h[0] = pf_bf16_of(prmt(w, 0x43434343u, 0x4140u));
    h[1] = pf_bf16_of(prmt(w, 0x43434343u, 0x4342u));
}
// nibbles (0, 4), (1, 5), (2, 6), (3, 7) as bf16 integers u - 8
__device__ __forceinline__ void pf_nibbles(uint32_t w, uint32_t (&h)[4]) {
    const uint32_t eight = 0x43084308u;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const uint32_t x = ((w >> (4 * i)) & 0x000F000Fu) | 0x43004300u;
        const __nv_bfloat162 r = __hsub2(*reinterpret_cast<const __nv_bfloat162*>(&x), *reinterpret_cast<const __nv_bfloat162*>(&eight));
        h[i] = *reinterpret_cast<const uint32_t*>(&r);
    }
}
// 8 columns, to be used after prompt_wait_ld on the same registers
__device__ __forceinline__ void pf_ld8(uint32_t taddr, float* v) {
    asm volatile("tcgen05.ld.sync.aligned.32x32b.x8.b32 {%0,%1,%2,%3,%4,%5,%6,%7}, [%8];"
                 : "=f"(v[0]), "=f"(v[1]), "=f"(v[2]), "=f"(v[3]), "=f"(v[4]), "=f"(v[5]), "=f"(v[6]), "=f"(v[7])
                 : "r"(taddr));
}
// keeps uses of v behind the wait
__device__ __forceinline__ void pf_tie8(float* v) {
    asm volatile("" : "+f"(v[0]), "+f"(v[1]), "+f"(v[2]), "+f"(v[3]), "+f"(v[4]), "+f"(v[5]), "+f"(v[6]), "+f"(v[7]));
}
__device__ __forceinline__ void pf_st4(uint32_t taddr, const uint32_t* v) {
    asm volatile("tcgen05.st.sync.aligned.32x32b.x4.b32 [%0], {%1,%2,%3,%4};" ::"r"(taddr), "r"(v[0]), "r"(v[1]), "r"(v[2]),
                 "r"(v[3]));
}
__device__ __forceinline__ void pf_st8(uint32_t taddr, const uint32_t* v) {
    asm volatile("tcgen05.st.sync.aligned.32x32b.x8.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8};" ::"r"(taddr), "r"(v[0]), "r"(v[1]),
                 "r"(v[2]), "r"(v[3]), "r"(v[4]), "r"(v[5]), "r"(v[6]), "r"(v[7]));
}
__device__ __forceinline__ float pf_half(uint32_t bits) { return __half2float(__ushort_as_half(static_cast<unsigned short>(bits))); }
// the warps of 32 rows
__device__ __forceinline__ void pf_rows_sync(int quarter) { asm volatile("bar.sync %0, %1;" ::"r"(quarter + 1), "n"(32 * kPfParts) : "memory"); }

template <bool K4, bool V4, int D>
__global__ void __launch_bounds__(kPfThreads, 1) k_attn_promptf(const __grid_constant__ AttnParams p) {
    using SH = PromptfShape<D>;
    constexpr int NB = SH::NB, KT = SH::kTile, KEYS = SH::kKeys, STEPS = SH::kSteps, KG = KT / 16;
    constexpr int HK = KEYS / kPfParts, HD = D / kPfParts;  // keys and channels of a softmax thread
    constexpr int KS = KEYS / 16, PC = 192 / KS;             // MMA depths of a step's keys, columns of one's probabilities
    extern __shared__ __align__(1024) uint8_t smem_raw[];
    uint8_t* const smem = smem_raw + ((1024 - (smem_addr(smem_raw) & 1023)) & 1023);
    const int tid = threadIdx.x, warp = __shfl_sync(0xffffffffu, tid >> 5, 0), lane = tid & 31;  // warp: uniform
    uint64_t* const bars = reinterpret_cast<uint64_t*>(smem + SH::oBar);
    uint64_t *const kfull = bars, *const kempty = bars + 2, *const vfull = bars + 4, *const vempty = bars + 6;
    uint64_t *const sfull = bars + 8, *const pfull = bars + 10, *const pdone = bars + 12, *const done = bars + 14;
    uint32_t* const tslot = reinterpret_cast<uint32_t*>(bars + 18);
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
    const int R = shown * p.G, r_begin = tile * 128;
    if (r_begin >= R) return;
    const int r_end = min(R, r_begin + 128);
    const int from = len - n;  // position of the first row
    const int pos_last = from + (r_end - 1) / p.G, pos_first = from + r_begin / p.G;
    const int glo = p.window > 0 && pos_first - p.window + 1 > 0 ? (pos_first - p.window + 1) >> 4 : 0;
    const int ghi = pos_last < 0 ? glo : (pos_last >> 4) + 1;
    const int tiles = ghi > glo ? (ghi - glo + KG - 1) / KG : 0;
    const int steps = ghi > glo ? ((ghi - glo) * 16 + KEYS - 1) / KEYS : 0;

    if (tid == 0) {
        for (int i = 0; i < 2; ++i) {
            mbar_init(kfull + i, kDecodeWarps * 32);
            mbar_init(vfull + i, kDecodeWarps * 32);
            mbar_init(kempty + i, 2 + kPfSoftmaxWarps);
            mbar_init(vempty + i, 2 + kPfSoftmaxWarps);
            mbar_init(sfull + i, 2);
            mbar_init(pfull + i, kPfSoftmaxWarps * 32);
            mbar_init(pdone + i, 2);
            mbar_init(done + i, 1);
            mbar_init(done + 2 + i, 1);
        }
        *abort = 0;
        for (int i = 0; i < NB; ++i) s_bad[2 * i] = 0x7fffffff, s_bad[2 * i + 1] = -1;
        fence_barrier_init();
    }
    if (warp == kPfFirstMma) {
        asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_addr(tslot)), "r"(512u)
                     : "memory");
        asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
    }
    // ---- queries: a warp takes 8 rows, whole rows at a time, the row's largest element in [2^13, 2^14)
    float* const s_top = reinterpret_cast<float*>(smem + SH::oTop);  // [2][parts][128]; before the first step: [7 * 128 + row] scale
    if (warp < kPfSoftmaxWarps) {
        constexpr int LR = D / 4, RL = 32 / LR, NL = 8 / RL;  // lanes of a row, rows of a load, loads
        const int d = 4 * (lane % LR);
        float4 x[NL];
#pragma unroll
        for (int k = 0; k < NL; ++k) {
            const int r = min(r_begin + warp * 8 + k * RL + lane / LR, r_end - 1), i = r / p.G;
            x[k] = ld4(static_cast<const float*>(p.q) + (first + i) * p.q_token + (hk * p.G + r - i * p.G) * p.q_head + d);
        }
        // the K tile's channel order: chunk t of block b holds 32 b + 16 j + 4 t + i
        uint8_t* const to = smem + (d >> 6) * (128 * 128) + 8 * ((d >> 4) & 1);
        const int chunk = 4 * ((d >> 5) & 1) + ((d >> 2) & 3);
#pragma unroll
        for (int k = 0; k < NL; ++k) {
            const int rr = warp * 8 + k * RL + lane / LR;
            float amax = fmaxf(fmaxf(fabsf(x[k].x), fabsf(x[k].y)), fmaxf(fabsf(x[k].z), fabsf(x[k].w)));
#pragma unroll
            for (int m = 1; m < LR; m <<= 1) amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, m));
            const int ex = static_cast<int>(__float_as_uint(amax) >> 23) - 127;
            const int sh = ex == 128 ? 0 : min(13 - ex, 100);
            const float up = copysignf(__uint_as_float(static_cast<uint32_t>(sh + 127) << 23), p.scale);
            const float4 y = make_float4(x[k].x * up, x[k].y * up, x[k].z * up, x[k].w * up);
            const uint2 hi = make_uint2(prompt_pack<false>(y.x, y.y), prompt_pack<false>(y.z, y.w));
            const uint2 lo = make_uint2(prompt_pack<false>(y.x - half_lo(hi.x), y.y - half_hi(hi.x)),
                                        prompt_pack<false>(y.z - half_lo(hi.y), y.w - half_hi(hi.y)));
            uint8_t* const at = to + rr * 128 + ((chunk ^ (rr & 7)) << 4);
            *reinterpret_cast<uint2*>(at) = hi;
            *reinterpret_cast<uint2*>(at + SH::kQ) = lo;
            // not negative: the largest product is the largest logit
            if (lane % LR == 0) s_top[7 * 128 + rr] = fabsf(p.scale) * scalbnf(1.0f, -sh);
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

    if (warp >= kPfFirstMma) {
        // ================================================================ MMA
        prompt_regs<false, kPfMmaRegs>();
        const int b0 = (warp & 1) * (NB / 2);  // its blocks
        if (elect_one() && steps > 0) {
            if (warp < kPfFirstMma + 2) {
                const uint64_t qd = umma_desc_sw128(smem_addr(smem));
                constexpr uint32_t id = prompt_idesc(KEYS, false);
                for (int i = 0; i < steps; ++i) {
                    const int j = i / STEPS, h = i % STEPS, buf = j & 1, sb = i & 1;
                    if (h == 0 && !wait1(kfull + buf, (j >> 1) & 1)) break;
                    if (i >= 2 && !wait1(pdone + sb, ((i >> 1) - 1) & 1)) break;
                    tc_fence_after();
                    const uint64_t kd = umma_desc_sw128(smem_addr(smem + SH::oK + buf * SH::kK + h * (KEYS * 128)));
#pragma unroll
                    for (int e = 0; e < NB / 2; ++e)
#pragma unroll
                        for (int k = 0; k < 4; ++k) {  // the low term's 32 channels, then the high one's
                            const int blk = b0 + e, at = (blk & 1) * 4 + 2 * (k & 1);
                            tc_mma(tmem + SH::cBuf * sb + blk * KEYS, qd + (k < 2 ? SH::kQ / 16 : 0) + (blk >> 1) * (128 * 128 / 16) + at,
                                   kd + (blk >> 1) * (KT * 128 / 16) + at, id, k > 0);
                        }
                    tc_commit(sfull + sb);
                    if (h == STEPS - 1) tc_commit(kempty + buf);
                }
            } else {
                constexpr uint32_t id = prompt_idesc(32, true);
                for (int i = 0; i < steps; ++i) {
                    const int j = i / STEPS, h = i % STEPS, buf = j & 1, sb = i & 1;
                    if (h == 0 && !wait1(vfull + buf, (j >> 1) & 1)) break;
                    if (!wait1(pfull + sb, (i >> 1) & 1)) break;
                    tc_fence_after();
                    // atoms of 64 keys; a step starts at its first or its 33rd
                    const uint64_t vd = umma_desc_sw128(smem_addr(smem + SH::oV + buf * SH::kV + (h * KEYS / 64) * (D * 128))) +
                                        (KEYS == 32 ? 4 * (h & 1) : 0);
#pragma unroll
                    for (int e = 0; e < NB / 2; ++e)
#pragma unroll
                        for (int term = 2; term >= 0; --term)
#pragma unroll
                            for (int k = 0; k < KS; ++k) {
                                const int blk = b0 + e;
                                tc_mma_ts(tmem + SH::cO + 32 * blk,
                                          tmem + SH::cBuf * sb + PC * k + (3 * blk + term) * 8,
                                          vd + blk * (32 * 128 / 16) + 2 * k, id, h > 0 || term < 2 || k > 0);
                            }
                    tc_commit(pdone + sb);
                    if (h == STEPS - 1) tc_commit(vempty + buf);
                }
            }
            tc_commit(done + warp - kPfFirstMma);
            mbar_wait(done + warp - kPfFirstMma, 0);  // every MMA has ended before tensor memory goes
        }
    } else if (warp >= kPfSoftmaxWarps) {
        // ================================================================ packed blobs -> operand tiles and scales
        prompt_regs<false, kPfDecodeRegs>();
        const int cw = warp - kPfSoftmaxWarps, g8 = lane >> 2, t4 = lane & 3, gpp = p.page >> 4;
        constexpr int kKB = kv_blob_bytes(K4, D), kVB = kv_blob_bytes(V4, D);
        static_assert(KG == kDecodeWarps, "a warp takes one group of a tile's keys");
        constexpr int KL = K4 ? D / 64 : D / 32, VB = NB / 2;  // 16-byte words of a lane; blocks of values of a warp
        const int pair = cw & 3, b0 = (cw >> 2) * VB;           // values: two neighbouring groups, half the blocks
        // blobs of the tile's groups, one a lane
        const auto locate = [&](int j) {
            const int g = glo + j * KG + (lane & (KG - 1));
            int64_t at = -1;
            if (j < tiles && g < ghi) {
                int pg = p.table[b * p.table_stride + g / gpp];
                if (pg < 0 || pg >= p.n_pages) {
                    set_error(p.err, DEV_ERR_BAD_PLACE);
                    pg = 0;
                }
                at = (static_cast<int64_t>(pg) * p.Hkv + hk) * gpp + g % gpp;
            }
            return at;
        };
        uint4 kq[KL], vq[2][VB];  // a block of values: four words of bytes, or two of nibbles
        uint32_t ks[2] = {0u, 0u}, vs = 0u;  // scales: block t4 of tokens g8, 8 + g8; the values' blocks of one key
        const auto load_k = [&](int64_t blobs) {
            const int64_t at = __shfl_sync(0xffffffffu, blobs, cw);
            if (at < 0) return;  // past the last key: the tile keeps what it held, every row masks it
            const uint8_t* const src = p.k + at * kKB;
#pragma unroll
            for (int i = 0; i < KL; ++i) kq[i] = __ldg(reinterpret_cast<const uint4*>(src + (i * 32 + lane) * 16));
            const uint16_t* const sc = reinterpret_cast<const uint16_t*>(src + kv_quant_bytes(K4, D)) + g8 * NB + (t4 & (NB - 1));
            ks[0] = __ldg(sc), ks[1] = __ldg(sc + 8 * NB);
        };
        const auto load_v = [&](int64_t blobs) {
            const int64_t mine = __shfl_sync(0xffffffffu, blobs, 2 * pair + (g8 >> 2));
            vs = 0u;
            if (mine >= 0) {  // key 8 o + 2 t + e of group c, lane 16 c + 8 o + 4 e + t
                const uint16_t* const sc = reinterpret_cast<const uint16_t*>(p.v + mine * kVB + kv_quant_bytes(V4, D)) +
                                           (8 * ((g8 >> 1) & 1) + 2 * t4 + (g8 & 1)) * NB + b0;
                vs = VB == 2 ? __ldg(reinterpret_cast<const uint32_t*>(sc)) : static_cast<uint32_t>(__ldg(sc));
            }
#pragma unroll
            for (int c = 0; c < 2; ++c) {
                const int64_t at = __shfl_sync(0xffffffffu, blobs, 2 * pair + c);
                const uint8_t* const src = p.v + at * kVB;
#pragma unroll
                for (int i = 0; i < VB; ++i) {
                    const int blk = b0 + i;
                    vq[c][i] = make_uint4(0u, 0u, 0u, 0u);
                    if (at < 0) continue;
                    if constexpr (V4) {
                        const uint2 u = __ldg(reinterpret_cast<const uint2*>(src + ((blk >> 1) * 32 + lane) * 16 + (blk & 1) * 8));
                        vq[c][i].x = u.x, vq[c][i].y = u.y;
                    } else {
                        vq[c][i] = __ldg(reinterpret_cast<const uint4*>(src + (blk * 32 + lane) * 16));
                    }
                }
            }
        };
        int64_t blobs = locate(0), next = locate(1);
        if (tiles > 0) {
            load_k(blobs);
            load_v(blobs);
        }
        // the row of this lane's token o in a tile: 32 (group / 2) + 8 (g / 2) + 4 (group % 2) + 2 o + g % 2
        const int k_low = 4 * (cw & 1) + (g8 & 1), k_row = 32 * (cw >> 1) + 8 * (g8 >> 1) + k_low;
        for (int j = 0; j < tiles; ++j) {
            const int buf = j & 1;
            blobs = next;
            next = locate(j + 2);
            // ---- keys: lane (g, t) writes chunk t of each block of its token's row
            if (j >= 2 && !wait(kempty + buf, ((j >> 1) - 1) & 1)) break;
            uint8_t* const kt = smem + SH::oK + buf * SH::kK + k_row * 128;
            float* const sk = reinterpret_cast<float*>(smem + SH::oSK + buf * SH::kS);
#pragma unroll
            for (int i = 0; i < KL; ++i) {
                const uint32_t w[4] = {kq[i].x, kq[i].y, kq[i].z, kq[i].w};
#pragma unroll
                for (int q = 0; q < 4; q += K4 ? 1 : 2) {  // a chunk: one word of 8 nibbles or two of 4 bytes
                    const int f = 4 * i + q, per = K4 ? NB : D / 16, o = f / per, blk = K4 ? f % per : (f % per) >> 1;
                    uint32_t h[4];
                    if constexpr (K4) {
                        prompt_ints4(w[q], h);
                    } else {
                        uint32_t a[2], e[2];
                        prompt_ints8(w[q], a);
                        prompt_ints8(w[q + 1 < 4 ? q + 1 : 3], e);
                        h[0] = a[0], h[1] = a[1], h[2] = e[0], h[3] = e[1];
                    }
                    *reinterpret_cast<uint4*>(kt + o * 256 + (blk >> 1) * (KT * 128) + (((4 * (blk & 1) + t4) ^ (k_low + 2 * o)) << 4)) =
                        make_uint4(h[0], h[1], h[2], h[3]);
                }
            }
            if (t4 < NB) sk[t4 * KT + k_row] = pf_half(ks[0]), sk[t4 * KT + k_row + 2] = pf_half(ks[1]);
            load_k(blobs);
            fence_proxy_async_smem();
            mbar_arrive(kfull + buf);
            // ---- values: the scales of whatever lies past the sequence's end count as 0
            if (j >= 2 && !wait(vempty + buf, ((j >> 1) - 1) & 1)) break;
            const int place = 32 * pair + 8 * t4 + g8;
            const int key = 16 * (glo + j * KG + 2 * pair + (g8 >> 2)) + 8 * ((g8 >> 1) & 1) + 2 * t4 + (g8 & 1);
            float* const sv = reinterpret_cast<float*>(smem + SH::oSV + buf * SH::kS);
#pragma unroll
            for (int i = 0; i < VB; ++i) {
                float x = key < len ? pf_half(vs >> (16 * i)) : 0.0f;
                if (!(fabsf(x) <= 65504.0f)) {  // 0 here, and the rows that see it are told
                    atomicMin(s_bad + 2 * (b0 + i), key), atomicMax(s_bad + 2 * (b0 + i) + 1, key);
                    x = 0.0f;
                }
                sv[(b0 + i) * KT + place] = x;
            }
            // lane (g, t) writes 8 keys of both groups as one chunk of channel 8 n + g
            uint8_t* const vt = smem + SH::oV + buf * SH::kV + (pair >> 1) * (D * 128) + (32 * b0 + g8) * 128 +
                                (((4 * (pair & 1) + t4) ^ g8) << 4);
#pragma unroll
            for (int i = 0; i < VB; ++i) {
                const uint32_t w0[4] = {vq[0][i].x, vq[0][i].y, vq[0][i].z, vq[0][i].w};
                const uint32_t w1[4] = {vq[1][i].x, vq[1][i].y, vq[1][i].z, vq[1][i].w};
#pragma unroll
                for (int q = 0; q < (V4 ? 2 : 4); ++q) {
                    if constexpr (V4) {
                        uint32_t x[4], y[4];
                        pf_nibbles(w0[q], x);
                        pf_nibbles(w1[q], y);
#pragma unroll
                        for (int k = 0; k < 2; ++k)  // even and odd eights of channels
                            *reinterpret_cast<uint4*>(vt + (4 * i + 2 * q + k) * (8 * 128)) = make_uint4(x[k], x[2 + k], y[k], y[2 + k]);
                    } else {
                        uint32_t x[2], y[2];
                        pf_bytes(w0[q], x);
                        pf_bytes(w1[q], y);
                        *reinterpret_cast<uint4*>(vt + (4 * i + q) * (8 * 128)) = make_uint4(x[0], x[1], y[0], y[1]);
                    }
                }
            }
            load_v(blobs);
            fence_proxy_async_smem();
            mbar_arrive(vfull + buf);
        }
    } else {
        // ================================================================ softmax: four threads a row
        prompt_regs<true, kPfSoftmaxRegs>();
        const int rr = tid & 127, part = tid >> 7, r = min(r_begin + rr, r_end - 1);
        const uint32_t lanes = static_cast<uint32_t>((warp & 3) * 32) << 16;
        const uint32_t cs = tmem + lanes, co = tmem + SH::cO + part * HD + lanes;
        const int i_row = r / p.G, h = hk * p.G + r - i_row * p.G, pos = from + i_row;
        const int first_key = p.window > 0 ? pos - p.window + 1 : 0;
        const float rscale = s_top[7 * 128 + rr];
        const bool plain = p.cap <= 0.0f && !p.slopes && rscale > 0.0f;
        constexpr float kLog2e = 1.44269504088896340736f;
        const float slope = p.slopes ? p.slopes[h] * kLog2e : 0.0f;
        const float sx = p.cap > 0.0f ? rscale : rscale * kLog2e, mul = plain ? sx : 1.0f;
        // steps that every row of the tile sees whole
        const int seen_from = p.window > 0 ? pos_last - p.window + 1 : 0;
        float tot[HD], m = -1e30f, l = 0.0f;
#pragma unroll
        for (int k = 0; k < HD; ++k) tot[k] = 0.0f;
        // adds the sums in tensor memory to the totals, or (SCALE) multiplies them by the row's factor where
        // they are, which is 1 for rows that others of the warp take along: a row's roundings are its own
        const auto fold = [&](auto SCALE, int last, float a) {
            wait(pdone + (last & 1), (last >> 1) & 1);
            tc_fence_after();
#pragma unroll
            for (int c = 0; c < HD; c += 16) {
                float o[16];
                pf_ld8(co + c, o);
                pf_ld8(co + c + 8, o + 8);
                prompt_wait_ld();
                pf_tie8(o);
                pf_tie8(o + 8);
                if constexpr (SCALE.value) {
                    uint32_t scaled[16];
#pragma unroll
                    for (int k = 0; k < 16; ++k) scaled[k] = __float_as_uint(o[k] * a);
                    pf_st8(co + c, scaled);
                    pf_st8(co + c + 8, scaled + 8);
                } else {
#pragma unroll
                    for (int k = 0; k < 16; k += 2) add2(tot[c + k], tot[c + k + 1], tot[c + k], tot[c + k + 1], o[k], o[k + 1]);
                }
            }
        };
        // A wait that gave up does not leave the loop: the other warps of the rows wait at their barrier.
        for (int i = 0; i < steps; ++i) {
            const int j = i / STEPS, at = (i % STEPS) * KEYS + part * HK, buf = j & 1, sb = i & 1;
            if (i % STEPS == 0) wait(kfull + buf, (j >> 1) & 1);
            wait(sfull + sb, (i >> 1) & 1);
            tc_fence_after();
            const int key0 = 16 * glo + i * KEYS, mine = key0 + (KEYS == 32 ? 2 * part : 32 * (part >> 1) + 4 * (part & 1));
            const bool whole = key0 + KEYS - 1 <= pos_first && key0 >= seen_from;
            float x[HK];
            const float* const sk = reinterpret_cast<const float*>(smem + SH::oSK + buf * SH::kS) + at;
#pragma unroll
            for (int b2 = 0; b2 < NB; b2 += 2) {  // two blocks at a time
                float s[2 * HK];
#pragma unroll
                for (int k = 0; k < 2 * HK; k += 8)
                    pf_ld8(cs + SH::cBuf * sb + (b2 + k / HK) * KEYS + part * HK + k % HK, s + k);
                prompt_wait_ld();
#pragma unroll
                for (int k = 0; k < 2 * HK; k += 8) pf_tie8(s + k);
#pragma unroll
                for (int blk = b2; blk < b2 + 2; ++blk)
#pragma unroll
                    for (int k = 0; k < HK; k += 4) {
                        const float4 d = *reinterpret_cast<const float4*>(sk + blk * KT + k);
                        const float* const y = s + (blk - b2) * HK + k;
                        if (blk == 0) {
                            mul2(x[k], x[k + 1], y[0], y[1], d.x, d.y);
                            mul2(x[k + 2], x[k + 3], y[2], y[3], d.z, d.w);
                        } else {
                            ffma2p(x[k], x[k + 1], y[0], y[1], d.x, d.y, x[k], x[k + 1]);
                            ffma2p(x[k + 2], x[k + 3], y[2], y[3], d.z, d.w, x[k + 2], x[k + 3]);
                        }
                    }
            }
            if (i % STEPS == STEPS - 1) {
                __syncwarp();
                if (lane == 0) mbar_arrive(kempty + buf);
            }
            // logits in units of log2 (plain: still to be multiplied by sx)
            constexpr auto key_at = [](int k) { return 16 * ((k >> 2) & 1) + 8 * ((k >> 1) & 1) + 2 * (k >> 3) + (k & 1); };
            if (!plain) {
                const float rel = static_cast<float>(mine - pos);
#pragma unroll
                for (int k = 0; k < HK; ++k) {
                    float y = x[k] * sx;
                    if (p.cap > 0.0f) y = kLog2e * (p.cap * tanhf(y / p.cap));
                    x[k] = fmaf(slope, rel + static_cast<float>(key_at(k)), y);
                }
            }
            if (!whole) {
#pragma unroll
                for (int k = 0; k < HK; ++k)
                    if (mine + key_at(k) > pos || mine + key_at(k) < first_key) x[k] = -INFINITY;
            }
            float tops[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
#pragma unroll
            for (int k = 0; k < HK; ++k) tops[k & 3] = fmaxf(tops[k & 3], x[k]);
            float top = fmaxf(fmaxf(tops[0], tops[1]), fmaxf(tops[2], tops[3])) * mul;
            s_top[(sb * kPfParts + part) * 128 + rr] = top;
            tc_fence_before();  // all of the rows' scores are read before probabilities go over them
            pf_rows_sync(warp & 3);
            tc_fence_after();
#pragma unroll
            for (int k = 0; k < kPfParts; ++k) top = fmaxf(top, s_top[(sb * kPfParts + k) * 128 + rr]);
            const bool raise = top > m + 8.0f, raised = __any_sync(0xffffffffu, raise), fresh = i % STEPS == 0;
            float a = 1.0f;
            if (raise) {
                a = prompt_ex2(m - top);
                m = top;
                l *= a;
            }
            float sum[4] = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
            for (int k = 0; k < HK; k += 2) {
                ffma2(x[k], x[k + 1], x[k], x[k + 1], mul, -m, -m);
                x[k] = prompt_ex2(x[k]);
                x[k + 1] = prompt_ex2(x[k + 1]);
                add2(sum[k & 2], sum[(k & 2) + 1], sum[k & 2], sum[(k & 2) + 1], x[k], x[k + 1]);
            }
            l += (sum[0] + sum[1]) + (sum[2] + sum[3]);
            if (i % STEPS == 0) wait(vfull + buf, (j >> 1) & 1);
            const float* const sv = reinterpret_cast<const float*>(smem + SH::oSV + buf * SH::kS) + at;
#pragma unroll
            for (int blk = 0; blk < NB; ++blk) {
                uint32_t w[3 * HK / 2];  // a block's terms
#pragma unroll
                for (int k = 0; k < HK; k += 4) {
                    const float4 d = *reinterpret_cast<const float4*>(sv + blk * KT + k);
                    float y[4];
                    mul2(y[0], y[1], x[k], x[k + 1], d.x, d.y);
                    mul2(y[2], y[3], x[k + 2], x[k + 3], d.z, d.w);
#pragma unroll
                    for (int z = 0; z < 4; z += 2)
#pragma unroll
                        for (int term = 0; term < 3; ++term) {
                            const uint32_t u = prmt(__float_as_uint(y[z]), __float_as_uint(y[z + 1]), 0x7632u);
                            w[term * (HK / 2) + (k + z) / 2] = u;
                            if (term < 2)
                                ffma2(y[z], y[z + 1], __uint_as_float(u << 16), __uint_as_float(u & 0xFFFF0000u), -1.0f, y[z], y[z + 1]);
                        }
                }
#pragma unroll
                for (int term = 0; term < 3; ++term) {
                    const uint32_t to = cs + SH::cBuf * sb + (3 * blk + term) * 8;
                    if constexpr (HK == 16) pf_st8(to + PC * part, w + 8 * term);
                    else pf_st4(to + PC * (part >> 1) + 4 * (part & 1), w + 4 * term);
                }
            }
            if (i % STEPS == STEPS - 1) {
                __syncwarp();
                if (lane == 0) mbar_arrive(vempty + buf);
            }
            if (i > 0 && (raised || fresh)) {
                if (fresh) fold(std::false_type{}, i - 1, 1.0f);
                else fold(std::true_type{}, i - 1, a);
                if (raised) {
#pragma unroll
                    for (int k = 0; k < HD; ++k) tot[k] *= a;
                }
            }
            tmem_wait_st();
            tc_fence_before();
            mbar_arrive(pfull + sb);
        }
        // ---- output rows
        if (steps > 0) fold(std::false_type{}, steps - 1, 1.0f);
        s_top[part * 128 + rr] = l;
        pf_rows_sync(warp & 3);
        l = (s_top[rr] + s_top[128 + rr]) + (s_top[256 + rr] + s_top[384 + rr]);
        const float inv = l > 0.0f || l != l ? 1.0f / l : 0.0f;
        if (r_begin + rr < r_end) {
            float* const out = static_cast<float*>(p.out) + (first + i_row) * p.out_token + h * p.out_head + part * HD;
            // an infinite or NaN value among those that the row sees
            const float f = prompt_spoilt<V4, D>(p, s_bad, b, hk, part * HD / 32, first_key, pos) ? NAN : inv;
#pragma unroll
            for (int k = 0; k < HD; k += 4)
                *reinterpret_cast<float4*>(out + k) = make_float4(tot[k] * f, tot[k + 1] * f, tot[k + 2] * f, tot[k + 3] * f);
        }
    }
    tc_fence_before();
    __syncthreads();
    if (warp == kPfFirstMma) {
        tc_fence_after();
        asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(512u) : "memory");
    }
}

template <bool K4, bool V4, int D>
cudaError_t launch_attn_promptf_one(const AttnParams& p, cudaStream_t s) {
    using SH = PromptfShape<D>;
    static_assert(SH::kTotal <= kSmemLimit, "shared memory");
    static std::atomic<bool> set[kMaxDevices] = {};
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    if (dev < 0 || dev >= kMaxDevices) return cudaErrorInvalidDevice;
    if (!set[dev].load(std::memory_order_acquire)) {
        cudaFuncAttributes at;
        e = cudaFuncGetAttributes(&at, k_attn_promptf<K4, V4, D>);
        if (e != cudaSuccess) return e;
        if (at.numRegs != kPfLaunchRegs) return cudaErrorInvalidConfiguration;  // the split would not add up
        e = cudaFuncSetAttribute(k_attn_promptf<K4, V4, D>, cudaFuncAttributeMaxDynamicSharedMemorySize, SH::kTotal);
        if (e != cudaSuccess) return e;
        set[dev].store(true, std::memory_order_release);
    }
    const int64_t tiles = (static_cast<int64_t>(p.max_q) * p.G + 127) / 128;
    return launch_pdl(k_attn_promptf<K4, V4, D>,
                      dim3(static_cast<unsigned>(p.n_seqs * p.Hkv), static_cast<unsigned>(tiles)), dim3(kPfThreads),
                      SH::kTotal, s, p);
}

template <int D>
cudaError_t launch_attn_promptf_dim(const AttnParams& p, cudaStream_t s) {
    if (p.k_q4) return p.v_q4 ? launch_attn_promptf_one<true, true, D>(p, s) : launch_attn_promptf_one<true, false, D>(p, s);
    return p.v_q4 ? launch_attn_promptf_one<false, true, D>(p, s) : launch_attn_promptf_one<false, false, D>(p, s);
}

}  // namespace ggq
