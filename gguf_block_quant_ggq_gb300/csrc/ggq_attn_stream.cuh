// ggq_attn_stream.cuh -- attention for few query rows per kv head: a stream
// over the packed cache on mma.sync.
//
// Mathematics: with the blocks' quants u (stored + 128 or + 8), scales d and
// query row q, s_j = sum_b dk_jb sum_{c in b} q_c (u_jc - off) and out_c = sum_j
// p_j dv_jb (u_jc - off) / sum_j p_j.  The matrix instruction multiplies query
// rows (16) by the integer quants, which fp16 holds exactly; the scales are
// applied to its fp32 results (scores) and to the probabilities (values), so the
// packed bytes are unpacked but never dequantized.
//   * Scores: two k16 steps per block of 32 channels.  The quants enter as fp16
//     subnormals u 2^-24 (a byte permutation, no arithmetic); the accumulator
//     starts at -off 2^-24 sum_c q_c, which takes the offset out again.
//   * Values: quants as exact signed fp16 integers; the other operand is p dv
//     times a power of two that keeps it in fp16's normal range.
//   * fp32 activations: 8 query rows; a 16-row operand holds the high and low
//     fp16 halves of each (22 bits), whose results add up.  16-bit activations:
//     8 or 16 rows in one fp16 operand (16-bit queries are exact in it).
//   * Softmax statistics are fp32.  Within a group of 16 keys the probabilities
//     are relative to the group's maximum, and the value scales are lifted by a
//     power of two that keeps p dv below fp16's range (the second half is lifted by
//     2^12 more); a group's result is added to the fp32 totals with its factor
//     2^(group maximum - reference).  No sum runs longer than a group on the tensor
//     cores (which truncate), no probability is lost for being small (those of a group
//     that lie more than 2^28 apart take a pass each), and the totals are rescaled only when the reference rises by 2^60.
//
// Bound by HBM: every attended blob is read once (17 or 9 bytes per 16
// channels).  Work is cut in equal shares of 16-token groups over all CTAs,
// whatever the lengths; a CTA walks its share item by item (an item is one
// sequence, kv head and tile of rows), its four consumer warps take every
// fourth group, and a producer warp keeps a ring of bulk copies in flight for
// each of them, across items.  An item that several CTAs share is joined by the
// last of them from partial results in scratch, in the order of the pieces.
#pragma once
#include "ggq_attn.cuh"
#include "ggq_device.cuh"
#include "ggq_internal.h"

namespace ggq {

constexpr int kAttnWarps = 4;                          // consumer warps
constexpr int kAttnThreads = (kAttnWarps + 1) * 32;    // and the producer
constexpr float kAttnNone = -1e30f;                    // reference maximum of a row that has seen nothing

// fp32 rows (high and low halves), 8 rows or 16 rows of 16-bit activations
enum AttnMode : int { A_SPLIT8 = 0, A_HALF8 = 1, A_HALF16 = 2 };

template <bool K4, bool V4, int D, int MODE>
struct AttnSmem {
    static constexpr int kRows = MODE == A_HALF16 ? 16 : 8;
    static constexpr int kKB = kv_blob_bytes(K4, D), kVB = kv_blob_bytes(V4, D);
    static constexpr int kStage = kKB + kVB;
    static constexpr int kStages = (kStage <= 2304 ? 8 : kStage <= 4352 ? 5 : 3);
    static constexpr int kRowPitch = D + 8;            // floats of a totals row (padding: conflict-free float2 stores)
    static constexpr int oRing = 0;
    static constexpr int oTot = kAttnWarps * kStages * kStage;
    static constexpr int oQ = oTot + kAttnWarps * kRows * kRowPitch * 4;
    static constexpr int oStat = oQ + D / 16 * 32 * 16;   // m, l [warps][rows]
    static constexpr int oScan = (oStat + 2 * kAttnWarps * kRows * 4 + 7) / 8 * 8;
    static constexpr int oBar = (oScan + (128 + 4) * 8 + 15) / 16 * 16;
    static constexpr int kTotal = oBar + 2 * kAttnWarps * kStages * 8 + 16;
    static constexpr int kCtas = 2 * kTotal <= kSmemLimit ? 2 : 1;  // per SM
};

// One sequence as the plan sees it.
struct AttnSeq {
    int len, rows, first;  // cached tokens, new tokens, first row of q
    int glo, ghi;          // 16-token groups that some row sees
    int items;             // kv heads x row tiles
};

__device__ __forceinline__ AttnSeq attn_seq(const AttnParams& p, int b, int tile_rows, bool report) {
    AttnSeq s;
    s.len = p.lens[b];
    s.first = b;
    int end = b + 1;
    if (p.q_start) {
        s.first = p.q_start[b];
        end = p.q_start[b + 1];
    }
    bool bad = false;
    if (s.first < 0 || end > p.n_tokens || s.first > end) {
        s.first = end = 0;
        bad = true;
    }
    s.rows = end - s.first;
    if (s.rows > p.max_q) bad = true;
    if (s.len > p.max_len || s.len < 0) {
        s.len = s.len < 0 ? 0 : p.max_len;
        bad = true;
    }
    if (bad && report) set_error(p.err, DEV_ERR_BAD_PLACE);
    s.glo = 0;
    const int from = s.len - s.rows;  // position of the first row
    if (p.window > 0 && from - p.window + 1 > 0) s.glo = (from - p.window + 1) >> 4;
    s.ghi = (s.len + 15) >> 4;
    const int shown = min(s.rows, p.max_q);
    s.items = p.Hkv * ((shown * p.G + tile_rows - 1) / tile_rows);
    if (s.items == 0) s.ghi = s.glo = 0;
    return s;
}
__device__ __forceinline__ int64_t attn_cost(const AttnSeq& s) { return static_cast<int64_t>(s.ghi - s.glo) * s.items; }

// A CTA's share, item by item.
struct AttnWalk {
    AttnSeq s;
    int b, item, ga;
    int64_t left;  // groups of the share that are not yet walked
    __device__ __forceinline__ int gb() const {  // end of the current segment
        const int64_t e = ga + left;
        return e < s.ghi ? static_cast<int>(e) : s.ghi;
    }
    __device__ __forceinline__ void next(const AttnParams& p, int tile_rows) {
        left -= gb() - ga;
        if (left <= 0) return;
        if (++item == s.items) {
            item = 0;
            do s = attn_seq(p, ++b, tile_rows, false); while (attn_cost(s) == 0);
        }
        ga = s.glo;
    }
};

__device__ __forceinline__ void attn_mma(float (&c)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
        : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
__device__ __forceinline__ float ex2(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}
__device__ __forceinline__ uint32_t pack_h2(float lo, float hi) {
    uint32_t r;
    asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
    return r;
}
__device__ __forceinline__ uint32_t h2_sub(uint32_t a, uint32_t b) {
    const __half2 r = __hsub2(*reinterpret_cast<const __half2*>(&a), *reinterpret_cast<const __half2*>(&b));
    return *reinterpret_cast<const uint32_t*>(&r);
}
__device__ __forceinline__ uint32_t h2_fma(uint32_t a, uint32_t b, uint32_t c) {
    const __half2 r = __hfma2(*reinterpret_cast<const __half2*>(&a), *reinterpret_cast<const __half2*>(&b),
                              *reinterpret_cast<const __half2*>(&c));
    return *reinterpret_cast<const uint32_t*>(&r);
}
// (d0, d1) = (a0, a1) * b + (c0, c1) in one instruction
__device__ __forceinline__ void fma2(float& d0, float& d1, float a0, float a1, float b, float c0, float c1) {
    asm("{\n\t.reg .b64 x, y, z;\n\tmov.b64 x, {%2, %3};\n\tmov.b64 y, {%4, %4};\n\tmov.b64 z, {%5, %6};\n\t"
        "fma.rn.f32x2 x, x, y, z;\n\tmov.b64 {%0, %1}, x;\n\t}"
        : "=f"(d0), "=f"(d1)
        : "f"(a0), "f"(a1), "f"(b), "f"(c0), "f"(c1));
}
__device__ __forceinline__ float pow2f(int e) { return __uint_as_float(static_cast<uint32_t>(e + 127) << 23); }
__device__ __forceinline__ float quad_sum(float v) {
    v += __shfl_xor_sync(0xffffffffu, v, 1);
    return v + __shfl_xor_sync(0xffffffffu, v, 2);
}
__device__ __forceinline__ float quad_max(float v) {
    v = fmaxf(v, __shfl_xor_sync(0xffffffffu, v, 1));
    return fmaxf(v, __shfl_xor_sync(0xffffffffu, v, 2));
}

template <typename T>
__device__ __forceinline__ const T* attn_q_row(const AttnParams& p, const AttnSeq& s, int hk, int r) {
    const int i = r / p.G, h = hk * p.G + r - i * p.G;
    return static_cast<const T*>(p.q) + (s.first + i) * p.q_token + h * p.q_head;
}
__device__ __forceinline__ float4 attn_q4(const AttnParams& p, const AttnSeq& s, int hk, int r, int d) {
    if (p.dtype == 0) return ld4(attn_q_row<float>(p, s, hk, r) + d);
    if (p.dtype == 1) return ld4(attn_q_row<__half>(p, s, hk, r) + d);
    return ld4(attn_q_row<__nv_bfloat16>(p, s, hk, r) + d);
}
__device__ __forceinline__ void attn_out4(const AttnParams& p, const AttnSeq& s, int hk, int r, int d, float4 v) {
    const int i = r / p.G, h = hk * p.G + r - i * p.G;
    const int64_t at = (s.first + i) * p.out_token + h * p.out_head + d;
    if (p.dtype == 0) st4(static_cast<float*>(p.out) + at, v);
    else if (p.dtype == 1) st4(static_cast<__half*>(p.out) + at, v);
    else st4(static_cast<__nv_bfloat16*>(p.out) + at, v);
}

// Position of the share [lo, ...) in the list of all groups: the runs' exclusive
// prefix sums in s_scan (128), each run `per` sequences.
__device__ __forceinline__ AttnWalk attn_find(const AttnParams& p, const int64_t* s_scan, int per, int64_t lo, int64_t n,
                                              int tile_rows, int lane) {
    int run = -1;
#pragma unroll
    for (int k = 0; k < 4; ++k) run += __popc(__ballot_sync(0xffffffffu, s_scan[lane + 32 * k] <= lo));
    AttnWalk w;
    w.left = n;
    w.b = run * per;
    int64_t rem = lo - s_scan[run];
    for (;;) {
        w.s = attn_seq(p, w.b, tile_rows, false);
        const int64_t c = attn_cost(w.s);
        if (rem < c) break;
        rem -= c;
        ++w.b;
    }
    const int ng = w.s.ghi - w.s.glo;
    w.item = static_cast<int>(rem / ng);
    w.ga = w.s.glo + static_cast<int>(rem - static_cast<int64_t>(w.item) * ng);
    return w;
}

__device__ __forceinline__ void consumer_sync() { asm volatile("bar.sync 1, %0;" ::"n"(kAttnWarps * 32) : "memory"); }

template <bool K4, bool V4, int D, int MODE>
__global__ void __launch_bounds__(kAttnThreads, AttnSmem<K4, V4, D, MODE>::kCtas)
    k_attn_stream(const __grid_constant__ AttnParams p) {
    using SM = AttnSmem<K4, V4, D, MODE>;
    constexpr int kRows = SM::kRows, NB = D / 32, KS = D / 16, NT = D / 8, S = SM::kStages;
    constexpr bool TWO = MODE == A_HALF16;  // operand rows 8..15 are query rows of their own
    constexpr int RS = TWO ? 2 : 1;
    extern __shared__ __align__(128) uint8_t smem[];
    float* const s_tot = reinterpret_cast<float*>(smem + SM::oTot);
    uint4* const s_q = reinterpret_cast<uint4*>(smem + SM::oQ);
    float* const s_m = reinterpret_cast<float*>(smem + SM::oStat);
    float* const s_l = s_m + kAttnWarps * kRows;
    int64_t* const s_scan = reinterpret_cast<int64_t*>(smem + SM::oScan);
    int64_t* const s_wsum = s_scan + 128;
    uint64_t* const s_full = reinterpret_cast<uint64_t*>(smem + SM::oBar);
    uint64_t* const s_empty = s_full + kAttnWarps * S;
    volatile int* const s_abort = reinterpret_cast<volatile int*>(s_empty + kAttnWarps * S);
    volatile int* const s_last = s_abort + 1;
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;

    pdl_launch_dependents();
    if (tid == 0) {
        for (int i = 0; i < kAttnWarps * S; ++i) {
            mbar_init(s_full + i, 1);
            mbar_init(s_empty + i, 1);
        }
        *s_abort = 0;
        fence_barrier_init();
    }
    pdl_wait();

    // ---- plan: prefix sums of the sequences' costs over 128 runs of `per` sequences
    const int nseq = static_cast<int>(p.n_seqs), per = (nseq + 127) >> 7;
    int64_t mine = 0, incl = 0;
    if (tid < 128) {
        for (int b = tid * per; b < min(nseq, (tid + 1) * per); ++b) {
            const AttnSeq s = attn_seq(p, b, kRows, blockIdx.x == 0);
            const int64_t cost = attn_cost(s);
            mine += cost;
            if (cost == 0 && b % static_cast<int>(gridDim.x) == static_cast<int>(blockIdx.x)) {
                for (int r = 0; r < min(s.rows, p.max_q) * p.H; ++r)  // nothing cached: zeros
                    for (int d = 0; d < D; d += 4)
                        attn_out4(p, s, (r % p.H) / p.G, (r / p.H) * p.G + (r % p.H) % p.G, d, make_float4(0.f, 0.f, 0.f, 0.f));
            }
        }
        incl = mine;
#pragma unroll
        for (int d = 1; d < 32; d <<= 1) {
            const int64_t y = __shfl_up_sync(0xffffffffu, incl, d);
            if (lane >= d) incl += y;
        }
        if (lane == 31) s_wsum[warp] = incl;
    }
    __syncthreads();
    if (tid < 128) {
        int64_t base = 0;
        for (int w = 0; w < warp; ++w) base += s_wsum[w];
        s_scan[tid] = base + incl - mine;
    }
    __syncthreads();
    const int64_t N = s_wsum[0] + s_wsum[1] + s_wsum[2] + s_wsum[3];
    const int64_t want = (N + p.min_share - 1) / p.min_share;
    const int C = static_cast<int>(want < gridDim.x ? want : gridDim.x);  // CTAs that get a share (N >= C)
    const int c = static_cast<int>(blockIdx.x);
    if (c >= C) return;
    const int64_t lo = N * c / C, hi = N * (c + 1) / C;
    AttnWalk w = attn_find(p, s_scan, per, lo, hi - lo, kRows, lane);

    if (warp == kAttnWarps) {
        // ---- producer: lane l fills consumer l's ring, a round of four groups at a time
        const uint64_t policy = policy_evict_first();
        const int gpp = p.page >> 4;
        int n = 0, base = w.ga;
        const auto page_of = [&](const AttnWalk& x, int g) {
            int pg = 0;
            if (lane < kAttnWarps && g < x.gb()) {
                pg = p.table[x.b * p.table_stride + g / gpp];
                if (pg < 0 || pg >= p.n_pages) {
                    set_error(p.err, DEV_ERR_BAD_PLACE);
                    pg = 0;
                }
            }
            return pg;
        };
        int pg = page_of(w, base + lane);
        bool ok = true;
        while (w.left > 0) {
            const int g = base + lane, gb = w.gb(), hk = w.item / (w.s.items / p.Hkv);
            const bool mine_g = lane < kAttnWarps && g < gb;
            const int pg_now = pg;
            base += kAttnWarps;
            if (base >= gb) {
                w.next(p, kRows);
                base = w.ga;
            }
            if (w.left > 0) pg = page_of(w, base + lane);  // on its way while this round waits for room
            if (mine_g) {
                const int slot = n % S, at = lane * S + slot;
                if (n >= S) ok = !*s_abort && mbar_wait(s_empty + at, ((n / S) - 1) & 1);
                if (ok) {
                    const int64_t blob = (static_cast<int64_t>(pg_now) * p.Hkv + hk) * gpp + g % gpp;
                    uint8_t* const dst = smem + SM::oRing + at * SM::kStage;
                    mbar_arrive_expect_tx(s_full + at, SM::kStage);
                    bulk_g2s(dst, p.k + blob * SM::kKB, SM::kKB, s_full + at, policy);
                    bulk_g2s(dst + SM::kKB, p.v + blob * SM::kVB, SM::kVB, s_full + at, policy);
                    ++n;
                }
            }
            if (!__all_sync(0xffffffffu, ok)) break;
        }
        if (!__all_sync(0xffffffffu, ok)) {
            *s_abort = 1;
            set_error(p.err, DEV_ERR_TIMEOUT);
            if (lane < kAttnWarps)  // let the copies in flight land before the CTA ends
                for (int i = n > S ? n - S : 0; i < n; ++i) mbar_wait(s_full + lane * S + i % S, (i / S) & 1);
        }
        return;
    }

    // ---- consumers
    const int g8 = lane >> 2, t4 = lane & 3;
    int slot = 0;
    uint32_t phase = 0;
    while (w.left > 0) {
        const AttnSeq sq = w.s;
        const int ga = w.ga, gb = w.gb(), item = w.item;
        const int64_t at0 = hi - w.left;               // position of the segment's first group
        const int shown = min(sq.rows, p.max_q), tiles = sq.items / p.Hkv, hk = item / tiles;
        const int r0 = (item - hk * tiles) * kRows, r_end = min(shown * p.G, r0 + kRows);
        const int from = sq.len - sq.rows;

        // query rows -> operand registers (through shared memory, each warp a part of the k-steps)
        float xs[RS];                                   // score of an accumulator unit, times log2 e
        int pos[RS], first_key[RS];
        float init[RS][NB], slope[RS];
        {
            uint32_t frag[KS][4];
#pragma unroll
            for (int rs = 0; rs < RS; ++rs) {
                const int r = min(r0 + g8 + 8 * rs, r_end - 1);  // rows past the end repeat the last one
                float4 x[KS];
                float amax = 0.0f;
#pragma unroll
                for (int j = 0; j < KS; ++j) {
                    x[j] = attn_q4(p, sq, hk, r, 16 * j + 4 * t4);
                    amax = fmaxf(fmaxf(amax, fmaxf(fabsf(x[j].x), fabsf(x[j].y))), fmaxf(fabsf(x[j].z), fabsf(x[j].w)));
                }
                amax = quad_max(amax);
                const int ex = static_cast<int>(__float_as_uint(amax) >> 23) - 127;
                const int sh = ex == 128 ? 0 : min(13 - ex, 100);  // largest element in [2^13, 2^14)
                const float up = pow2f(sh);
                xs[rs] = p.scale * scalbnf(1.0f, 24 - sh);
                pos[rs] = from + r / p.G;
                first_key[rs] = p.window > 0 ? pos[rs] - p.window + 1 : 0;
                slope[rs] = p.slopes ? p.slopes[hk * p.G + r % p.G] : 0.0f;
#pragma unroll
                for (int b = 0; b < NB; ++b) {
                    float sum = 0.0f;
#pragma unroll
                    for (int j = 2 * b; j < 2 * b + 2; ++j) {
                        const float v[4] = {x[j].x * up, x[j].y * up, x[j].z * up, x[j].w * up};
                        float h[4], l[4];
#pragma unroll
                        for (int i = 0; i < 4; ++i) {
                            h[i] = __half2float(__float2half_rn(v[i]));
                            l[i] = __half2float(__float2half_rn(v[i] - h[i]));
                            sum += MODE == A_SPLIT8 ? h[i] + l[i] : h[i];
                        }
                        // 4-bit quants of channels 2, 3 of four enter 16 times too large
                        const float k16 = K4 ? 0.0625f : 1.0f;
                        frag[j][rs] = pack_h2(h[0], h[1]);
                        frag[j][2 + rs] = pack_h2(h[2] * k16, h[3] * k16);
                        if (!TWO) {
                            frag[j][1] = MODE == A_SPLIT8 ? pack_h2(l[0], l[1]) : 0u;
                            frag[j][3] = MODE == A_SPLIT8 ? pack_h2(l[2] * k16, l[3] * k16) : 0u;
                        }
                    }
                    init[rs][b] = quad_sum(sum) * (K4 ? -8.0f : -128.0f) * 5.9604644775390625e-8f;  // 2^-24
                }
            }
#pragma unroll
            for (int j = 0; j < KS; ++j)
                if ((j & (kAttnWarps - 1)) == warp) s_q[j * 32 + lane] = make_uint4(frag[j][0], frag[j][1], frag[j][2], frag[j][3]);
        }
        consumer_sync();
        const bool plain = p.cap <= 0.0f && !p.slopes;
        constexpr float kLog2e = 1.44269504088896340736f;
        if (plain)
            for (int rs = 0; rs < RS; ++rs) xs[rs] *= kLog2e;
        // groups that every row of the tile sees whole
        const int whole_end = (from + r0 / p.G + 1) >> 4;
        const int last_first = p.window > 0 ? from + (r_end - 1) / p.G - p.window + 1 : 0;
        const int whole_begin = last_first > 0 ? (last_first + 15) >> 4 : 0;

        float m[RS], l[RS], tot[RS][NT][2];
#pragma unroll
        for (int rs = 0; rs < RS; ++rs) {
            m[rs] = kAttnNone, l[rs] = 0.0f;
#pragma unroll
            for (int n = 0; n < NT; ++n) tot[rs][n][0] = tot[rs][n][1] = 0.0f;
        }
        float vs = 0x1p40f;  // power of two on the value scales

        for (int g = ga + warp; g < gb; g += kAttnWarps) {
            const int at = warp * S + slot;
            bool ok = !*s_abort && mbar_wait(s_full + at, phase);
            ok = __all_sync(0xffffffffu, ok);
            if (!ok) {
                *s_abort = 1;
                set_error(p.err, DEV_ERR_TIMEOUT);
                break;
            }
            const uint8_t* const kb = smem + SM::oRing + at * SM::kStage;
            const uint8_t* const vb = kb + SM::kKB;

            // scores of two octets of keys
            float sc[2][4];
#pragma unroll
            for (int o = 0; o < 2; ++o)
#pragma unroll
                for (int i = 0; i < 4; ++i) sc[o][i] = 0.0f;
            constexpr int KW = K4 ? NB : KS;  // words of an octet
            uint32_t kw[2 * KW];
#pragma unroll
            for (int v = 0; v < KW / 2; ++v) {
                const uint4 u = *reinterpret_cast<const uint4*>(kb + (v * 32 + lane) * 16);
                kw[4 * v] = u.x, kw[4 * v + 1] = u.y, kw[4 * v + 2] = u.z, kw[4 * v + 3] = u.w;
            }
            uint32_t kd[2][2][NB / 2];  // scales of keys 8 o + 2 t + e
#pragma unroll
            for (int o = 0; o < 2; ++o) {
                const uint32_t* const d = reinterpret_cast<const uint32_t*>(
                    kb + kv_quant_bytes(K4, D) + (8 * o + 2 * t4) * NB * 2);
#pragma unroll
                for (int e = 0; e < 2; ++e)
#pragma unroll
                    for (int i = 0; i < NB / 2; ++i) kd[o][e][i] = d[e * (NB / 2) + i];
            }
#pragma unroll
            for (int b = 0; b < NB; ++b) {
                const uint4 qa = s_q[(2 * b) * 32 + lane], qb = s_q[(2 * b + 1) * 32 + lane];
                const uint32_t fa[4] = {qa.x, qa.y, qa.z, qa.w}, fb[4] = {qb.x, qb.y, qb.z, qb.w};
#pragma unroll
                for (int o = 0; o < 2; ++o) {
                    float cc[4] = {init[0][b], init[0][b], TWO ? init[RS - 1][b] : 0.0f, TWO ? init[RS - 1][b] : 0.0f};
                    if constexpr (K4) {
                        const uint32_t u = kw[o * NB + b], y = u >> 8;
                        attn_mma(cc, fa, u & 0x000F000Fu, u & 0x00F000F0u);
                        attn_mma(cc, fb, y & 0x000F000Fu, y & 0x00F000F0u);
                    } else {
                        const uint32_t u = kw[o * KS + 2 * b], y = kw[o * KS + 2 * b + 1];
                        attn_mma(cc, fa, prmt(u, 0u, 0x4140u), prmt(u, 0u, 0x4342u));
                        attn_mma(cc, fb, prmt(y, 0u, 0x4140u), prmt(y, 0u, 0x4342u));
                    }
                    const float d0 = (b & 1) ? half_hi(kd[o][0][b >> 1]) : half_lo(kd[o][0][b >> 1]);
                    const float d1 = (b & 1) ? half_hi(kd[o][1][b >> 1]) : half_lo(kd[o][1][b >> 1]);
                    if constexpr (MODE == A_SPLIT8) cc[0] += cc[2], cc[1] += cc[3];
                    sc[o][0] = fmaf(d0, cc[0], sc[o][0]);
                    sc[o][1] = fmaf(d1, cc[1], sc[o][1]);
                    if constexpr (TWO) {
                        sc[o][2] = fmaf(d0, cc[2], sc[o][2]);
                        sc[o][3] = fmaf(d1, cc[3], sc[o][3]);
                    }
                }
            }
            uint32_t vd[2][2][NB / 2];
#pragma unroll
            for (int o = 0; o < 2; ++o) {
                const uint32_t* const d = reinterpret_cast<const uint32_t*>(
                    vb + kv_quant_bytes(V4, D) + (8 * o + 2 * t4) * NB * 2);
#pragma unroll
                for (int e = 0; e < 2; ++e)
#pragma unroll
                    for (int i = 0; i < NB / 2; ++i) vd[o][e][i] = d[e * (NB / 2) + i];
            }

            // logits in units of log2, masks
            float x[RS][4];
#pragma unroll
            for (int rs = 0; rs < RS; ++rs)
#pragma unroll
                for (int i = 0; i < 4; ++i) x[rs][i] = sc[i >> 1][2 * rs + (i & 1)] * xs[rs];
            if (!plain) {
#pragma unroll
                for (int rs = 0; rs < RS; ++rs)
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        const int key = 16 * g + 8 * (i >> 1) + 2 * t4 + (i & 1);
                        float y = x[rs][i];
                        if (p.cap > 0.0f) y = p.cap * tanhf(__fdividef(y, p.cap));
                        x[rs][i] = fmaf(slope[rs], static_cast<float>(key - pos[rs]), y) * kLog2e;
                    }
            }
            if (g < whole_begin || g >= whole_end) {
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const int key = 16 * g + 8 * (i >> 1) + 2 * t4 + (i & 1);
#pragma unroll
                    for (int rs = 0; rs < RS; ++rs)
                        if (key > pos[rs] || key < first_key[rs]) x[rs][i] = -INFINITY;
                    if (key >= sq.len)  // never written: whatever the place holds
#pragma unroll
                        for (int k = 0; k < NB / 2; ++k) vd[i >> 1][i & 1][k] = 0u;
                }
            }

            // the group's maximum is its probabilities' reference
            float pr[RS][4], f[RS];
            bool raise = false;
#pragma unroll
            for (int rs = 0; rs < RS; ++rs) {
                f[rs] = quad_max(fmaxf(fmaxf(x[rs][0], x[rs][1]), fmaxf(x[rs][2], x[rs][3])));
                raise |= f[rs] > m[rs] + 60.0f ||
                         fminf(fminf(x[rs][0], x[rs][1]), fminf(x[rs][2], x[rs][3])) < f[rs] - 28.0f;
            }
            uint32_t dm = 0u;
#pragma unroll
            for (int i = 0; i < 4; ++i)
#pragma unroll
                for (int k = 0; k < NB / 2; ++k) dm = __vmaxu2(dm, vd[i >> 1][i & 1][k] & 0x7FFF7FFFu);
            raise |= !(fmaxf(half_lo(dm), half_hi(dm)) * vs <= 46341.0f) || (dm & 0x7FFFu) >= 0x7C00u || (dm >> 16) >= 0x7C00u;
            bool dirty = false;  // a value scale is not finite
            bool more = false;   // some probabilities are too small for fp16 beside the group's largest
            if (__any_sync(0xffffffffu, raise)) {
                float dfin = 0.0f;
#pragma unroll
                for (int i = 0; i < 4; ++i)
#pragma unroll
                    for (int k = 0; k < NB / 2; ++k) {
                        const uint32_t u = vd[i >> 1][i & 1][k] & 0x7FFF7FFFu;
                        if ((u & 0xFFFFu) < 0x7C00u) dfin = fmaxf(dfin, half_lo(u)); else dirty = true;
                        if ((u >> 16) < 0x7C00u) dfin = fmaxf(dfin, half_hi(u)); else dirty = true;
                    }
                dirty = __any_sync(0xffffffffu, dirty);
                dfin = warp_max(dfin);
                if (dfin * vs > 46341.0f)  // the largest to [2^13, 2^14)
                    vs = pow2f(13 - (static_cast<int>(__float_as_uint(dfin) >> 23) - 127));
#pragma unroll
                for (int rs = 0; rs < RS; ++rs)
                    if (f[rs] > m[rs] + 60.0f) {
                        const float a = ex2(m[rs] - f[rs]);
                        m[rs] = f[rs];
                        l[rs] *= a;
#pragma unroll
                        for (int n = 0; n < NT; ++n) tot[rs][n][0] *= a, tot[rs][n][1] *= a;
                    }
#pragma unroll
                for (int rs = 0; rs < RS; ++rs)
#pragma unroll
                    for (int i = 0; i < 4; ++i) more |= x[rs][i] < f[rs] - 28.0f && x[rs][i] > m[rs] - 126.0f;
                more = __any_sync(0xffffffffu, more);
            }
            for (;;) {  // once, but for probabilities more than 2^28 apart: those below wait for a pass of their own
                float rest[RS];
#pragma unroll
                for (int rs = 0; rs < RS; ++rs) {
                    const float top = fmaxf(f[rs], kAttnNone);  // a group that the row does not see: all probabilities 0
                    float sum = 0.0f;
                    rest[rs] = -INFINITY;
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        pr[rs][i] = ex2(x[rs][i] - top);
                        if (more) {
                            if (x[rs][i] < top - 28.0f) {
                                pr[rs][i] = 0.0f;
                                rest[rs] = fmaxf(rest[rs], x[rs][i]);
                            } else {
                                x[rs][i] = -INFINITY;
                            }
                        }
                        sum += pr[rs][i];
                        pr[rs][i] *= vs;
                    }
                    const float w = ex2(top - m[rs]);
                    l[rs] = fmaf(sum, w, l[rs]);
                    f[rs] = w * (1.0f / vs);
                }

                // values, block by block of 32 channels
#pragma unroll
                for (int b = 0; b < NB; ++b) {
                    uint32_t a[4];
                    float dv[4], acc[4][4];
#pragma unroll
                    for (int k = 0; k < 4; ++k)
#pragma unroll
                        for (int i = 0; i < 4; ++i) acc[k][i] = 0.0f;
#pragma unroll
                    for (int i = 0; i < 4; ++i)
                        dv[i] = (b & 1) ? half_hi(vd[i >> 1][i & 1][b >> 1]) : half_lo(vd[i >> 1][i & 1][b >> 1]);
                    float pd[RS][4];
#pragma unroll
                    for (int rs = 0; rs < RS; ++rs)
#pragma unroll
                        for (int i = 0; i < 4; ++i) {
                            pd[rs][i] = pr[rs][i] * dv[i];
                            if (dirty && pr[rs][i] == 0.0f) pd[rs][i] = 0.0f;  // an infinite scale that the row does not see
                        }
                    if constexpr (MODE == A_SPLIT8) {
#pragma unroll
                        for (int o = 0; o < 2; ++o) {
                            // rounded to fp16, and 2^12 times what that leaves
                            const uint32_t h = pack_h2(pd[0][2 * o], pd[0][2 * o + 1]);
                            a[2 * o] = h;
                            a[2 * o + 1] = pack_h2((pd[0][2 * o] - half_lo(h)) * 4096.0f, (pd[0][2 * o + 1] - half_hi(h)) * 4096.0f);
                        }
                    } else {
#pragma unroll
                        for (int o = 0; o < 2; ++o) {
                            a[2 * o] = pack_h2(pd[0][2 * o], pd[0][2 * o + 1]);
                            a[2 * o + 1] = TWO ? pack_h2(pd[RS - 1][2 * o], pd[RS - 1][2 * o + 1]) : 0u;
                        }
                    }
                    if constexpr (V4) {
                        const uint2 u2 = *reinterpret_cast<const uint2*>(vb + ((b >> 1) * 32 + lane) * 16 + (b & 1) * 8);
                        const uint32_t uw[2] = {u2.x, u2.y};
#pragma unroll
                        for (int k = 0; k < 2; ++k) {
                            const uint32_t u = uw[k], y = u >> 8;
                            // 1024 + q - 1032, and (1024 + 16 q) / 16 - 72
                            attn_mma(acc[2 * k], a, h2_sub((u & 0x000F000Fu) | 0x64006400u, 0x64086408u),
                                     h2_sub((y & 0x000F000Fu) | 0x64006400u, 0x64086408u));
                            attn_mma(acc[2 * k + 1], a, h2_fma((u & 0x00F000F0u) | 0x64006400u, 0x2C002C00u, 0xD480D480u),
                                     h2_fma((y & 0x00F000F0u) | 0x64006400u, 0x2C002C00u, 0xD480D480u));
                        }
                    } else {
                        const uint4 u4 = *reinterpret_cast<const uint4*>(vb + (b * 32 + lane) * 16);
                        const uint32_t uw[4] = {u4.x, u4.y, u4.z, u4.w};
#pragma unroll
                        for (int k = 0; k < 4; ++k)  // 1024 + (q + 128) - 1152
                            attn_mma(acc[k], a, h2_sub(prmt(uw[k], 0x64646464u, 0x4140u), 0x64806480u),
                                     h2_sub(prmt(uw[k], 0x64646464u, 0x4342u), 0x64806480u));
                    }
#pragma unroll
                    for (int k = 0; k < 4; ++k) {
                        float(&o)[2] = tot[0][4 * b + k];
                        if constexpr (MODE == A_SPLIT8) fma2(acc[k][0], acc[k][1], acc[k][2], acc[k][3], 0x1p-12f, acc[k][0], acc[k][1]);
                        fma2(o[0], o[1], acc[k][0], acc[k][1], f[0], o[0], o[1]);
                        if constexpr (TWO) {
                            float(&o2)[2] = tot[RS - 1][4 * b + k];
                            fma2(o2[0], o2[1], acc[k][2], acc[k][3], f[RS - 1], o2[0], o2[1]);
                        }
                    }
                }
                if (!more) break;
                more = false;
#pragma unroll
                for (int rs = 0; rs < RS; ++rs) {
                    f[rs] = quad_max(rest[rs]);
                    more |= f[rs] > m[rs] - 126.0f;
                }
                more = __any_sync(0xffffffffu, more);
                if (!more) break;
            }
            __syncwarp();
            if (lane == 0) mbar_arrive(s_empty + at);
            if (++slot == S) slot = 0, phase ^= 1u;
        }
        float* const s_mine = s_tot + warp * kRows * SM::kRowPitch;
#pragma unroll
        for (int rs = 0; rs < RS; ++rs)
#pragma unroll
            for (int n = 0; n < NT; ++n)
                *reinterpret_cast<float2*>(s_mine + (g8 + 8 * rs) * SM::kRowPitch + 8 * n + 2 * t4) =
                    make_float2(tot[rs][n][0], tot[rs][n][1]);
#pragma unroll
        for (int rs = 0; rs < RS; ++rs) {
            const float sum = quad_sum(l[rs]);
            if (t4 == 0) {
                s_m[warp * kRows + g8 + 8 * rs] = m[rs];
                s_l[warp * kRows + g8 + 8 * rs] = sum;
            }
        }
        consumer_sync();

        // ---- the segment's result: the four warps' parts
        const bool whole = ga == sq.glo && gb == sq.ghi;
        float* const part = p.parts + (static_cast<int64_t>(c) * 2 + (at0 == lo ? 0 : 1)) * attn_part_floats(D);
        for (int i = tid; i < kRows * D / 4; i += kAttnWarps * 32) {
            const int row = i / (D / 4), d = 4 * (i - row * (D / 4));
            if (r0 + row >= r_end) break;
            float M = kAttnNone, L = 0.0f;
#pragma unroll
            for (int k = 0; k < kAttnWarps; ++k) M = fmaxf(M, s_m[k * kRows + row]);
            float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
            for (int k = 0; k < kAttnWarps; ++k) {
                const float f = ex2(s_m[k * kRows + row] - M);
                const float4 v = *reinterpret_cast<const float4*>(s_tot + (k * kRows + row) * SM::kRowPitch + d);
                L = fmaf(s_l[k * kRows + row], f, L);
                o.x = fmaf(v.x, f, o.x), o.y = fmaf(v.y, f, o.y), o.z = fmaf(v.z, f, o.z), o.w = fmaf(v.w, f, o.w);
            }
            if (whole) {
                const float inv = L != 0.0f ? 1.0f / L : 0.0f;
                attn_out4(p, sq, hk, r0 + row, d, make_float4(o.x * inv, o.y * inv, o.z * inv, o.w * inv));
            } else {
                if (d == 0) part[row] = M, part[16 + row] = L;
                *reinterpret_cast<float4*>(part + 32 + row * D + d) = o;
            }
        }
        if (!whole) {
            // pieces of this item: the CTAs c0 .. c1 whose shares it crosses
            const int64_t p0 = at0 - (ga - sq.glo), p1 = p0 + (sq.ghi - sq.glo);  // the item's positions [p0, p1)
            const int c0 = static_cast<int>(((p0 + 1) * C - 1) / N), c1 = static_cast<int>((p1 * C - 1) / N);
            __threadfence();
            consumer_sync();
            if (tid == 0) {
                const int before = atomicAdd(p.pieces + c0, 1);
                *s_last = before == c1 - c0;
                if (before == c1 - c0) p.pieces[c0] = 0;
                __threadfence();
            }
            consumer_sync();
            if (*s_last) {
                const int64_t size = attn_part_floats(D);
                const int slot0 = N * c0 / C == p0 ? 0 : 1;  // the first piece; every other piece begins its CTA's share
                for (int i = tid; i < kRows * D / 4; i += kAttnWarps * 32) {
                    const int row = i / (D / 4), d = 4 * (i - row * (D / 4));
                    if (r0 + row >= r_end) break;
                    float M = kAttnNone, L = 0.0f;
                    for (int k = c0; k <= c1; ++k)
                        M = fmaxf(M, __ldcg(p.parts + (2 * k + (k == c0 ? slot0 : 0)) * size + row));
                    float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 4
                    for (int k = c0; k <= c1; ++k) {
                        const float* const q = p.parts + (2 * k + (k == c0 ? slot0 : 0)) * size;
                        const float f = ex2(__ldcg(q + row) - M);
                        const float4 v = __ldcg(reinterpret_cast<const float4*>(q + 32 + row * D + d));
                        L = fmaf(__ldcg(q + 16 + row), f, L);
                        o.x = fmaf(v.x, f, o.x), o.y = fmaf(v.y, f, o.y), o.z = fmaf(v.z, f, o.z), o.w = fmaf(v.w, f, o.w);
                    }
                    const float inv = L != 0.0f ? 1.0f / L : 0.0f;
                    attn_out4(p, sq, hk, r0 + row, d, make_float4(o.x * inv, o.y * inv, o.z * inv, o.w * inv));
                }
            }
        }
        consumer_sync();  // the totals and the query operand are free again
        w.next(p, kRows);
    }
}

// Launch of one (K format, V format, D, mode); the grid fills the SMs once.
template <bool K4, bool V4, int D, int MODE>
cudaError_t launch_attn_stream(const AttnParams& p, int nsm, cudaStream_t s) {
    using SM = AttnSmem<K4, V4, D, MODE>;
    static bool set[kMaxDevices] = {};
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    if (dev >= kMaxDevices || !set[dev]) {
        e = cudaFuncSetAttribute(k_attn_stream<K4, V4, D, MODE>, cudaFuncAttributeMaxDynamicSharedMemorySize, SM::kTotal);
        if (e != cudaSuccess) return e;
        if (dev < kMaxDevices) set[dev] = true;
    }
    const int64_t tiles = (static_cast<int64_t>(p.max_q) * p.G + SM::kRows - 1) / SM::kRows;
    const int64_t groups = p.n_seqs * p.Hkv * tiles * ((static_cast<int64_t>(p.max_len) + 15) / 16);
    int64_t grid = (groups + p.min_share - 1) / p.min_share;
    if (grid > static_cast<int64_t>(nsm) * SM::kCtas) grid = static_cast<int64_t>(nsm) * SM::kCtas;
    if (grid > kAttnMaxCtas) grid = kAttnMaxCtas;
    if (grid < 1) grid = 1;
    return launch_pdl(k_attn_stream<K4, V4, D, MODE>, dim3(static_cast<unsigned>(grid)), dim3(kAttnThreads), SM::kTotal, s, p);
}

template <bool K4, bool V4, int D>
cudaError_t launch_attn_stream_mode(const AttnParams& p, int nsm, cudaStream_t s) {
    if (p.dtype == 0) return launch_attn_stream<K4, V4, D, A_SPLIT8>(p, nsm, s);
    if (static_cast<int64_t>(p.max_q) * p.G <= 8) return launch_attn_stream<K4, V4, D, A_HALF8>(p, nsm, s);
    return launch_attn_stream<K4, V4, D, A_HALF16>(p, nsm, s);
}

}  // namespace ggq
