// ggq_attn_stream.cuh -- attention for few query rows per kv head: a stream
// over the packed cache on mma.sync.
//
// Mathematics: with the blocks' quants u (stored + 128 or + 8), scales d and
// query row q, s_j = sum_b dk_jb sum_{c in b} q_c (u_jc - off) and out_c = sum_j
// p_j dv_jb (u_jc - off) / sum_j p_j.  The matrix instruction multiplies query
// rows (16) by the integer quants, which fp16 holds exactly; the scales are
// applied to its fp32 results (scores) and to the probabilities (values), so the
// packed bytes are unpacked but never dequantized.
//   * Scores: two k16 steps per block of 32 channels.  For 16-bit activations the
//     quants enter as fp16 subnormals u 2^-24 (a byte permutation, no arithmetic);
//     the accumulator starts at -off 2^-24 sum_c q_c, which takes the offset out again.
//     For fp32 the sums would lose bits to the offset: signed integers.
//   * Values: quants as exact signed fp16 integers; the other operand is p dv
//     times a power of two that keeps it in fp16's normal range.
//   * fp32 activations: 8 query rows; a 16-row operand holds the high and low
//     fp16 parts of each (22 bits of the row's largest element), whose results add up.
//     16-bit activations: 8 or 16 rows in one fp16 operand (16-bit queries are exact in it).
//   * Softmax statistics are fp32.  Within a unit the probabilities are relative to
//     the unit's maximum and lifted by a power of two that keeps p dv below fp16's
//     range (the second half by 2^12 more); a unit's result is added to the fp32
//     totals with its factor 2^(unit's maximum - reference).  No sum runs longer than
//     a unit on the tensor cores (which truncate), no probability is lost for being
//     small (those of a unit that lie more than 2^28 apart take a pass each), and the
//     totals are rescaled only when the reference rises by 2^60.
//
// Bound by HBM: every attended blob is read once (17 or 9 bytes per 16
// channels).  Work is cut in equal shares of units (two 16-token groups; one for
// heads of 256 channels) over all CTAs,
// whatever the lengths; a CTA walks its share item by item (an item is one
// sequence, kv head and tile of rows), its four warps take every fourth unit, each
// keeping a ring of bulk copies in flight, across items.  An item that several CTAs
// share is joined by the last of them from partial results in scratch, in the order of
// the pieces.
//
// Measured (32 heads on 8 of 128 channels, Q8_0): one token of 4 sequences of 131072,
// fp32: 204 us, 5.6 TB/s, 83% of the copy's rate; 64 ragged sequences of up to 4096,
// bf16: 63 us, 5.0 TB/s (shares end together, but an item's start and join cost what 12
// units do); one of 777, fp32: 11.7 us, all latency.  64 heads on 8 of 64 channels, Q4_0,
// 33 of up to 16384, f16: 66 us, 2.6 TB/s, bound by each warp's chain of product, maximum,
// exponential and product at 12 warps an SM (issue slots 50% used: half the bytes a value,
// the same unpacking); 5 rows of 16 heads on 8 of 256 channels: 86 us, the same at 8 warps
// an SM and with spilled totals (36%).
#pragma once
#include <atomic>

#include "ggq_attn.cuh"
#include "ggq_device.cuh"
#include "ggq_internal.h"

namespace ggq {

constexpr int kAttnWarps = 4;
constexpr int kAttnThreads = kAttnWarps * 32;
constexpr float kAttnNone = -1e30f;                    // reference maximum of a row that has seen nothing

// fp32 rows (high and low halves), 8 rows or 16 rows of 16-bit activations
enum AttnMode : int { A_SPLIT8 = 0, A_HALF8 = 1, A_HALF16 = 2 };

// cap * tanh(y / cap).  For fp32 rows tanhf; else 1 - 2 / (1 + exp(2 z)), whose error
// of a few 2^-23 cap (cap <= kWideCap) is below the roundings of 16-bit activations.
template <int MODE>
__device__ __forceinline__ float attn_cap(float y, float cap) {
    const float z = __fdividef(y, cap);
    if (MODE == A_SPLIT8) return cap * tanhf(z);
    const float e = z * 2.88539008177792681f;  // 2 log2 e
    float x;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(x) : "f"(e > 120.0f ? 120.0f : e));
    return cap - __fdividef(2.0f * cap, 1.0f + x);
}

template <bool K4, bool V4, int D, int MODE>
struct AttnSmem {
    static constexpr int kRows = MODE == A_HALF16 ? 16 : 8;
    // 16-token groups a warp takes at once: what the registers hold.  (8 rows of 64 4-bit
    // channels, 33 ragged sequences of up to 8192: 43 us at 4, 47 at 2; 16 rows 184 and
    // 133, fp32 57 and 53, 16 rows with one 8-bit side 219 and 137.)
    static constexpr int kUnit = D == 256 ? 1 : D == 64 && K4 && V4 && MODE == A_HALF8 ? 4 : 2;
    static constexpr int kKB = kv_blob_bytes(K4, D), kVB = kv_blob_bytes(V4, D);
    static constexpr int kStage = kUnit * (kKB + kVB); // keys of the unit's groups, then their values
    // Ring bytes that leave an SM its CTAs, and heads of 256 channels some first-level cache
    // for what their registers do not hold (Q4_0, 33 ragged sequences of up to 8192, 16
    // rows: 186 us, with 72 KB 300; 128 channels, Q8_0: 147, with 104 KB and so one CTA an
    // SM 227).
    static constexpr int kFit = (D == 64 ? 52 : D == 128 ? 72 : 64) * 1024 / (kAttnWarps * kStage);
    static constexpr int kStages = kFit < 2 ? 2 : kFit > 6 ? 6 : kFit;
    static constexpr int kMerge = D == 256 ? 128 : D;  // channels that the warps' totals are merged by
    static constexpr int kRowPitch = kMerge + 8;       // floats of a totals row (padding: conflict-free float2 stores)
    static constexpr int oRing = 0;
    static constexpr int oTot = kAttnWarps * kStages * kStage;
    static constexpr int oQ = oTot + kAttnWarps * 8 * kRowPitch * 4;  // totals of 8 rows a warp
    static constexpr int oStat = oQ + D / 16 * 32 * 16;   // m, l [warps][8]
    static constexpr int oScan = (oStat + 2 * kAttnWarps * 8 * 4 + 7) / 8 * 8;
    static constexpr int oBar = (oScan + (128 + 4) * 8 + 15) / 16 * 16;
    static constexpr int oLast = oBar + kAttnWarps * kStages * 8 + 16;
    static constexpr int kTotal = oLast + kAttnWarps * 4;
    // CTAs an SM: 12 warps leave 168 registers a thread (64-channel heads), 8 warps 255
    static constexpr int kCtas = D == 64 && 3 * (kTotal + 1024) <= 228 * 1024 ? 3 : 2 * (kTotal + 1024) <= 228 * 1024 ? 2 : 1;
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
// Units of UNIT groups of an item, and of the sequence's items together.
template <int UNIT>
__device__ __forceinline__ int attn_units(const AttnSeq& s) { return (s.ghi - s.glo + UNIT - 1) / UNIT; }
// Positions of an item in the list of all items: kItemCost, then its units.
template <int UNIT>
__device__ __forceinline__ int attn_span(const AttnSeq& s) {
    const int n = attn_units<UNIT>(s);
    return n > 0 ? n + kItemCost : 0;
}
template <int UNIT>
__device__ __forceinline__ int64_t attn_cost(const AttnSeq& s) { return static_cast<int64_t>(attn_span<UNIT>(s)) * s.items; }

// A CTA's share, item by item.
template <int UNIT>
struct AttnWalk {
    AttnSeq s;
    int b, item, ua;
    int64_t left;  // positions of the share that are not yet walked
    __device__ __forceinline__ int ub() const {  // end of the current segment
        const int64_t e = ua + left;
        const int n = attn_span<UNIT>(s);
        return e < n ? static_cast<int>(e) : n;
    }
    __device__ __forceinline__ int first() const { return ua > kItemCost ? ua - kItemCost : 0; }  // its units
    __device__ __forceinline__ int last() const { return ub() - kItemCost; }
    __device__ __forceinline__ void next(const AttnParams& p, int tile_rows) {
        left -= ub() - ua;
        if (left <= 0) return;
        if (++item == s.items) {
            item = 0;
            do s = attn_seq(p, ++b, tile_rows, false); while (attn_cost<UNIT>(s) == 0);
        }
        ua = 0;
    }
};

// D = A B, D = A B + C, and D += A B
__device__ __forceinline__ void attn_mma_c(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1, const float (&c)[4]) {
    asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%10,%11,%12,%13};"
        : "=f"(d[0]), "=f"(d[1]), "=f"(d[2]), "=f"(d[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1), "f"(c[0]), "f"(c[1]), "f"(c[2]), "f"(c[3]));
}
// A register of any content: operand rows whose results nobody reads.
__device__ __forceinline__ uint32_t attn_any() {
    uint32_t r;
    asm volatile("" : "=r"(r));
    return r;
}
__device__ __forceinline__ void attn_mma0(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
    asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%10,%10,%10,%10};"
        : "=f"(d[0]), "=f"(d[1]), "=f"(d[2]), "=f"(d[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1), "f"(0.0f));
}
__device__ __forceinline__ void attn_mma(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
    asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
__device__ __forceinline__ float ex2(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}
// the same with subnormal results: factors of sums that the unit's lift has raised
__device__ __forceinline__ float ex2_small(float x) {
    float y;
    asm("ex2.approx.f32 %0, %1;" : "=f"(y) : "f"(x));
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
// Two fp32 operations in one instruction: a b + c, a + b, a b
__device__ __forceinline__ float2 fma2(float2 a, float2 b, float2 c) {
    float2 d;
    asm("{\n\t.reg .b64 x, y, z;\n\tmov.b64 x, {%2, %3};\n\tmov.b64 y, {%4, %5};\n\tmov.b64 z, {%6, %7};\n\t"
        "fma.rn.f32x2 x, x, y, z;\n\tmov.b64 {%0, %1}, x;\n\t}"
        : "=f"(d.x), "=f"(d.y)
        : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y), "f"(c.x), "f"(c.y));
    return d;
}
__device__ __forceinline__ float2 add2(float2 a, float2 b) {
    float2 d;
    asm("{\n\t.reg .b64 x, y;\n\tmov.b64 x, {%2, %3};\n\tmov.b64 y, {%4, %5};\n\tadd.rn.f32x2 x, x, y;\n\t"
        "mov.b64 {%0, %1}, x;\n\t}"
        : "=f"(d.x), "=f"(d.y)
        : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y));
    return d;
}
__device__ __forceinline__ float2 mul2(float2 a, float2 b) {
    float2 d;
    asm("{\n\t.reg .b64 x, y;\n\tmov.b64 x, {%2, %3};\n\tmov.b64 y, {%4, %5};\n\tmul.rn.f32x2 x, x, y;\n\t"
        "mov.b64 {%0, %1}, x;\n\t}"
        : "=f"(d.x), "=f"(d.y)
        : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y));
    return d;
}
__device__ __forceinline__ float2 both(float v) { return make_float2(v, v); }
__device__ __forceinline__ float2 half2_f32(uint32_t u) { return __half22float2(*reinterpret_cast<const __half2*>(&u)); }
__device__ __forceinline__ uint32_t h2_mul(uint32_t a, uint32_t b) {
    const __half2 r = __hmul2(*reinterpret_cast<const __half2*>(&a), *reinterpret_cast<const __half2*>(&b));
    return *reinterpret_cast<const uint32_t*>(&r);
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

// The rows of an item: kv head, first row and end of its tile.
struct AttnTile {
    int hk, r0, r_end;
};
__device__ __forceinline__ AttnTile attn_tile(const AttnParams& p, const AttnSeq& s, int item, int tile_rows) {
    const int tiles = s.items / p.Hkv;
    AttnTile t;
    t.hk = item / tiles;
    t.r0 = (item - t.hk * tiles) * tile_rows;
    t.r_end = min(min(s.rows, p.max_q) * p.G, t.r0 + tile_rows);
    return t;
}

template <typename T>
__device__ __forceinline__ const T* attn_q_row(const AttnParams& p, const AttnSeq& s, int hk, int r) {
    const int i = r / p.G, h = hk * p.G + r - i * p.G;
    return static_cast<const T*>(p.q) + (s.first + i) * p.q_token + h * p.q_head;
}
// Elements 16 j + 4 t .. + 3 of a row: all loads in flight at once.
template <typename T, int KS>
__device__ __forceinline__ void attn_load_row(const T* q, float4 (&x)[KS]) {
#pragma unroll
    for (int j = 0; j < KS; ++j) x[j] = ld4(q + 16 * j);
}
template <int KS>
__device__ __forceinline__ void attn_row(const AttnParams& p, const AttnSeq& s, int hk, int r, int t4, float4 (&x)[KS]) {
    if (p.dtype == 0) attn_load_row(attn_q_row<float>(p, s, hk, r) + 4 * t4, x);
    else if (p.dtype == 1) attn_load_row(attn_q_row<__half>(p, s, hk, r) + 4 * t4, x);
    else attn_load_row(attn_q_row<__nv_bfloat16>(p, s, hk, r) + 4 * t4, x);
}
__device__ __forceinline__ void attn_out4(const AttnParams& p, const AttnSeq& s, int hk, int r, int d, float4 v) {
    const int i = r / p.G, h = hk * p.G + r - i * p.G;
    const int64_t at = (s.first + i) * p.out_token + h * p.out_head + d;
    if (p.dtype == 0) st4(static_cast<float*>(p.out) + at, v);
    else if (p.dtype == 1) st4(static_cast<__half*>(p.out) + at, v);
    else st4(static_cast<__nv_bfloat16*>(p.out) + at, v);
}

// A warp's query rows (8, or 16) against units of the cache: what a thread keeps of
// them, and one step.  A thread's rows: g (16 rows: and g + 8).
template <bool K4, bool V4, int D, int MODE, int UNIT>
struct AttnRows {
    static constexpr bool TWO = MODE == A_HALF16;  // operand rows 8..15 are query rows of their own
    static constexpr int RS = TWO ? 2 : 1, NB = D / 32, KS = D / 16, NT = D / 8;
    static constexpr int kKB = kv_blob_bytes(K4, D), kVB = kv_blob_bytes(V4, D);
    static constexpr float kLog2e = 1.44269504088896340736f;
    // power of two that lifts the probabilities: p * lift * (largest value scale) stays below 32000;
    // 8 rows of 256 channels: the offsets are added to the results, one register a block
    // instead of an accumulator's four (Q8_0, 33 ragged sequences of up to 8192: 129 -> 123
    // us; 16 rows, which spill either way: 182 -> 184)
    static constexpr bool kOffsetLater = D == 256 && MODE == A_HALF8;
    // fp16 probabilities (16-bit activations) must not pass 2^15 themselves
    static constexpr float kMaxLift = MODE == A_SPLIT8 ? 40.0f : 15.0f;

    float xs[RS];                    // score of an accumulator unit (plain: times log2 e)
    int pos[RS], first_key[RS];
    float offset[NB][4], slope[RS];  // -offset * sum of the queries of a block, as an accumulator
    int whole_begin, whole_end;      // groups that every row sees whole
    bool plain;                      // no cap, no slopes
    float m[RS], l[RS];              // reference maximum and sum
    float2 tot[RS][NT];              // channels 8 n + 2 t, + 1
    float lift, dlimit;

    // Query rows r0 .. of an item -> operand fragments in s_q (k-steps j with j % PARTS == part) and what a
    // thread keeps of its rows; nothing seen yet.
    template <int PARTS>
    __device__ __forceinline__ void begin(const AttnParams& p, const AttnSeq& sq, int hk, int r0, int r_end, uint4* s_q,
                                          int part, int lane) {
        const int g8 = lane >> 2, t4 = lane & 3, from = sq.len - sq.rows;
        {
            float4 x[RS][KS];
#pragma unroll
            for (int rs = 0; rs < RS; ++rs)  // rows past the end repeat the last one
                attn_row<KS>(p, sq, hk, min(r0 + g8 + 8 * rs, r_end - 1), t4, x[rs]);
            float up[RS];
#pragma unroll
            for (int rs = 0; rs < RS; ++rs) {
                float amax = 0.0f;
#pragma unroll
                for (int j = 0; j < KS; ++j) {
                    const float4 y = x[rs][j];
                    amax = fmaxf(fmaxf(amax, fmaxf(fabsf(y.x), fabsf(y.y))), fmaxf(fabsf(y.z), fabsf(y.w)));
                }
                amax = quad_max(amax);
                const int ex = static_cast<int>(__float_as_uint(amax) >> 23) - 127;
                // largest element in [2^13, 2^14); fp32 rows: in [2^10, 2^11), the high halves being integers,
                // whose products and sums of a block the matrix unit holds exactly
                const int sh = ex == 128 ? 0 : min((MODE == A_SPLIT8 ? 10 : 13) - ex, 100);
                up[rs] = copysignf(pow2f(sh), p.scale);
                xs[rs] = fabsf(p.scale) * scalbnf(1.0f, (MODE == A_SPLIT8 ? 0 : 24) - sh);
                const int r = min(r0 + g8 + 8 * rs, r_end - 1);
                pos[rs] = from + r / p.G;
                first_key[rs] = p.window > 0 ? pos[rs] - p.window + 1 : 0;
                slope[rs] = p.slopes ? p.slopes[hk * p.G + r % p.G] : 0.0f;
            }
#pragma unroll
            for (int b = 0; b < NB; ++b) {
                float sum[RS];
#pragma unroll
                for (int rs = 0; rs < RS; ++rs) sum[rs] = 0.0f;
#pragma unroll
                for (int j = 2 * b; j < 2 * b + 2; ++j) {
                    uint32_t frag[4];
#pragma unroll
                    for (int rs = 0; rs < RS; ++rs) {
                        const float4 y = x[rs][j];
                        const float v[4] = {y.x * up[rs], y.y * up[rs], y.z * up[rs], y.w * up[rs]};
                        float h[4], l[4];
#pragma unroll
                        for (int i = 0; i < 4; ++i) {
                            h[i] = MODE == A_SPLIT8 ? rintf(v[i]) : __half2float(__float2half_rn(v[i]));
                            l[i] = __half2float(__float2half_rn(v[i] - h[i]));
                            sum[rs] += h[i];
                        }
                        // 4-bit quants of channels 2, 3 of four enter 16 times too large
                        const float k16 = K4 && MODE != A_SPLIT8 ? 0.0625f : 1.0f;
                        frag[rs] = pack_h2(h[0], h[1]);
                        frag[2 + rs] = pack_h2(h[2] * k16, h[3] * k16);
                        if (!TWO) {
                            frag[1] = MODE == A_SPLIT8 ? pack_h2(l[0], l[1]) : 0u;
                            frag[3] = MODE == A_SPLIT8 ? pack_h2(l[2] * k16, l[3] * k16) : 0u;
                        }
                    }
                    if ((j & (PARTS - 1)) == part) s_q[j * 32 + lane] = make_uint4(frag[0], frag[1], frag[2], frag[3]);
                }
#pragma unroll
                for (int rs = 0; rs < 2; ++rs)
                    offset[b][2 * rs] = offset[b][2 * rs + 1] = quad_sum(sum[rs < RS ? rs : 0]) * (K4 ? -8.0f : -128.0f) * 0x1p-24f;
            }
        }
        plain = p.cap <= 0.0f && !p.slopes;
        if (plain)
            for (int rs = 0; rs < RS; ++rs) xs[rs] *= kLog2e;
        whole_end = (from + r0 / p.G + 1) >> 4;
        const int last_first = p.window > 0 ? from + (r_end - 1) / p.G - p.window + 1 : 0;
        whole_begin = last_first > 0 ? (last_first + 15) >> 4 : 0;
#pragma unroll
        for (int rs = 0; rs < RS; ++rs) {
            m[rs] = kAttnNone, l[rs] = 0.0f;
#pragma unroll
            for (int n = 0; n < NT; ++n) tot[rs][n] = both(0.0f);
        }
        lift = kMaxLift;
        dlimit = 32000.0f * pow2f(-static_cast<int>(kMaxLift));
    }

    // A unit: groups g .. g + UNIT - 1, their key blobs at kb and value blobs at vb.
    __device__ __forceinline__ void unit(const AttnParams& p, const uint4* s_q, const uint8_t* kb, const uint8_t* vb, int g,
                                         int lane) {
        const int t4 = lane & 3;
        // ---- scores, index 4 group + 2 octet + e: keys 2 t + e of the octet
        constexpr int KW = K4 ? NB : KS;  // words of an octet
        float sc[RS][4 * UNIT];
        uint32_t kw[UNIT][2 * KW];
        float kd[UNIT][2][2][NB];  // scales of keys 8 o + 2 t + e
#pragma unroll
        for (int c = 0; c < UNIT; ++c) {
            const uint8_t* const blob = kb + c * kKB;
#pragma unroll
            for (int v = 0; v < KW / 2; ++v) {
                const uint4 q = *reinterpret_cast<const uint4*>(blob + (v * 32 + lane) * 16);
                kw[c][4 * v] = q.x, kw[c][4 * v + 1] = q.y, kw[c][4 * v + 2] = q.z, kw[c][4 * v + 3] = q.w;
            }
#pragma unroll
            for (int o = 0; o < 2; ++o) {
                const uint32_t* const d = reinterpret_cast<const uint32_t*>(
                    blob + kv_quant_bytes(K4, D) + (8 * o + 2 * t4) * NB * 2);
#pragma unroll
                for (int e = 0; e < 2; ++e)
#pragma unroll
                    for (int i = 0; i < NB / 2; ++i) {
                        const float2 f = half2_f32(d[e * (NB / 2) + i]);
                        kd[c][o][e][2 * i] = f.x, kd[c][o][e][2 * i + 1] = f.y;
                    }
            }
        }
#pragma unroll
        for (int b = 0; b < NB; ++b) {
            const uint4 qa = s_q[(2 * b) * 32 + lane], qb = s_q[(2 * b + 1) * 32 + lane];
            const uint32_t fa[4] = {qa.x, qa.y, qa.z, qa.w}, fb[4] = {qb.x, qb.y, qb.z, qb.w};
#pragma unroll
            for (int c = 0; c < UNIT; ++c)
#pragma unroll
                for (int o = 0; o < 2; ++o) {
                    float cc[4];
                    if constexpr (K4 && MODE == A_SPLIT8) {
                        const uint32_t q = kw[c][o * NB + b], y = q >> 8;
                        attn_mma0(cc, fa, h2_sub((q & 0x000F000Fu) | 0x64006400u, 0x64086408u),
                                  h2_fma((q & 0x00F000F0u) | 0x64006400u, 0x2C002C00u, 0xD480D480u));
                        attn_mma(cc, fb, h2_sub((y & 0x000F000Fu) | 0x64006400u, 0x64086408u),
                                 h2_fma((y & 0x00F000F0u) | 0x64006400u, 0x2C002C00u, 0xD480D480u));
                    } else if constexpr (MODE == A_SPLIT8) {
                        const uint32_t q = kw[c][o * KS + 2 * b], y = kw[c][o * KS + 2 * b + 1];
                        attn_mma0(cc, fa, h2_sub(prmt(q, 0x64646464u, 0x4140u), 0x64806480u),
                                  h2_sub(prmt(q, 0x64646464u, 0x4342u), 0x64806480u));
                        attn_mma(cc, fb, h2_sub(prmt(y, 0x64646464u, 0x4140u), 0x64806480u),
                                 h2_sub(prmt(y, 0x64646464u, 0x4342u), 0x64806480u));
                    } else if constexpr (K4) {
                        const uint32_t q = kw[c][o * NB + b], y = q >> 8;
                        if constexpr (kOffsetLater) attn_mma0(cc, fa, q & 0x000F000Fu, q & 0x00F000F0u);
                        else attn_mma_c(cc, fa, q & 0x000F000Fu, q & 0x00F000F0u, offset[b]);
                        attn_mma(cc, fb, y & 0x000F000Fu, y & 0x00F000F0u);
                    } else {
                        const uint32_t q = kw[c][o * KS + 2 * b], y = kw[c][o * KS + 2 * b + 1];
                        if constexpr (kOffsetLater) attn_mma0(cc, fa, prmt(q, 0u, 0x4140u), prmt(q, 0u, 0x4342u));
                        else attn_mma_c(cc, fa, prmt(q, 0u, 0x4140u), prmt(q, 0u, 0x4342u), offset[b]);
                        attn_mma(cc, fb, prmt(y, 0u, 0x4140u), prmt(y, 0u, 0x4342u));
                    }
                    if constexpr (MODE == A_SPLIT8) cc[0] += cc[2], cc[1] += cc[3];
                    else if constexpr (kOffsetLater) cc[0] += offset[b][0], cc[1] += offset[b][0];
#pragma unroll
                    for (int rs = 0; rs < RS; ++rs)
#pragma unroll
                        for (int e = 0; e < 2; ++e) {
                            float& to = sc[rs][4 * c + 2 * o + e];
                            to = b ? fmaf(kd[c][o][e][b], cc[2 * rs + e], to) : kd[c][o][e][b] * cc[2 * rs + e];
                        }
                }
        }
        uint32_t vd[UNIT][4][NB / 2];  // value scales of keys 8 o + 2 t + e, index 2 o + e
#pragma unroll
        for (int c = 0; c < UNIT; ++c)
#pragma unroll
            for (int o = 0; o < 2; ++o) {
                const uint32_t* const d = reinterpret_cast<const uint32_t*>(
                    vb + c * kVB + kv_quant_bytes(V4, D) + (8 * o + 2 * t4) * NB * 2);
#pragma unroll
                for (int e = 0; e < 2; ++e)
#pragma unroll
                    for (int i = 0; i < NB / 2; ++i) vd[c][2 * o + e][i] = d[e * (NB / 2) + i];
            }

        // ---- logits in units of log2, masks
        float lg[RS][4 * UNIT];
#pragma unroll
        for (int rs = 0; rs < RS; ++rs)
#pragma unroll
            for (int i = 0; i < 4 * UNIT; ++i) lg[rs][i] = sc[rs][i] * xs[rs];
        if (!plain) {
#pragma unroll
            for (int rs = 0; rs < RS; ++rs)
#pragma unroll
                for (int i = 0; i < 4 * UNIT; ++i) {
                    const int key = 16 * g + 8 * (i >> 1) + 2 * t4 + (i & 1);
                    float y = lg[rs][i];
                    if (p.cap > 0.0f) y = attn_cap<MODE>(y, p.cap);
                    lg[rs][i] = fmaf(slope[rs], static_cast<float>(key - pos[rs]), y) * kLog2e;
                }
        }
        float lowest[RS];  // before the masks: a bound
#pragma unroll
        for (int rs = 0; rs < RS; ++rs) {
            lowest[rs] = lg[rs][0];
#pragma unroll
            for (int i = 1; i < 4 * UNIT; ++i) lowest[rs] = fminf(lowest[rs], lg[rs][i]);
        }
        if (g < whole_begin || g + UNIT > whole_end) {
#pragma unroll
            for (int i = 0; i < 4 * UNIT; ++i) {
                const int key = 16 * g + 8 * (i >> 1) + 2 * t4 + (i & 1);
                bool seen = false;
#pragma unroll
                for (int rs = 0; rs < RS; ++rs) {
                    if (key > pos[rs] || key < first_key[rs]) lg[rs][i] = -INFINITY;
                    else seen = true;
                }
                if (!seen)  // whatever the place holds (it may never have been written) takes no part in the lift
#pragma unroll
                    for (int k = 0; k < NB / 2; ++k) vd[i >> 2][i & 3][k] = 0u;
            }
        }

        // ---- the unit's maximum is its probabilities' reference
        float top[RS];
        bool raise = false;
#pragma unroll
        for (int rs = 0; rs < RS; ++rs) {
            float highest = lg[rs][0];
#pragma unroll
            for (int i = 1; i < 4 * UNIT; ++i) highest = fmaxf(highest, lg[rs][i]);
            top[rs] = quad_max(highest);
            raise |= top[rs] > m[rs] + 60.0f || lowest[rs] < top[rs] - 28.0f;
        }
        uint32_t dm = 0u;
#pragma unroll
        for (int c = 0; c < UNIT; ++c)
#pragma unroll
            for (int i = 0; i < 4; ++i)
#pragma unroll
                for (int k = 0; k < NB / 2; ++k) dm = __vmaxu2(dm, vd[c][i][k] & 0x7FFF7FFFu);
        raise |= !(half_lo(dm) <= dlimit && half_hi(dm) <= dlimit);  // larger, or not a number
        bool more = false;   // some probabilities are too small for fp16 beside the unit's largest
        if (__any_sync(0xffffffffu, raise)) {
            float dfin = 0.0f;
            uint32_t spoilt[RS] = {};  // blocks of 32 channels in which a row sees a scale that is not finite
#pragma unroll
            for (int c = 0; c < UNIT; ++c)
#pragma unroll
                for (int i = 0; i < 4; ++i)
#pragma unroll
                    for (int b = 0; b < NB; ++b) {
                        const uint32_t d = (vd[c][i][b >> 1] >> (16 * (b & 1))) & 0x7FFFu;
                        if (d < 0x7C00u) {
                            dfin = fmaxf(dfin, half_lo(d));
                        } else {
                            vd[c][i][b >> 1] &= (b & 1) ? 0x0000FFFFu : 0xFFFF0000u;
#pragma unroll
                            for (int rs = 0; rs < RS; ++rs)
                                if (lg[rs][4 * c + i] != -INFINITY) spoilt[rs] |= 1u << b;
                        }
                    }
            dfin = quad_max(dfin);  // of the rows' own keys
            if (dfin > dlimit) {  // the largest times the lift to [2^13, 2^14)
                const int e = 13 - (static_cast<int>(__float_as_uint(dfin) >> 23) - 127);
                lift = fminf(static_cast<float>(e), kMaxLift);
                dlimit = 32000.0f * pow2f(-static_cast<int>(lift));
            }
#pragma unroll
            for (int rs = 0; rs < RS; ++rs) {
                spoilt[rs] |= __shfl_xor_sync(0xffffffffu, spoilt[rs], 1);
                spoilt[rs] |= __shfl_xor_sync(0xffffffffu, spoilt[rs], 2);
                const bool up = top[rs] > m[rs] + 60.0f;
                // in two halves: the totals may be 2^60 above the old reference, the new one 2^126 and more
                const float a = up ? ex2(0.5f * (m[rs] - top[rs])) : 1.0f;
                if (up) m[rs] = top[rs];
                l[rs] = l[rs] * a * a;
#pragma unroll
                for (int n = 0; n < NT; ++n)
                    tot[rs][n] = mul2(mul2(tot[rs][n], both(((spoilt[rs] >> (n >> 2)) & 1u) ? NAN : a)), both(a));
#pragma unroll
                for (int i = 0; i < 4 * UNIT; ++i) more |= lg[rs][i] < top[rs] - 28.0f && lg[rs][i] > m[rs] - 126.0f;
            }
            more = __any_sync(0xffffffffu, more);
        }
        for (;;) {  // once, but for probabilities more than 2^28 apart: those below wait for a pass of their own
            float rest[RS], f[RS], pr[RS][4 * UNIT];
#pragma unroll
            for (int rs = 0; rs < RS; ++rs) {
                const float ref = fmaxf(top[rs], kAttnNone);  // a unit that the row does not see: all probabilities 0
                const float sub = ref - lift;
                rest[rs] = -INFINITY;
#pragma unroll
                for (int i = 0; i < 4 * UNIT; ++i) {
                    pr[rs][i] = ex2(lg[rs][i] - sub);
                    if (more) {
                        if (lg[rs][i] < ref - 28.0f) {
                            pr[rs][i] = 0.0f;
                            rest[rs] = fmaxf(rest[rs], lg[rs][i]);
                        } else {
                            lg[rs][i] = -INFINITY;
                        }
                    }
                }
                float2 sum = make_float2(pr[rs][0], pr[rs][1]);
#pragma unroll
                for (int i = 2; i < 4 * UNIT; i += 2) sum = add2(sum, make_float2(pr[rs][i], pr[rs][i + 1]));
                f[rs] = ex2_small(sub - m[rs]);
                l[rs] = fmaf(sum.x + sum.y, f[rs], l[rs]);
            }
            uint32_t ph[RS][2 * UNIT];  // 16-bit activations: the probabilities in fp16
#pragma unroll
            for (int rs = 0; rs < RS; ++rs)
#pragma unroll
                for (int i = 0; i < 2 * UNIT; ++i) ph[rs][i] = MODE == A_SPLIT8 ? 0u : pack_h2(pr[rs][2 * i], pr[rs][2 * i + 1]);

            // ---- values, block by block of 32 channels
#pragma unroll
            for (int b = 0; b < NB; ++b) {
                float acc[4][4];
#pragma unroll
                for (int c = 0; c < UNIT; ++c) {
                    uint32_t a[4];
#pragma unroll
                    for (int o = 0; o < 2; ++o) {
                        const uint32_t d2 = prmt(vd[c][2 * o][b >> 1], vd[c][2 * o + 1][b >> 1], (b & 1) ? 0x7632u : 0x5410u);
                        if constexpr (MODE == A_SPLIT8) {
                            // rounded to fp16, and 2^12 times what that leaves
                            const float2 v = mul2(make_float2(pr[0][4 * c + 2 * o], pr[0][4 * c + 2 * o + 1]), half2_f32(d2));
                            const uint32_t h = pack_h2(v.x, v.y);
                            const float2 hv = half2_f32(h);
                            const float2 r = mul2(add2(v, make_float2(-hv.x, -hv.y)), both(4096.0f));
                            a[2 * o] = h;
                            a[2 * o + 1] = pack_h2(r.x, r.y);
                        } else {
                            a[2 * o] = h2_mul(ph[0][2 * c + o], d2);
                            a[2 * o + 1] = TWO ? h2_mul(ph[RS - 1][2 * c + o], d2) : attn_any();
                        }
                    }
                    const uint8_t* const blob = vb + c * kVB;
                    if constexpr (V4) {
                        const uint2 u2 = *reinterpret_cast<const uint2*>(blob + ((b >> 1) * 32 + lane) * 16 + (b & 1) * 8);
                        const uint32_t uw[2] = {u2.x, u2.y};
#pragma unroll
                        for (int k = 0; k < 2; ++k) {
                            const uint32_t q = uw[k], y = q >> 8;
                            // 1024 + q - 1032, and (1024 + 16 q) / 16 - 72
                            const uint32_t e0 = h2_sub((q & 0x000F000Fu) | 0x64006400u, 0x64086408u);
                            const uint32_t e1 = h2_sub((y & 0x000F000Fu) | 0x64006400u, 0x64086408u);
                            const uint32_t o0 = h2_fma((q & 0x00F000F0u) | 0x64006400u, 0x2C002C00u, 0xD480D480u);
                            const uint32_t o1 = h2_fma((y & 0x00F000F0u) | 0x64006400u, 0x2C002C00u, 0xD480D480u);
                            if (c == 0) attn_mma0(acc[2 * k], a, e0, e1), attn_mma0(acc[2 * k + 1], a, o0, o1);
                            else attn_mma(acc[2 * k], a, e0, e1), attn_mma(acc[2 * k + 1], a, o0, o1);
                        }
                    } else {
                        const uint4 u4 = *reinterpret_cast<const uint4*>(blob + (b * 32 + lane) * 16);
                        const uint32_t uw[4] = {u4.x, u4.y, u4.z, u4.w};
#pragma unroll
                        for (int k = 0; k < 4; ++k) {  // 1024 + (q + 128) - 1152
                            const uint32_t e0 = h2_sub(prmt(uw[k], 0x64646464u, 0x4140u), 0x64806480u);
                            const uint32_t e1 = h2_sub(prmt(uw[k], 0x64646464u, 0x4342u), 0x64806480u);
                            if (c == 0) attn_mma0(acc[k], a, e0, e1);
                            else attn_mma(acc[k], a, e0, e1);
                        }
                    }
                }
#pragma unroll
                for (int k = 0; k < 4; ++k) {
                    float2 r = make_float2(acc[k][0], acc[k][1]);
                    if constexpr (MODE == A_SPLIT8) r = fma2(make_float2(acc[k][2], acc[k][3]), both(0x1p-12f), r);
                    tot[0][4 * b + k] = fma2(r, both(f[0]), tot[0][4 * b + k]);
                    if constexpr (TWO)
                        tot[RS - 1][4 * b + k] = fma2(make_float2(acc[k][2], acc[k][3]), both(f[RS - 1]), tot[RS - 1][4 * b + k]);
                }
            }
            if (!more) break;
            more = false;
#pragma unroll
            for (int rs = 0; rs < RS; ++rs) {
                top[rs] = quad_max(rest[rs]);
                more |= top[rs] > m[rs] - 126.0f;
            }
            more = __any_sync(0xffffffffu, more);
            if (!more) break;
        }
    }

    // The reference moves to the sum's power of two (it may lag the largest score by 2^60); the row's sum.
    __device__ __forceinline__ float settle_reference(int rs, float* factor) {
        float sum = quad_sum(l[rs]);
        const int e = static_cast<int>(__float_as_uint(sum) >> 23) - 127;
        *factor = 1.0f;
        if (sum > 0.0f && e < 127) {
            *factor = pow2f(-e);
            sum *= *factor;
            m[rs] += static_cast<float>(e);
        }
        return sum;
    }
};

// Position of the share [lo, ...) in the list of all groups: the runs' exclusive
// prefix sums in s_scan (128), each run `per` sequences.
template <int UNIT>
__device__ __forceinline__ AttnWalk<UNIT> attn_find(const AttnParams& p, const int64_t* s_scan, int per, int64_t lo, int64_t n,
                                              int tile_rows, int lane) {
    int run = -1;
#pragma unroll
    for (int k = 0; k < 4; ++k) run += __popc(__ballot_sync(0xffffffffu, s_scan[lane + 32 * k] <= lo));
    AttnWalk<UNIT> w;
    w.left = n;
    w.b = run * per;
    int64_t rem = lo - s_scan[run];
    for (;;) {
        w.s = attn_seq(p, w.b, tile_rows, false);
        const int64_t c = attn_cost<UNIT>(w.s);
        if (rem < c) break;
        rem -= c;
        ++w.b;
    }
    const int span = attn_span<UNIT>(w.s);
    w.item = static_cast<int>(rem / span);
    w.ua = static_cast<int>(rem - static_cast<int64_t>(w.item) * span);
    return w;
}

// ---- items that several CTAs share (ggq_attn_plan.h)
template <int D>
__device__ __forceinline__ float* attn_part(const AttnParams& p, int c, int slot) {
    return p.parts + (2 * static_cast<int64_t>(c) + slot) * attn_part_floats(D);
}

__device__ __forceinline__ int atomic_add_acq_rel(int* p, int v) {
    int old;
    asm volatile("atom.add.acq_rel.gpu.global.s32 %0, [%1], %2;" : "=r"(old) : "l"(p), "r"(v) : "memory");
    return old;
}

// One thread, after the CTA's barrier: this CTA's piece has arrived.  *last: 1 if it
// completes its group of kJoin pieces.
template <int UNIT>
__device__ __forceinline__ void attn_arrive(const AttnParams& p, const AttnWalk<UNIT>& w, int64_t p0, int64_t N, int C,
                                            volatile int* last) {
    const AttnPieces q(p0, attn_span<UNIT>(w.s), N, C);
    const int g0 = q.group(static_cast<int>(blockIdx.x));
    int* const counter = p.pieces + q.piece_counter(g0);
    const bool is_last = atomic_add_acq_rel(counter, 1) == q.group_pieces(g0) - 1;
    if (is_last) *counter = 0;
    *last = is_last;
}

// The whole CTA, after the barrier that follows attn_arrive.
template <int D, int ROWS, int UNIT>
__device__ __noinline__ void attn_join(const AttnParams& p, const AttnWalk<UNIT>& w, int64_t p0, int64_t N, int C, int tid,
                                       volatile int* last) {
    if (!*last) return;
    const AttnPieces q(p0, attn_span<UNIT>(w.s), N, C);
    const AttnTile tile = attn_tile(p, w.s, w.item, ROWS);
    const int g0 = q.group(static_cast<int>(blockIdx.x));
    const bool groups = q.groups() > 1;
    for (int level = 0; level < 2; ++level) {
        const int from = level ? q.c0 : g0, step = level ? kJoin : 1, to = level ? q.c1 : g0 + q.group_pieces(g0) - 1;
        const bool done = level == 1 || !groups;
        constexpr int kQuads = (ROWS * D / 4 + kAttnThreads - 1) / kAttnThreads;
        float4 o[kQuads];
        float M[kQuads], L[kQuads];
#pragma unroll
        for (int k = 0; k < kQuads; ++k) {
            const int i = tid + k * kAttnThreads, row = i / (D / 4), d = 4 * (i - row * (D / 4));
            M[k] = kAttnNone, L[k] = 0.0f;
            o[k] = make_float4(0.f, 0.f, 0.f, 0.f);
            if (row >= ROWS) continue;
            for (int b = from; b <= to; b += 4 * step) {  // four pieces' loads in flight
                float pm[4], pl[4];
                float4 v[4];
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    const int c = min(b + e * step, to - (to - from) % step);
                    const float* const a = attn_part<D>(p, c, q.slot(c));
                    pm[e] = __ldcg(a + row), pl[e] = __ldcg(a + 16 + row);
                    v[e] = __ldcg(reinterpret_cast<const float4*>(a + 32 + row * D + d));
                }
                float top = M[k];
#pragma unroll
                for (int e = 0; e < 4; ++e)
                    if (b + e * step <= to) top = fmaxf(top, pm[e]);
                const float f0 = ex2(M[k] - top);
                M[k] = top;
                L[k] *= f0, o[k].x *= f0, o[k].y *= f0, o[k].z *= f0, o[k].w *= f0;
#pragma unroll
                for (int e = 0; e < 4; ++e)
                    if (b + e * step <= to) {
                        const float f = ex2(pm[e] - top);
                        L[k] = fmaf(pl[e], f, L[k]);
                        o[k].x = fmaf(v[e].x, f, o[k].x), o[k].y = fmaf(v[e].y, f, o[k].y);
                        o[k].z = fmaf(v[e].z, f, o[k].z), o[k].w = fmaf(v[e].w, f, o[k].w);
                    }
            }
        }
        float* const to_part = attn_part<D>(p, g0, q.slot(g0));
        if (!done) __syncthreads();  // the group's first piece is read: its place takes the result
#pragma unroll
        for (int k = 0; k < kQuads; ++k) {
            const int i = tid + k * kAttnThreads, row = i / (D / 4), d = 4 * (i - row * (D / 4));
            if (row >= ROWS) continue;
            if (done) {
                const float inv = L[k] != 0.0f ? 1.0f / L[k] : 0.0f;
                if (tile.r0 + row < tile.r_end)
                    attn_out4(p, w.s, tile.hk, tile.r0 + row, d, make_float4(o[k].x * inv, o[k].y * inv, o[k].z * inv, o[k].w * inv));
            } else {
                if (d == 0) to_part[row] = M[k], to_part[16 + row] = L[k];
                *reinterpret_cast<float4*>(to_part + 32 + row * D + d) = o[k];
            }
        }
        if (done) return;
        __syncthreads();
        if (tid == 0) {
            int* const counter = p.pieces + q.group_counter();
            const bool is_last = atomic_add_acq_rel(counter, 1) == q.groups() - 1;
            if (is_last) *counter = 0;
            *last = is_last;
        }
        __syncthreads();
        if (!*last) return;
    }
}

template <bool K4, bool V4, int D, int MODE>
__global__ void __launch_bounds__(kAttnThreads, AttnSmem<K4, V4, D, MODE>::kCtas)
    k_attn_stream(const __grid_constant__ AttnParams p) {
    using SM = AttnSmem<K4, V4, D, MODE>;
    constexpr int kRows = SM::kRows, NT = D / 8, S = SM::kStages, UNIT = SM::kUnit, RS = MODE == A_HALF16 ? 2 : 1;
    extern __shared__ __align__(128) uint8_t smem[];
    float* const s_tot = reinterpret_cast<float*>(smem + SM::oTot);
    uint4* const s_q = reinterpret_cast<uint4*>(smem + SM::oQ);
    float* const s_m = reinterpret_cast<float*>(smem + SM::oStat);
    float* const s_l = s_m + kAttnWarps * 8;
    int64_t* const s_scan = reinterpret_cast<int64_t*>(smem + SM::oScan);
    int64_t* const s_wsum = s_scan + 128;
    uint64_t* const s_full = reinterpret_cast<uint64_t*>(smem + SM::oBar);
    volatile int* const s_abort = reinterpret_cast<volatile int*>(s_full + kAttnWarps * S);
    volatile int* const s_last = s_abort + 1;
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    int* const s_copy = reinterpret_cast<int*>(smem + SM::oLast) + warp;  // this warp's last copy

    pdl_launch_dependents();
    if (tid == 0) {
        for (int i = 0; i < kAttnWarps * S; ++i) mbar_init(s_full + i, 1);
        *s_abort = 0;
        fence_barrier_init();
    }
    pdl_wait();

    // ---- plan: prefix sums of the sequences' costs over 128 runs of `per` sequences
    const int nseq = static_cast<int>(p.n_seqs), per = (nseq + 127) >> 7;
    int64_t mine = 0, incl = 0;
    for (int b = tid * per; b < min(nseq, (tid + 1) * per); ++b) {
        const AttnSeq s = attn_seq(p, b, kRows, blockIdx.x == 0);
        const int64_t cost = attn_cost<UNIT>(s);
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
    __syncthreads();
    {
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
    AttnWalk<UNIT> w = attn_find<UNIT>(p, s_scan, per, lo, hi - lo, kRows, lane);

    // ---- this warp's ring: it takes every fourth unit of the segments; a unit's copies start as
    // soon as the warp has done with the place's last one, the page id having been read a turn before
    const uint64_t policy = policy_evict_first();
    const int gpp = p.page >> 4;  // groups of a page
    AttnWalk<UNIT> fw = w;        // the segment whose units are fetched
    int fu = fw.first() + warp, fend = 0, fglo = 0, fghi = 0, fhk = 0;
    const int32_t* ftable = nullptr;
    const auto enter = [&]() {  // what the units of segment fw share; empty segments are passed over
        while (fw.left > 0 && fu >= fw.last()) {
            fw.next(p, kRows);
            fu = fw.first() + warp;
        }
        fend = fw.left > 0 ? fw.last() : 0;
        fglo = fw.s.glo;
        fghi = fw.s.ghi;
        fhk = fw.item / (fw.s.items / p.Hkv);
        ftable = p.table + fw.b * p.table_stride;
    };
    // lane l: page and place of the unit's group l (division by gpp as a multiplication that is at most
    // one too large)
    int fplace = 0, fpage = 0;
    bool bad_page = false;
    const auto seek = [&]() {
        const int g = fglo + UNIT * fu + lane;
        if (lane >= UNIT || fu >= fend || g >= fghi) return;
        int q = g;
        fplace = 0;
        if (gpp > 1) {
            q = static_cast<int>(__umulhi(static_cast<uint32_t>(g), p.page_magic));
            fplace = g - q * gpp;
            if (fplace < 0) --q, fplace += gpp;
        }
        fpage = ftable[q];
    };
    const auto fetch = [&](int place, uint32_t parity) {
        if (fu >= fend) return;
        const int at = warp * S + place;
        const int n = min(UNIT, fghi - fglo - UNIT * fu);  // groups of the unit
        const bool joined = __shfl_sync(0xffffffffu, fplace, 0) + n <= gpp;  // of one page: one copy
        if (lane == 0) mbar_arrive_expect_tx(s_full + at, n * (SM::kStage / UNIT));
        __syncwarp();
        if (lane < (joined ? 1 : n)) {
            const int copies = joined ? n : 1;
            if (static_cast<uint32_t>(fpage) >= static_cast<uint32_t>(p.n_pages)) fpage = 0, bad_page = true;
            const int64_t blob = (static_cast<int64_t>(fpage) * p.Hkv + fhk) * gpp + fplace;
            uint8_t* const dst = smem + SM::oRing + at * SM::kStage;
            bulk_g2s(dst + lane * SM::kKB, p.k + blob * SM::kKB, copies * SM::kKB, s_full + at, policy);
            bulk_g2s(dst + UNIT * SM::kKB + lane * SM::kVB, p.v + blob * SM::kVB, copies * SM::kVB, s_full + at, policy);
        }
        fu += kAttnWarps;
        if (fu >= fend) {
            enter();
            if (fend == 0) *s_copy = attn_last_copy(place, parity);
        }
        seek();
    };
    enter();
    *s_copy = fend == 0 ? kNoCopies : kMoreCopies;
    seek();
    for (int i = 0; i < S; ++i) fetch(i, 0u);

    // ---- segments
    const int g8 = lane >> 2, t4 = lane & 3;
    int slot = 0;
    uint32_t phase = 0;
    const auto skip_empty = [&](AttnWalk<UNIT>& at) {  // a share may end before an item's units
        while (at.left > 0 && at.last() <= 0) at.next(p, kRows);
    };
    // an item that this CTA has added a piece to: whether it was the last one is known after the next barrier
    bool pending = false;
    AttnWalk<UNIT> pw = w;
    int64_t pp0 = 0;
    const auto settle = [&]() {
        if (!pending) return;
        pending = false;
        attn_join<D, kRows, UNIT>(p, pw, pp0, N, C, tid, s_last);
    };
    skip_empty(w);
    while (w.left > 0) {
        const AttnSeq sq = w.s;
        const int ua = w.first(), ub = w.last();
        const int64_t at0 = hi - w.left;               // the segment's first position
        const AttnTile tile = attn_tile(p, sq, w.item, kRows);
        const int hk = tile.hk, r0 = tile.r0, r_end = tile.r_end;
        AttnRows<K4, V4, D, MODE, UNIT> rows;
        rows.template begin<kAttnWarps>(p, sq, hk, r0, r_end, s_q, warp, lane);
        __syncthreads();
        settle();
        for (int u = ua + warp; u < ub; u += kAttnWarps) {
            const int at = warp * S + slot, g = sq.glo + UNIT * u;
            if (!__all_sync(0xffffffffu, mbar_test(s_full + at, phase))) {
                bool ok = !*s_abort && mbar_wait(s_full + at, phase);
                ok = __all_sync(0xffffffffu, ok);
                if (!ok) {
                    *s_abort = 1;
                    set_error(p.err, DEV_ERR_TIMEOUT);
                    break;
                }
            }
            const uint8_t* const kb = smem + SM::oRing + at * SM::kStage;
            const uint8_t* const vb = kb + UNIT * SM::kKB;

            rows.unit(p, s_q, kb, vb, g, lane);
            __syncwarp();
            fetch(slot, phase ^ 1u);
            if (++slot == S) slot = 0, phase ^= 1u;
        }
        // ---- the segment's result: the four warps' parts, 8 rows at a time
        const int n_units = attn_units<UNIT>(sq);
        const bool whole = ua == 0 && ub == n_units;
        float* const part = attn_part<D>(p, c, at0 == lo ? 0 : 1);
        float* const s_mine = s_tot + warp * 8 * SM::kRowPitch;
#pragma unroll
        for (int rs = 0; rs < RS; ++rs) {
            float a;
            const float sum = rows.settle_reference(rs, &a);
#pragma unroll
            for (int c0 = 0; c0 < D; c0 += SM::kMerge) {
                if (rs > 0 || c0 > 0) __syncthreads();
#pragma unroll
                for (int n = 0; n < SM::kMerge / 8; ++n)
                    *reinterpret_cast<float2*>(s_mine + g8 * SM::kRowPitch + 8 * n + 2 * t4) = mul2(rows.tot[rs][c0 / 8 + n], both(a));
                if (t4 == 0) {
                    s_m[warp * 8 + g8] = rows.m[rs];
                    s_l[warp * 8 + g8] = sum;
                }
                __syncthreads();
                for (int i = tid; i < 8 * SM::kMerge / 4; i += kAttnThreads) {
                    const int r8 = i / (SM::kMerge / 4), d = 4 * (i - r8 * (SM::kMerge / 4)), row = 8 * rs + r8;
                    if (whole && r0 + row >= r_end) break;
                    float M = kAttnNone, L = 0.0f;
#pragma unroll
                    for (int k = 0; k < kAttnWarps; ++k) M = fmaxf(M, s_m[k * 8 + r8]);
                    float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
                    for (int k = 0; k < kAttnWarps; ++k) {
                        const float f = ex2(s_m[k * 8 + r8] - M);
                        const float4 v = *reinterpret_cast<const float4*>(s_tot + (k * 8 + r8) * SM::kRowPitch + d);
                        L = fmaf(s_l[k * 8 + r8], f, L);
                        o.x = fmaf(v.x, f, o.x), o.y = fmaf(v.y, f, o.y), o.z = fmaf(v.z, f, o.z), o.w = fmaf(v.w, f, o.w);
                    }
                    if (whole) {
                        const float inv = L != 0.0f ? 1.0f / L : 0.0f;
                        attn_out4(p, sq, hk, r0 + row, c0 + d, make_float4(o.x * inv, o.y * inv, o.z * inv, o.w * inv));
                    } else {
                        if (c0 + d == 0) part[row] = M, part[16 + row] = L;
                        *reinterpret_cast<float4*>(part + 32 + row * D + c0 + d) = o;
                    }
                }
            }
        }
        if (!whole) {
            pending = true;
            pw = w;
            pp0 = at0 - w.ua;  // the item's first position
            __syncthreads();
            if (tid == 0) attn_arrive<UNIT>(p, pw, pp0, N, C, s_last);
        }
        w.next(p, kRows);
        skip_empty(w);
    }
    if (bad_page) set_error(p.err, DEV_ERR_BAD_PLACE);
    // a wait gave up: let the copies in flight land before the CTA ends
    if (*s_abort) attn_drain(*s_copy, S, slot, phase, [&](int at, uint32_t parity) { mbar_wait(s_full + warp * S + at, parity); });
    __syncthreads();
    settle();
}

// Launch of one (K format, V format, D, mode); the grid fills the SMs once.
template <bool K4, bool V4, int D, int MODE>
cudaError_t launch_attn_stream(const AttnParams& p, int nsm, cudaStream_t s) {
    using SM = AttnSmem<K4, V4, D, MODE>;
    static std::atomic<bool> set[kMaxDevices] = {};
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    if (dev < 0 || dev >= kMaxDevices) return cudaErrorInvalidDevice;
    if (!set[dev].load(std::memory_order_acquire)) {
        e = cudaFuncSetAttribute(k_attn_stream<K4, V4, D, MODE>, cudaFuncAttributeMaxDynamicSharedMemorySize, SM::kTotal);
        if (e != cudaSuccess) return e;
        set[dev].store(true, std::memory_order_release);
    }
    static_assert(SM::kCtas * attn_part_floats(D) <= kAttnWideCtas * attn_part_floats(256), "scratch of the partial results");
    const int64_t tiles = (static_cast<int64_t>(p.max_q) * p.G + SM::kRows - 1) / SM::kRows;
    const int64_t units = p.n_seqs * p.Hkv * tiles * ((static_cast<int64_t>(p.max_len) + 16 * SM::kUnit - 1) / (16 * SM::kUnit) + 1 + kItemCost);
    int64_t grid = (units + p.min_share - 1) / p.min_share;
    if (grid > static_cast<int64_t>(nsm) * SM::kCtas) grid = static_cast<int64_t>(nsm) * SM::kCtas;
    if (grid > kAttnMaxCtas) grid = kAttnMaxCtas;
    if (grid < 1) grid = 1;
    return launch_pdl(k_attn_stream<K4, V4, D, MODE>, dim3(static_cast<unsigned>(grid)), dim3(kAttnThreads), SM::kTotal, s, p);
}

template <bool K4, bool V4, int D>
cudaError_t launch_attn_stream_mode(const AttnParams& p, int nsm, cudaStream_t s) {
    if (p.dtype == 0 || p.cap > kWideCap) return launch_attn_stream<K4, V4, D, A_SPLIT8>(p, nsm, s);
    if (static_cast<int64_t>(p.max_q) * p.G <= 8) return launch_attn_stream<K4, V4, D, A_HALF8>(p, nsm, s);
    return launch_attn_stream<K4, V4, D, A_HALF16>(p, nsm, s);
}

}  // namespace ggq
