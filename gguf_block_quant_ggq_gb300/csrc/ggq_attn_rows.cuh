// ggq_attn_rows.cuh -- attention of many fp32 query rows (prompts) over the packed
// cache on mma.sync, for heads of 256 channels (whose scores, probabilities and outputs
// tensor memory does not hold at once).
//
// The same step as the streaming kernel's (a warp's 8 rows against a unit of keys,
// operands split so that 22 bits of the products count), laid out for many rows: a
// CTA takes 64 rows of one kv head of one sequence, 8 a warp, and all its warps read
// the same ring of units in shared memory, up to the last key that a row sees.
// Bound by instructions (unpacking and scaling, about 1000 a warp, unit and 8 rows):
// 4096 causal rows, 16 heads on 8: 1.73 ms (the streaming kernel: 3.5 ms), 79 TFLOP/s.
#pragma once
#include <atomic>

#include "ggq_attn_stream.cuh"

namespace ggq {

constexpr int kRowsWarps = 8, kRowsThreads = kRowsWarps * 32, kRowsTile = 8 * kRowsWarps;

template <bool K4, bool V4, int D>
struct RowsSmem {
    static constexpr int kUnit = 1;  // 16 keys: a warp's 8 rows of outputs leave no registers for more
    static constexpr int kKB = kv_blob_bytes(K4, D), kVB = kv_blob_bytes(V4, D), kStage = kUnit * (kKB + kVB);
    static constexpr int kStages = 6;
    static constexpr int kQ = D / 16 * 32 * 16;  // bytes of a warp's query operand
    static constexpr int oQ = kStages * kStage, oBar = oQ + kRowsWarps * kQ, kTotal = oBar + 2 * kStages * 8 + 16;
};

template <bool K4, bool V4, int D>
__global__ void __launch_bounds__(kRowsThreads, 1) k_attn_rows(const __grid_constant__ AttnParams p) {
    using SM = RowsSmem<K4, V4, D>;
    constexpr int UNIT = SM::kUnit, S = SM::kStages, NT = D / 8;
    extern __shared__ __align__(128) uint8_t smem[];
    uint64_t* const s_full = reinterpret_cast<uint64_t*>(smem + SM::oBar);
    uint64_t* const s_empty = s_full + S;
    volatile int* const s_abort = reinterpret_cast<volatile int*>(s_empty + S);
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, g8 = lane >> 2, t4 = lane & 3;

    pdl_launch_dependents();
    pdl_wait();
    const int b = static_cast<int>(blockIdx.x / static_cast<unsigned>(p.Hkv)), hk = static_cast<int>(blockIdx.x) - b * p.Hkv;
    const int tile = static_cast<int>(gridDim.y - 1 - blockIdx.y);  // the heaviest (last) rows first
    const AttnSeq sq = attn_seq(p, b, kRowsTile, blockIdx.y == 0 && hk == 0);
    const int R = min(sq.rows, p.max_q) * p.G, c0 = tile * kRowsTile;
    if (c0 >= R) return;
    const int active = min(kRowsWarps, (R - c0 + 7) / 8);  // warps that have rows
    const int r0 = c0 + 8 * warp, r_end = min(R, r0 + 8), from = sq.len - sq.rows;
    // units that some row of the tile sees, and some row of this warp
    const auto group_of = [&](int r) { return p.window > 0 && from + r / p.G - p.window + 1 > 0 ? (from + r / p.G - p.window + 1) >> 4 : 0; };
    const auto end_of = [&](int r) { return from + r / p.G < 0 ? 0 : ((from + r / p.G) >> 4) + 1; };
    const int glo = group_of(c0), ghi = end_of(min(R, c0 + kRowsTile) - 1);
    const int units = ghi > glo ? (ghi - glo + UNIT - 1) / UNIT : 0;
    if (tid == 0) {
        for (int i = 0; i < S; ++i) {
            mbar_init(s_full + i, 1);
            mbar_init(s_empty + i, static_cast<uint32_t>(active));
        }
        *s_abort = 0;
        fence_barrier_init();
    }
    __syncthreads();
    if (warp >= active) return;  // no rows: no barrier follows

    // ---- warp 0 feeds the ring: lane l the unit's group l, whose page id it has read a unit before
    const uint64_t policy = policy_evict_last();  // the other tiles of the head read it too
    const int gpp = p.page >> 4;
    const int32_t* const table = p.table + b * p.table_stride;
    int fu = 0, fplace = 0, fpage = 0;
    bool bad_page = false;
    const auto seek = [&]() {
        const int g = glo + UNIT * fu + lane;
        if (lane >= UNIT || fu >= units || g >= ghi) return;
        int q = g;
        fplace = 0;
        if (gpp > 1) {
            q = static_cast<int>(__umulhi(static_cast<uint32_t>(g), p.page_magic));
            fplace = g - q * gpp;
            if (fplace < 0) --q, fplace += gpp;
        }
        fpage = table[q];
    };
    const auto fetch = [&]() {  // unit fu into its place
        if (fu >= units) return true;
        const int at = fu % S, n = min(UNIT, ghi - glo - UNIT * fu);
        if (fu >= S) {
            bool ok = !*s_abort && mbar_wait(s_empty + at, ((fu / S) - 1) & 1);
            ok = __all_sync(0xffffffffu, ok);
            if (!ok) return false;
        }
        if (lane == 0) mbar_arrive_expect_tx(s_full + at, n * (SM::kStage / UNIT));
        __syncwarp();
        if (lane < n) {
            if (static_cast<uint32_t>(fpage) >= static_cast<uint32_t>(p.n_pages)) fpage = 0, bad_page = true;
            const int64_t blob = (static_cast<int64_t>(fpage) * p.Hkv + hk) * gpp + fplace;
            uint8_t* const dst = smem + at * SM::kStage;
            bulk_g2s(dst + lane * SM::kKB, p.k + blob * SM::kKB, SM::kKB, s_full + at, policy);
            bulk_g2s(dst + UNIT * SM::kKB + lane * SM::kVB, p.v + blob * SM::kVB, SM::kVB, s_full + at, policy);
        }
        ++fu;
        seek();
        return true;
    };
    if (warp == 0) {
        seek();
        for (int i = 0; i < S; ++i) fetch();
    }

    AttnRows<K4, V4, D, A_SPLIT8, UNIT> rows;
    uint4* const s_q = reinterpret_cast<uint4*>(smem + SM::oQ + warp * SM::kQ);
    rows.template begin<1>(p, sq, hk, r0, r_end, s_q, 0, lane);
    __syncwarp();
    const int my_lo = group_of(r0), my_hi = end_of(r_end - 1);
    for (int u = 0; u < units; ++u) {
        const int at = u % S, g = glo + UNIT * u;
        if (!__all_sync(0xffffffffu, mbar_test(s_full + at, (u / S) & 1))) {
            bool ok = !*s_abort && mbar_wait(s_full + at, (u / S) & 1);
            ok = __all_sync(0xffffffffu, ok);
            if (!ok) {
                *s_abort = 1;
                set_error(p.err, DEV_ERR_TIMEOUT);
                break;
            }
        }
        const uint8_t* const kb = smem + at * SM::kStage;
        if (g < my_hi && g + UNIT > my_lo) rows.unit(p, s_q, kb, kb + UNIT * SM::kKB, g, lane);
        __syncwarp();
        if (lane == 0) mbar_arrive(s_empty + at);
        // the place of the unit before this one: every warp has left it, or soon will
        if (warp == 0 && u >= 1 && !fetch()) {
            *s_abort = 1;
            set_error(p.err, DEV_ERR_TIMEOUT);
            break;
        }
    }
    if (warp == 0) {
        if (bad_page) set_error(p.err, DEV_ERR_BAD_PLACE);
        if (*s_abort)  // let the copies in flight land before the CTA ends
            for (int i = fu > S ? fu - S : 0; i < fu; ++i) mbar_wait(s_full + i % S, (i / S) & 1);
    }
    float a;
    const float sum = rows.settle_reference(0, &a);
    const float inv = sum != 0.0f ? a / sum : 0.0f;
    if (r0 + g8 < r_end) {
        const int r = r0 + g8, i = r / p.G, h = hk * p.G + r - i * p.G;
        float* const out = static_cast<float*>(p.out) + (sq.first + i) * p.out_token + h * p.out_head + 2 * t4;
#pragma unroll
        for (int n = 0; n < NT; ++n) *reinterpret_cast<float2*>(out + 8 * n) = mul2(rows.tot[0][n], both(inv));
    }
}

template <bool K4, bool V4, int D>
cudaError_t launch_attn_rows_one(const AttnParams& p, cudaStream_t s) {
    using SM = RowsSmem<K4, V4, D>;
    static_assert(SM::kTotal <= kSmemLimit, "shared memory");
    static std::atomic<bool> set[kMaxDevices] = {};
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    if (dev < 0 || dev >= kMaxDevices) return cudaErrorInvalidDevice;
    if (!set[dev].load(std::memory_order_acquire)) {
        e = cudaFuncSetAttribute(k_attn_rows<K4, V4, D>, cudaFuncAttributeMaxDynamicSharedMemorySize, SM::kTotal);
        if (e != cudaSuccess) return e;
        set[dev].store(true, std::memory_order_release);
    }
    const int64_t tiles = (static_cast<int64_t>(p.max_q) * p.G + kRowsTile - 1) / kRowsTile;
    return launch_pdl(k_attn_rows<K4, V4, D>, dim3(static_cast<unsigned>(p.n_seqs * p.Hkv), static_cast<unsigned>(tiles)),
                      dim3(kRowsThreads), SM::kTotal, s, p);
}

template <int D>
cudaError_t launch_attn_rows_dim(const AttnParams& p, cudaStream_t s) {
    if (p.k_q4) return p.v_q4 ? launch_attn_rows_one<true, true, D>(p, s) : launch_attn_rows_one<true, false, D>(p, s);
    return p.v_q4 ? launch_attn_rows_one<false, true, D>(p, s) : launch_attn_rows_one<false, false, D>(p, s);
}

}  // namespace ggq
