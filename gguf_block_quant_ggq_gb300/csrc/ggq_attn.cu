// ggq_attn.cu -- attention over the packed key/value cache, one warp for each
// query row and head: channels over the lanes, keys one after the other with
// the running maximum and sum of the softmax.
#include "ggq_attn.cuh"
#include "ggq_device.cuh"
#include "ggq_internal.h"

namespace ggq {

namespace {

__device__ __forceinline__ float cache_value(const uint8_t* blob, bool q4, bool v, int D, int r, int d) {
    const int o = r >> 3;
    int lane, f, nib;
    if (!v) {
        const int j = d >> 4, i = d & 3;
        lane = 4 * (r & 7) + ((d & 15) >> 2);
        f = q4 ? o * (D >> 5) + (j >> 1) : o * (D >> 4) + j;
        nib = q4 ? 4 * (i & 1) + (i >> 1) + 2 * (j & 1) : 2 * i;
    } else {
        const int n = d >> 3;
        lane = 4 * (d & 7) + ((r & 7) >> 1);
        f = q4 ? n >> 1 : n;
        nib = q4 ? 4 * (r & 1) + 2 * o + (n & 1) : 2 * (2 * o + (r & 1));
    }
    const int byte = blob[kv_word(f, lane) + (nib >> 1)];
    const float q = q4 ? static_cast<float>(((byte >> (4 * (nib & 1))) & 15) - 8) : static_cast<float>(byte - 128);
    return q * __half2float(reinterpret_cast<const __half*>(blob + kv_quant_bytes(q4, D))[r * (D >> 5) + (d >> 5)]);
}

template <typename T>
__global__ void __launch_bounds__(128) k_attn(const __grid_constant__ AttnParams p) {
    pdl_launch_dependents();
    pdl_wait();
    const int lane = threadIdx.x & 31;
    const int64_t w = (static_cast<int64_t>(blockIdx.x) * blockDim.x + threadIdx.x) >> 5;
    if (w >= p.n_tokens * p.H) return;
    const int64_t row = w / p.H;
    const int h = static_cast<int>(w - row * p.H), hk = h / p.G, nb = p.D >> 5;
    int64_t b = row, first = row, end = row + 1;
    if (p.q_start) {
        int64_t lo = 0, hi = p.n_seqs;  // the last sequence that starts at or before the row
        while (lo + 1 < hi) {
            const int64_t mid = (lo + hi) >> 1;
            if (p.q_start[mid] <= row) lo = mid; else hi = mid;
        }
        b = lo;
        first = p.q_start[b];
        end = p.q_start[b + 1];
        if (row < first || row >= end) return;
    }
    int len = p.lens[b];
    if (len > p.max_len || end - first > p.max_q) {
        set_error(p.err, DEV_ERR_BAD_PLACE);
        len = min(len, p.max_len);
        if (row - first >= p.max_q) return;
    }
    const int64_t pos = static_cast<int64_t>(len) - (end - first) + (row - first);
    const T* const qp = static_cast<const T*>(p.q) + row * p.q_token + h * p.q_head;
    float q[8], acc[8];
    for (int c = 0; c < nb; ++c) {
        q[c] = ld1(qp + 32 * c + lane) * p.scale;
        acc[c] = 0.0f;
    }
    const float slope = p.slopes ? p.slopes[h] : 0.0f;
    float m = -INFINITY, l = 0.0f;
    const int64_t from = p.window > 0 && pos - p.window + 1 > 0 ? pos - p.window + 1 : 0;
    const int64_t kb = kv_blob_bytes(p.k_q4, p.D), vb = kv_blob_bytes(p.v_q4, p.D);
    for (int64_t j = from; j <= pos; ++j) {
        int64_t pg = p.table[b * p.table_stride + j / p.page];
        if (pg < 0 || pg >= p.n_pages) {
            set_error(p.err, DEV_ERR_BAD_PLACE);
            pg = 0;
        }
        const int64_t blob = (pg * p.Hkv + hk) * (p.page >> 4) + ((j % p.page) >> 4);
        const int r = static_cast<int>(j & 15);
        float s = 0.0f;
        for (int c = 0; c < nb; ++c) s += q[c] * cache_value(p.k + blob * kb, p.k_q4, false, p.D, r, 32 * c + lane);
        for (int d = 16; d >= 1; d >>= 1) s += __shfl_xor_sync(0xffffffffu, s, d);
        if (p.cap > 0.0f) s = p.cap * tanhf(s / p.cap);
        s += slope * static_cast<float>(j - pos);
        const float mn = fmaxf(m, s);
        const float a = m == -INFINITY ? 0.0f : expf(m - mn), e = mn == -INFINITY ? 0.0f : expf(s - mn);
        m = mn;
        l = l * a + e;
        for (int c = 0; c < nb; ++c)
            acc[c] = acc[c] * a + e * cache_value(p.v + blob * vb, p.v_q4, true, p.D, r, 32 * c + lane);
    }
    T* const op = static_cast<T*>(p.out) + row * p.out_token + h * p.out_head;
    for (int c = 0; c < nb; ++c) st1(op + 32 * c + lane, l > 0.0f ? acc[c] / l : 0.0f);
}

}  // namespace

cudaError_t launch_attention(const AttnParams& p, cudaStream_t s) {
    const dim3 grid(static_cast<unsigned>((p.n_tokens * p.H + 3) / 4));
    if (p.dtype == 0) return launch_pdl(k_attn<float>, grid, dim3(128), 0, s, p);
    if (p.dtype == 1) return launch_pdl(k_attn<__half>, grid, dim3(128), 0, s, p);
    return launch_pdl(k_attn<__nv_bfloat16>, grid, dim3(128), 0, s, p);
}

}  // namespace ggq
