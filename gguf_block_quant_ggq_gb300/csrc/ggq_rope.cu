// ggq_rope.cu -- the rotation of positions by itself, and its table.
//
// The rotation reads and writes each value once: bound by memory at many tokens, by the launch
// at few.  A thread keeps its pairs' table entries (8 bytes a pair, fetched once) while it goes
// through the heads, so the table costs nothing next to the rows.
//
// The table: an angle is position * frequency, and only its fraction of a turn matters.  A
// frequency is held as a 64-bit fraction of a turn (rounded from fp64: off by 2^-56 of a turn),
// the product with the position wraps around by itself, and what is left, less than an eighth
// of a turn from a quarter, goes to fp32 with 2^-28 of a turn and to sincospi: exact to the
// last bits at any position, with no fp64 instruction (whose rate is a sixty-fourth of fp32's
// on this part).  Made once: bound by the division and the 64-bit products of each entry (131072 positions of 64
// pairs 58 us, where the writes take 10).
#include <algorithm>

#include "ggq_internal.h"
#include "ggq_rope.cuh"

namespace ggq {

namespace {

template <int V, typename T>
__global__ void __launch_bounds__(kRotateThreads) k_rotate(const __grid_constant__ RotateParams p) {
    pdl_launch_dependents();
    pdl_wait();
    const int64_t r0 = static_cast<int64_t>(blockIdx.x) * p.rows_at_once;
    const int h0 = static_cast<int>(blockIdx.y) * p.heads_at_once;
    rotate_tile<V, T>(p, r0, min(p.T, r0 + p.rows_at_once), h0, min(p.H, h0 + p.heads_at_once));
}

template <typename T>
cudaError_t launch(RotateParams p, int v, cudaStream_t s) {
    p.units = p.r.half / v + ((p.D - 2 * p.r.half) / v + 1) / 2;
    p.rows_at_once = std::max(1, kRotateThreads / p.units);
    // The heads are split while there are few CTAs
    const int64_t tiles = (p.T + p.rows_at_once - 1) / p.rows_at_once;
    p.heads_at_once = p.H;
    while (p.heads_at_once > 1 && tiles * ((p.H + p.heads_at_once - 1) / p.heads_at_once) < 1216) p.heads_at_once = (p.heads_at_once + 1) / 2;
    const dim3 grid(static_cast<unsigned>(tiles), static_cast<unsigned>((p.H + p.heads_at_once - 1) / p.heads_at_once));
    if (v == 8) {
        if constexpr (sizeof(T) == 2) return launch_pdl(k_rotate<8, T>, grid, dim3(kRotateThreads), 0, s, p);
    }
    if (v == 4) return launch_pdl(k_rotate<4, T>, grid, dim3(kRotateThreads), 0, s, p);
    return launch_pdl(k_rotate<1, T>, grid, dim3(kRotateThreads), 0, s, p);
}

__global__ void __launch_bounds__(256) k_rotary_table(const __grid_constant__ RotaryTableParams p) {
    pdl_launch_dependents();
    pdl_wait();
    const int64_t n = p.n * p.half;
    for (int64_t i = static_cast<int64_t>(blockIdx.x) * 256 + threadIdx.x; i < n; i += static_cast<int64_t>(gridDim.x) * 256) {
        const int64_t row = i / p.half;
        const uint64_t turn = static_cast<uint64_t>(p.first + row) * p.turns[i - row * p.half];
        const uint64_t near = turn + (1ull << 61);  // its quarter is the nearest one
        const int quarter = static_cast<int>(near >> 62);
        const int rest = static_cast<int>(static_cast<int64_t>((near & ((1ull << 62) - 1)) - (1ull << 61)) >> 30);
        float s, c;
        sincospif(static_cast<float>(rest) * 0x1p-33f, &s, &c);
        const float a = quarter & 1 ? s : c, b = quarter & 1 ? c : s;
        p.table[i] = make_float2((quarter == 1 || quarter == 2 ? -a : a) * p.magnitude, (quarter & 2 ? -b : b) * p.magnitude);
    }
}

}  // namespace

int rotate_vector(const RotateParams& p, int dtype) {
    const int size = dtype == 0 ? 4 : 2;
    for (int v = dtype == 0 ? 4 : 8; v > 1; v -= 4) {
        const int bytes = v * size;
        const auto whole = [&](const void* at, int64_t token, int64_t head) {
            return aligned_to(at, bytes) && (p.T < 2 || token % v == 0) && (p.H < 2 || head % v == 0);
        };
        if (p.r.half % v == 0 && p.r.first % v == 0 && p.D % v == 0 && aligned_to(p.r.table, 16) &&
            whole(p.x, p.x_token, p.x_head) && whole(p.out, p.out_token, p.out_head))
            return v;
    }
    return 1;
}

cudaError_t launch_rotate(RotateParams p, int dtype, cudaStream_t s) {
    if (p.T == 0) return cudaSuccess;
    const int v = rotate_vector(p, dtype);
    if (dtype == 0) return launch<float>(p, v, s);
    if (dtype == 1) return launch<__half>(p, v, s);
    return launch<__nv_bfloat16>(p, v, s);
}

cudaError_t launch_rotary_table(const RotaryTableParams& p, cudaStream_t s) {
    const int64_t n = p.n * p.half;
    if (n == 0) return cudaSuccess;
    return launch_pdl(k_rotary_table, dim3(static_cast<unsigned>(std::min<int64_t>((n + 255) / 256, 152 * 8))), dim3(256), 0, s, p);
}

}  // namespace ggq
