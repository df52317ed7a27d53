// ggq_kv.cu -- quantizing keys and values into the paged cache and reading them back.
//
// Mathematics: per token and 32 channels, Q8_0 d = amax * (1/127), q = round(x / d);
// Q4_0 d = m / -8 with m the first value of the largest magnitude, q = floor(x /
// d + 8.5) in 0..15.  Bound by memory at a prompt's sizes: each value is read once
// and stands in the cache for 17/16 (Q8_0) or 9/16 (Q4_0) bytes.
//
// A CTA takes 16 consecutive rows of some heads' keys or values, the windows being
// laid so that the first row's run of slots meets them on groups of 16.  A thread
// has eight channels of a row, four threads a block.  Rows whose slots fill an
// aligned group (the tokens of a prompt) pass through the group's blob in shared
// memory, which is written or read in whole lines; other rows (one token of each
// sequence) go to or come from their blob directly.  Bound at 16384 tokens of 8 heads of
// 128 channels by instructions (bf16 to Q8_0 and Q4_0: 33 us, issue slots 65% used, where
// its 94 MB take 14; back to fp32: 30 us, its 161 MB 24), at a decode step's by latency (5
// us for both).
#include <algorithm>

#include "ggq_device.cuh"
#include "ggq_internal.h"
#include "ggq_kv.cuh"
#include "ggq_rope.cuh"

namespace ggq {

namespace {

constexpr int kKvThreads = 128;
constexpr int kKvRows = 16;

// Byte offsets inside a blob; in its image in shared memory (IMAGE) the 512-byte
// lines are 592 bytes apart and their upper halves 64 bytes further on, so that the
// lanes that take a row's channels apart meet different banks.
template <bool IMAGE>
__device__ __forceinline__ constexpr int place(int f, int l) {
    return (f >> 2) * (IMAGE ? 592 : 512) + l * 16 + (IMAGE ? (l >> 4) * 64 : 0) + (f & 3) * 4;
}
template <bool IMAGE>
__host__ __device__ constexpr int scales_at(bool q4, int D) { return kv_quant_bytes(q4, D) / 512 * (IMAGE ? 592 : 512); }

// Eight consecutive channels of a row; four neighbouring lanes hold a block of 32.
// Returns the stored quants and the block's scale.
template <bool Q4>
__device__ __forceinline__ float quantize8(const float (&x)[8], uint32_t (&q)[8]) {
    float amax = 0.0f;
#pragma unroll
    for (int i = 0; i < 8; ++i) amax = fmaxf(amax, fabsf(x[i]));
    amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, 1));
    amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, 2));
    float d;
    if constexpr (Q4) {
        // the sign of the first value of that magnitude
        uint32_t first = 255u;
        const uint32_t base = 16u * (threadIdx.x & 3u);
#pragma unroll
        for (int i = 7; i >= 0; --i)
            if (fabsf(x[i]) == amax) first = base + 2u * i + (__float_as_uint(x[i]) >> 31);
        first = min(first, __shfl_xor_sync(0xffffffffu, first, 1));
        first = min(first, __shfl_xor_sync(0xffffffffu, first, 2));
        d = __fmul_rn((first & 1u) ? -amax : amax, -0.125f);
    } else {
        d = __fmul_rn(amax, 1.0f / 127.0f);
    }
    const float id = d != 0.0f ? __frcp_rn(d) : 0.0f;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        const float v = __fmul_rn(x[i], id);
        if constexpr (Q4) {
            q[i] = static_cast<uint32_t>(static_cast<int>(fminf(fmaxf(__fadd_rn(v, 8.5f), 0.0f), 15.0f)));
        } else {
            // round half away from zero: the largest float below 1/2 added, then truncated
            const float c = fminf(fmaxf(v, -127.0f), 127.0f);
            q[i] = static_cast<uint32_t>(static_cast<int>(__fadd_rn(c, copysignf(0x1.fffffep-2f, c))) + 128);
        }
    }
    return d;
}

// Writes eight quantized channels c .. c + 7 of the token at place r of a blob (in
// shared or global memory).  All lanes of the warp take part; `there`: this one writes.
template <bool IMAGE, bool Q4, bool V, int D>
__device__ __forceinline__ void put8(uint8_t* blob, int r, int c, const uint32_t (&q)[8], float d, bool there) {
    constexpr int NB = D / 32;
    if (there && (threadIdx.x & 3) == 0)
        reinterpret_cast<__half*>(blob + scales_at<IMAGE>(Q4, D))[r * NB + (c >> 5)] = __float2half_rn(d);
    const int o = r >> 3;
    if constexpr (!V) {
        const int lane = 4 * (r & 7) + ((c & 15) >> 2), j = c >> 4;  // words of lanes `lane` and `lane` + 1
        if constexpr (Q4) {
            uint32_t w[2];
#pragma unroll
            for (int k = 0; k < 2; ++k) {
                w[k] = (q[4 * k] | q[4 * k + 1] << 16 | q[4 * k + 2] << 4 | q[4 * k + 3] << 20) << (8 * (j & 1));
                w[k] |= __shfl_xor_sync(0xffffffffu, w[k], 2);
            }
            // both halves of 16 channels have the words: each writes one
            if (there) *reinterpret_cast<uint32_t*>(blob + place<IMAGE>(o * NB + (j >> 1), lane + (j & 1))) = w[j & 1];
        } else if (there) {
#pragma unroll
            for (int k = 0; k < 2; ++k)
                *reinterpret_cast<uint32_t*>(blob + place<IMAGE>(o * (D / 16) + j, lane + k)) =
                    q[4 * k] | q[4 * k + 1] << 8 | q[4 * k + 2] << 16 | q[4 * k + 3] << 24;
        }
    } else {
        const int t = (r & 7) >> 1, e = r & 1, n = c >> 3;
        if constexpr (Q4) {
            // channels d (n even) and d + 8 share a byte: the two lanes exchange, each writes four
            uint32_t w = 0u;
#pragma unroll
            for (int i = 0; i < 8; ++i) w |= q[i] << (4 * i);
            const uint32_t other = __shfl_xor_sync(0xffffffffu, w, 1);
            const uint32_t lo = (n & 1) ? other >> 16 : w, hi = (n & 1) ? w >> 16 : other;
            uint8_t* const at = blob + place<IMAGE>(n >> 1, 4 * (4 * (n & 1)) + t) + 2 * e + o;
            if (there)
#pragma unroll
                for (int i = 0; i < 4; ++i) at[64 * i] = static_cast<uint8_t>(((lo >> (4 * i)) & 15u) | (((hi >> (4 * i)) & 15u) << 4));
        } else if (there) {
            uint8_t* const at = blob + place<IMAGE>(n, t) + 2 * o + e;
#pragma unroll
            for (int i = 0; i < 8; ++i) at[place<IMAGE>(0, 4 * i)] = static_cast<uint8_t>(q[i]);
        }
    }
}

// The values of four channels of the token at place r of a blob.
template <bool IMAGE, bool Q4, bool V, int D>
__device__ __forceinline__ float4 get4(const uint8_t* blob, int r, int c) {
    constexpr int NB = D / 32;
    const float d = __half2float(reinterpret_cast<const __half*>(blob + scales_at<IMAGE>(Q4, D))[r * NB + (c >> 5)]);
    const int o = r >> 3;
    uint32_t q[4];
    if constexpr (!V) {
        const int lane = 4 * (r & 7) + ((c & 15) >> 2), j = c >> 4;
        const uint32_t w = *reinterpret_cast<const uint32_t*>(blob + place<IMAGE>(Q4 ? o * NB + (j >> 1) : o * (D / 16) + j, lane)) >>
                           (Q4 ? 8 * (j & 1) : 0);
#pragma unroll
        for (int i = 0; i < 4; ++i) q[i] = Q4 ? (w >> (4 * (4 * (i & 1) + (i >> 1)))) & 15u : (w >> (8 * i)) & 255u;
    } else {
        const int t = (r & 7) >> 1, e = r & 1, n = c >> 3;
        const uint8_t* const at = blob + place<IMAGE>(Q4 ? n >> 1 : n, 4 * (c & 4) + t) + (Q4 ? 2 * e + o : 2 * o + e);
#pragma unroll
        for (int i = 0; i < 4; ++i) q[i] = Q4 ? (at[64 * i] >> (4 * (n & 1))) & 15u : at[64 * i];
    }
    float x[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) x[i] = d * static_cast<float>(static_cast<int>(q[i]) - (Q4 ? 8 : 128));
    return make_float4(x[0], x[1], x[2], x[3]);
}

struct Window {
    int64_t slot[3 * kKvRows];  // of rows row0 - 15 .. row0 + 32
    int start;                  // first row (from row0) of the group that begins in the window, or -1
    int singles, zeros;         // rows that go one by one; rows without a place
    int single[kKvRows], zero[kKvRows];
};

// Table entries of the positions of rows row0 .. row0 + 31 (keys that are turned on the way).
struct WindowTurns {
    const float2* entry[2 * kKvRows];
};

// Blob of a slot: division by the groups of a page as a multiplication that is at most one too large.
__device__ __forceinline__ int64_t blob_of(const KvParams& p, int64_t slot, int h) {
    const int g = static_cast<int>(slot >> 4), gpp = p.page >> 4;
    int pg = g, place = 0;
    if (gpp > 1) {
        pg = static_cast<int>(__umulhi(static_cast<uint32_t>(g), p.page_magic));
        place = g - pg * gpp;
        if (place < 0) --pg, place += gpp;
    }
    return (static_cast<int64_t>(pg) * p.H + h) * gpp + place;
}

// turns: null, or of keys that are turned before they are quantized
template <bool STORE, bool Q4, bool V, int D, bool TURN = false, typename T>
__device__ __forceinline__ void kv_rows(const KvParams& p, const Rotary* turn, const WindowTurns* turns, const Window& w,
                                        int64_t row0, T* rows, int64_t head, int64_t st, uint8_t* pool, int h0, int h1, uint8_t* image, float* tile = nullptr) {
    // threads a row (eight channels each; four to read back) and rows at once
    constexpr int kChannels = STORE ? 8 : 4, kPer = D / kChannels, kAtOnce = kKvThreads / kPer, kPasses = kKvRows / kAtOnce;
    constexpr int kBlob = kv_blob_bytes(Q4, D), kLines = kBlob / 16, kQuants = kv_quant_bytes(Q4, D) / 16;
    const int tid = threadIdx.x, r_at = tid / kPer, c = kChannels * (tid % kPer);
    const auto load8 = [&](const T* src, int row, float (&x)[8]) {  // row: from row0
        if constexpr (TURN) {
            turned8(*turn, src - c, c, turns->entry[row], x);
            return;
        }
        const float4 a = ld4(src), b = ld4(src + 4);
        x[0] = a.x, x[1] = a.y, x[2] = a.z, x[3] = a.w, x[4] = b.x, x[5] = b.y, x[6] = b.z, x[7] = b.w;
    };
    const auto line = [&](int i) {  // 16 bytes i of the blob in its image
        return reinterpret_cast<uint4*>(image + (i < kQuants ? place<true>(4 * (i >> 5), i & 31) : scales_at<true>(Q4, D) + 16 * (i - kQuants)));
    };
    constexpr int kUnits = D / 64;  // of eight channels that a thread turns: 16 rows of D / 8
    Turn4 mine4[kUnits];
    for (int h = h0; h < h1; ++h) {
        T* const mine = rows + h * head + c;
        if (w.start >= 0) {
            uint4* const blob = reinterpret_cast<uint4*>(pool + blob_of(p, w.slot[kKvRows - 1 + w.start], h) * kBlob);
            T* const first = mine + (row0 + w.start + r_at) * st;
            if constexpr (STORE) {
                float x[kPasses][8];
                bool done = false;
                if constexpr (TURN) {
                    if (turn->whole) {
                        // a thread turns the same places of every head, four pairs at a time, into a tile of the group's rows
                        if (h == h0)
#pragma unroll
                            for (int k = 0; k < kUnits; ++k) mine4[k] = turn4_of(*turn, (tid + k * kKvThreads) % (D / 8),
                                                                                 turns->entry[w.start + (tid + k * kKvThreads) / (D / 8)]);
                        float4 a[kUnits], b[kUnits];
#pragma unroll
                        for (int k = 0; k < kUnits; ++k) {
                            const T* const src = rows + h * head + (row0 + w.start + (tid + k * kKvThreads) / (D / 8)) * st;
                            a[k] = ld4(src + mine4[k].ca), b[k] = ld4(src + mine4[k].cb);
                        }
#pragma unroll
                        for (int k = 0; k < kUnits; ++k) {
                            turn4(mine4[k], turn->pairs, a[k], b[k]);
                            float* const to = tile + (tid + k * kKvThreads) / (D / 8) * (D + 4);
                            st4(to + mine4[k].ca, a[k]);
                            st4(to + mine4[k].cb, b[k]);
                        }
                        __syncthreads();
#pragma unroll
                        for (int k = 0; k < kPasses; ++k) {
                            const float* const from = tile + (r_at + k * kAtOnce) * (D + 4) + c;
                            const float4 lo = ld4(from), hi = ld4(from + 4);
                            x[k][0] = lo.x, x[k][1] = lo.y, x[k][2] = lo.z, x[k][3] = lo.w;
                            x[k][4] = hi.x, x[k][5] = hi.y, x[k][6] = hi.z, x[k][7] = hi.w;
                        }
                        done = true;
                    }
                }
                if (!done)
#pragma unroll
                for (int k = 0; k < kPasses; ++k) load8(first + k * kAtOnce * st, w.start + r_at + k * kAtOnce, x[k]);
                if (h > h0) __syncthreads();  // the blob before this one has left
#pragma unroll
                for (int k = 0; k < kPasses; ++k) {
                    uint32_t q[8];
                    const float d = quantize8<Q4>(x[k], q);
                    put8<true, Q4, V, D>(image, r_at + k * kAtOnce, c, q, d, true);
                }
                __syncthreads();
#pragma unroll
                for (int i = tid; i < kLines; i += kKvThreads) blob[i] = *line(i);
            } else {
                if (h > h0) __syncthreads();
#pragma unroll
                for (int i = tid; i < kLines; i += kKvThreads) *line(i) = blob[i];
                __syncthreads();
#pragma unroll
                for (int k = 0; k < kPasses; ++k) st4(first + k * kAtOnce * st, get4<true, Q4, V, D>(image, r_at + k * kAtOnce, c));
            }
        }
        for (int k0 = 0; k0 < w.singles; k0 += kAtOnce) {
            const bool there = k0 + r_at < w.singles;
            const int row = w.single[there ? k0 + r_at : 0];
            const int64_t slot = w.slot[kKvRows - 1 + row];
            uint8_t* const blob = pool + blob_of(p, slot, h) * kBlob;
            T* const at = mine + (row0 + row) * st;
            if constexpr (STORE) {
                float x[8];
                uint32_t q[8];
                load8(at, row, x);
                const float d = quantize8<Q4>(x, q);
                put8<false, Q4, V, D>(blob, static_cast<int>(slot & 15), c, q, d, there);
            } else if (there) {
                st4(at, get4<false, Q4, V, D>(blob, static_cast<int>(slot & 15), c));
            }
        }
        if constexpr (!STORE) {  // places outside the cache read as zeros
            for (int k = r_at; k < w.zeros; k += kAtOnce) st4(mine + (row0 + w.zero[k]) * st, make_float4(0.f, 0.f, 0.f, 0.f));
        }
    }
}

// The rows of a window: the slots around it, the group that begins in it, single rows and those without a place.
// False: no row.
__device__ __forceinline__ bool kv_window(const KvParams& p, Window& w, unsigned window, int64_t& row0) {
    const int tid = threadIdx.x;
    const int64_t s0 = p.slots[0];
    row0 = static_cast<int64_t>(window) * kKvRows - (s0 > 0 ? s0 & 15 : 0);
    if (row0 >= p.n) return false;
    if (tid < 3 * kKvRows) {
        const int64_t r = row0 - (kKvRows - 1) + tid;
        w.slot[tid] = r >= 0 && r < p.n ? p.slots[r] : -1;
    }
    __syncthreads();
    if (tid < 32) {
        // a group: 16 consecutive slots from a multiple of 16, inside the cache
        bool ok = tid < 2 * kKvRows - 1;
        if (ok) {
            const int64_t s = w.slot[tid];
            ok = s >= 0 && (s & 15) == 0 && s + 15 < p.n_slots;
            if (ok) {
#pragma unroll
                for (int i = 1; i < 16; ++i) ok &= w.slot[tid + i] == s + i;
            }
        }
        const uint32_t starts = __ballot_sync(0xffffffffu, ok);  // bit i: one starts at row row0 - 15 + i
        bool single = false, zero = false;
        const int64_t row = row0 + tid;
        if (tid < kKvRows && row >= 0 && row < p.n) {
            const int64_t s = w.slot[kKvRows - 1 + tid];
            if (s >= p.n_slots) set_error(p.err, DEV_ERR_BAD_PLACE);
            zero = s < 0 || s >= p.n_slots;
            // in a group: it started at one of the 16 rows up to this one
            single = !zero && !((starts >> tid) & 0xFFFFu);
        }
        const uint32_t singles = __ballot_sync(0xffffffffu, single), zeros = __ballot_sync(0xffffffffu, zero);
        const uint32_t below = (1u << tid) - 1u;
        if (single) w.single[__popc(singles & below)] = tid;
        if (zero) w.zero[__popc(zeros & below)] = tid;
        if (tid == 0) {
            const uint32_t mine = starts >> (kKvRows - 1);
            w.start = mine ? __ffs(mine) - 1 : -1;
            w.singles = __popc(singles);
            w.zeros = __popc(zeros);
        }
    }
    __syncthreads();
    return true;
}

// Grid: (windows of 16 rows, 2 * parts of the heads); the first half of the parts: keys.
template <bool STORE, int D, typename T>
__global__ void __launch_bounds__(kKvThreads) k_kv(const __grid_constant__ KvParams p) {
    pdl_launch_dependents();
    pdl_wait();
    __shared__ __align__(16) uint8_t image[D / 32 * 592 + D];
    __shared__ Window w;
    int64_t row0;
    if (!kv_window(p, w, blockIdx.x, row0)) return;
    const int parts = static_cast<int>(gridDim.y) >> 1;
    const bool is_v = static_cast<int>(blockIdx.y) >= parts;
    const int part = static_cast<int>(blockIdx.y) - (is_v ? parts : 0);
    const int h0 = part * p.heads_at_once, h1 = min(p.H, h0 + p.heads_at_once);
    T* const rows = static_cast<T*>(const_cast<void*>(is_v ? p.vs : p.ks));
    if (is_v) {
        if (p.v.q4) kv_rows<STORE, true, true, D>(p, nullptr, nullptr, w, row0, rows, p.v_head, p.v_token, p.v.p, h0, h1, image);
        else kv_rows<STORE, false, true, D>(p, nullptr, nullptr, w, row0, rows, p.v_head, p.v_token, p.v.p, h0, h1, image);
    } else {
        if (p.k.q4) kv_rows<STORE, true, false, D>(p, nullptr, nullptr, w, row0, rows, p.k_head, p.k_token, p.k.p, h0, h1, image);
        else kv_rows<STORE, false, false, D>(p, nullptr, nullptr, w, row0, rows, p.k_head, p.k_token, p.k.p, h0, h1, image);
    }
}

struct AppendParams {
    KvParams kv;
    RotateParams q;  // of the keys too: the rotation; no heads: no queries
    int kv_parts;    // of the keys' heads, and of the values'
    unsigned parts;  // of a window
};

// The same with the keys turned before they are quantized, and the queries turned in further parts.  Grid: windows, in
// each the parts of the keys' heads, of the values' and of the queries', so that the quantizers, which are bound by
// instructions, run beside the queries, which are bound by memory.
// (six CTAs an SM: 16384 tokens with their queries 77 us, with the four that 128 registers leave 93)
template <int D, int QV, typename T>
__global__ void __launch_bounds__(kKvThreads, D == 256 ? 4 : 6) k_kv_append(const __grid_constant__ AppendParams a) {
    pdl_launch_dependents();
    pdl_wait();
    __shared__ __align__(16) uint8_t image[D / 32 * 592 + D];
    __shared__ Window w;
    __shared__ WindowTurns turns;
    __shared__ __align__(16) float tile[kKvRows * (D + 4)];
    const KvParams& p = a.kv;
    const unsigned window = blockIdx.x / a.parts;
    const int part = static_cast<int>(blockIdx.x - window * a.parts);
    if (part >= 2 * a.kv_parts) {
        const int64_t r0 = static_cast<int64_t>(window) * kKvRows;
        const int h0 = (part - 2 * a.kv_parts) * a.q.heads_at_once;
        rotate_tile<QV, T>(a.q, r0, min(p.n, r0 + kKvRows), h0, min(a.q.H, h0 + a.q.heads_at_once));
        return;
    }
    int64_t row0;
    if (!kv_window(p, w, window, row0)) return;
    const bool is_v = part >= a.kv_parts;
    const int h0 = (part - (is_v ? a.kv_parts : 0)) * p.heads_at_once, h1 = min(p.H, h0 + p.heads_at_once);
    if (is_v) {
        T* const rows = static_cast<T*>(const_cast<void*>(p.vs));
        if (p.v.q4) kv_rows<true, true, true, D>(p, nullptr, nullptr, w, row0, rows, p.v_head, p.v_token, p.v.p, h0, h1, image);
        else kv_rows<true, false, true, D>(p, nullptr, nullptr, w, row0, rows, p.v_head, p.v_token, p.v.p, h0, h1, image);
        return;
    }
    if (threadIdx.x < 2 * kKvRows) {
        const int64_t row = row0 + threadIdx.x;
        const float2* entry = nullptr;
        if (row >= 0 && row < p.n) {
            entry = rotary_row(a.q.r, row);
            if (!entry && p.slots[row] >= 0) set_error(p.err, DEV_ERR_BAD_POSITION);
        }
        turns.entry[threadIdx.x] = entry;
    }
    __syncthreads();
    T* const rows = static_cast<T*>(const_cast<void*>(p.ks));
    if (p.k.q4) kv_rows<true, true, false, D, true>(p, &a.q.r, &turns, w, row0, rows, p.k_head, p.k_token, p.k.p, h0, h1, image, tile);
    else kv_rows<true, false, false, D, true>(p, &a.q.r, &turns, w, row0, rows, p.k_head, p.k_token, p.k.p, h0, h1, image, tile);
}

// the first window may begin up to 15 rows before the first row
int64_t kv_windows(const KvParams& p) { return (p.n + 2 * kKvRows - 2) / kKvRows; }

template <bool STORE, int D>
cudaError_t launch_kv_dim(KvParams p, int dtype, cudaStream_t s) {
    const int64_t windows = kv_windows(p);
    // One head a CTA while the CTAs are few, four once there are plenty (store and load
    // of 8 heads of 128 channels, us, one / four: 64 tokens 5.0 / 8.8, 1024 7.8 / 13.5,
    // 4096 18.6 / 19.5, 16384 70 / 60).
    p.heads_at_once = windows * 2 * p.H < 8192 ? 1 : 4;
    const int parts = (p.H + p.heads_at_once - 1) / p.heads_at_once;
    const dim3 grid(static_cast<unsigned>(windows), static_cast<unsigned>(2 * parts));
    if (dtype == 0) return launch_pdl(k_kv<STORE, D, float>, grid, dim3(kKvThreads), 0, s, p);
    if (dtype == 1) return launch_pdl(k_kv<STORE, D, __half>, grid, dim3(kKvThreads), 0, s, p);
    return launch_pdl(k_kv<STORE, D, __nv_bfloat16>, grid, dim3(kKvThreads), 0, s, p);
}

template <bool STORE>
cudaError_t launch_kv(const KvParams& p, int dtype, cudaStream_t s) {
    if (p.n == 0) return cudaSuccess;
    if (p.D == 64) return launch_kv_dim<STORE, 64>(p, dtype, s);
    if (p.D == 128) return launch_kv_dim<STORE, 128>(p, dtype, s);
    return launch_kv_dim<STORE, 256>(p, dtype, s);
}

template <int D, typename T>
cudaError_t launch_append_type(AppendParams a, int v, cudaStream_t s) {
    const int64_t windows = kv_windows(a.kv);
    a.kv.heads_at_once = windows * 2 * a.kv.H < 8192 ? 1 : 4;
    a.kv_parts = (a.kv.H + a.kv.heads_at_once - 1) / a.kv.heads_at_once;
    a.q.units = a.q.r.half / v + ((D - 2 * a.q.r.half) / v + 1) / 2;
    a.q.heads_at_once = std::max(1, std::min(a.q.H, windows < 64 ? 1 : 8));
    const int q_parts = (a.q.H + a.q.heads_at_once - 1) / a.q.heads_at_once;
    a.parts = static_cast<unsigned>(2 * a.kv_parts + q_parts);
    if (windows * a.parts > INT32_MAX) return cudaErrorInvalidConfiguration;
    const dim3 grid(static_cast<unsigned>(windows * a.parts));
    if (v == 8) {
        if constexpr (sizeof(T) == 2) return launch_pdl(k_kv_append<D, 8, T>, grid, dim3(kKvThreads), 0, s, a);
    }
    if (v == 4) return launch_pdl(k_kv_append<D, 4, T>, grid, dim3(kKvThreads), 0, s, a);
    return launch_pdl(k_kv_append<D, 1, T>, grid, dim3(kKvThreads), 0, s, a);
}

template <int D>
cudaError_t launch_append_dim(const AppendParams& a, int dtype, int v, cudaStream_t s) {
    if (dtype == 0) return launch_append_type<D, float>(a, v, s);
    if (dtype == 1) return launch_append_type<D, __half>(a, v, s);
    return launch_append_type<D, __nv_bfloat16>(a, v, s);
}

}  // namespace

cudaError_t launch_kv_store(const KvParams& p, int dtype, cudaStream_t s) { return launch_kv<true>(p, dtype, s); }
cudaError_t launch_kv_load(const KvParams& p, int dtype, cudaStream_t s) { return launch_kv<false>(p, dtype, s); }

cudaError_t launch_kv_append(const KvParams& kv, const RotateParams& q, int dtype, cudaStream_t s) {
    if (kv.n == 0) return cudaSuccess;
    AppendParams a{kv, q, 0, 0};
    const int both = q.r.half | q.r.first;
    a.q.r.whole = !aligned_to(q.r.table, 16) ? 0 : both % 8 == 0 ? 8 : both % 4 == 0 ? 4 : 0;
    const int v = q.H ? rotate_vector(q, dtype) : dtype == 0 ? 4 : 8;
    if (kv.D == 64) return launch_append_dim<64>(a, dtype, v, s);
    if (kv.D == 128) return launch_append_dim<128>(a, dtype, v, s);
    return launch_append_dim<256>(a, dtype, v, s);
}

}  // namespace ggq
