// ggq_adapt.cu -- low-rank adapters of many requests beside a shared projection.
//
// Mathematics: out[t] = y[t] + s_a B_a (A_a x[t]) with the adapter a of row t's sequence.  What has to move
// is x, y and out once and the banks of the adapters in use, 2 rank (K + N) bytes each; products are few.
//
// One launch: a cluster of CTAs takes a group of rows of one adapter.  Its CTAs share the inputs: each multiplies
// its part of K, the partial A x (rows x rank, fp32) meet through distributed shared memory, summed in the order
// of the CTAs, and each CTA then takes its part of the N outputs.  So one row's banks are read by up to 16 SMs,
// with no scratch and no second launch.  Groups are 64 rows of a sequence (prompts) or 16: of a sequence, or of
// single tokens, where a cluster stands for a row and works if its row is the first, 17th, ... of its adapter, so
// that a bank is read once for 16 rows whatever the order of the ids is.
//
// Inside a CTA, blocks of x and bank (then of y and bank) come through a ring of shared memory by asynchronous
// copies; memory is the bound, so what counts is bytes in flight: 50 to 100 KB an SM.  Eight warps are 4 tiles of
// 16 rows times 2 parts of a block of 64 channels (outputs), or 1 times 8 parts of 256 (four: 128).  The order of the summed
// index is free as long as both operands of the matrix instruction share it, so a lane takes eight neighbouring
// values as its elements of four k = 8 steps; the order of the outputs is free too: a lane's columns of four
// 8-column tiles are eight neighbouring outputs, so y moves in whole vectors.
//
// 16-bit rows with banks of the same type: their own m16n8k16 instruction, operands exact.  Others: m16n8k8 of
// tf32, in which either 16-bit type is exact and an fp32 value is two terms of 11 bits (off by 2^-22).  A x as an
// operand of the second product is two terms, of 11 bits, or of 8 for bf16 rows and banks (off by 2^-17, a
// hundredth of the output's rounding).
#include <algorithm>

#include "ggq_adapt.cuh"
#include "ggq_cluster.cuh"
#include "ggq_device.cuh"
#include "ggq_internal.h"
#include "ggq_kv.cuh"

namespace ggq {

namespace {

constexpr uint32_t kFull = 0xffffffffu;
constexpr int kMaxWarps = 8;

// ---------------------------------------------------------------- groups

template <int ROWS>
struct Group {
    int64_t row[ROWS];
    int64_t first;
    int count[kMaxWarps];
    int rows, adapter;
};

// The block's exclusive sum of `v` over its threads, and the total.  count: an int a warp, in shared memory.
template <int WARPS>
__device__ __forceinline__ int block_scan(int v, int* count, int& total) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    int sum = v;
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
        const int o = __shfl_up_sync(kFull, sum, d);
        if (lane >= d) sum += o;
    }
    __syncthreads();
    if (lane == 31) count[warp] = sum;
    __syncthreads();
    int before = 0;
    total = 0;
#pragma unroll
    for (int w = 0; w < WARPS; ++w) {
        const int c = count[w];
        if (w < warp) before += c;
        total += c;
    }
    return before + sum - v;
}

// An adapter id that counts: -1 for none, one outside the adapters or of rank 0.
__device__ __forceinline__ int adapter_of(const AdaptParams& p, int64_t seq) {
    const int a = p.ids[seq];
    if (a >= p.n) set_error(p.err, DEV_ERR_BAD_ADAPTER);
    return a < 0 || a >= p.n || (p.ranks && p.ranks[a] <= 0) ? -1 : a;
}

// Finds the rows of cluster `c`: sh.rows of them (0: none) of adapter sh.adapter (-1: rows that stay as they are).
template <int WARPS, int ROWS>
__device__ __forceinline__ void find_group(const AdaptParams& p, Group<ROWS>& sh, int64_t c) {
    constexpr int kThreads = 32 * WARPS;
    const int tid = threadIdx.x;
    if (tid == 0) sh.rows = 0;
    if (!p.q_start) {
        const int id = p.ids[c];
        if (tid == 0) sh.adapter = adapter_of(p, c);
        __syncthreads();
        if (sh.adapter < 0) {
            if (tid == 0) sh.rows = 1, sh.row[0] = c;
            __syncthreads();
            return;
        }
        // rows of the adapter before this one, then this one and the next ones
        int64_t seen = 0;
        int first = -1;  // this row's place among them
        for (int64_t j0 = 0; j0 < p.seqs; j0 += kThreads) {
            const int64_t j = j0 + tid;
            const bool mine = j < p.seqs && p.ids[j] == id;
            int total;
            const int at = static_cast<int>(seen) + block_scan<WARPS>(mine, sh.count, total);
            if (first < 0 && c < j0 + kThreads) {
                if (j == c) sh.rows = at;
                __syncthreads();
                first = sh.rows;
                __syncthreads();
                if (first % ROWS) {  // another cluster has it
                    if (tid == 0) sh.rows = 0;
                    __syncthreads();
                    return;
                }
            }
            if (first >= 0 && mine && at >= first && at < first + ROWS) sh.row[at - first] = j;
            seen += total;
            if (first >= 0 && seen >= first + ROWS) break;
        }
        if (tid == 0) sh.rows = min(ROWS, static_cast<int>(seen) - first);
        __syncthreads();
        return;
    }
    // the c-th group, counted through the sequences
    int64_t seen = 0;
    __syncthreads();
    for (int64_t j0 = 0; j0 < p.seqs && seen <= c; j0 += kThreads) {
        const int64_t j = j0 + tid;
        int64_t r0 = 0, len = 0;
        if (j < p.seqs) {
            r0 = p.q_start[j];
            const int64_t end = p.q_start[j + 1];
            if (r0 < 0 || end < r0 || end > p.T) {
                set_error(p.err, DEV_ERR_BAD_ADAPTER);
                r0 = max(static_cast<int64_t>(0), min(r0, p.T));
            }
            len = max(static_cast<int64_t>(0), min(end, p.T) - r0);
        }
        const int groups = static_cast<int>((len + ROWS - 1) / ROWS);
        int total;
        const int64_t at = seen + block_scan<WARPS>(groups, sh.count, total);
        if (c >= at && c < at + groups) {
            sh.first = r0 + (c - at) * ROWS;
            sh.rows = static_cast<int>(min(static_cast<int64_t>(ROWS), r0 + len - sh.first));
            sh.adapter = adapter_of(p, j);
        }
        seen += total;
    }
    __syncthreads();
    if (tid < sh.rows) sh.row[tid] = sh.first + tid;
    __syncthreads();
}

// ---------------------------------------------------------------- copies, matrix instructions, terms

// `bytes` (0 .. 16 or 8) of src, the rest zeros
__device__ __forceinline__ void copy16(uint32_t dst, const void* src, int bytes) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(bytes) : "memory");
}
__device__ __forceinline__ void copy8(uint32_t dst, const void* src, int bytes) {
    asm volatile("cp.async.ca.shared.global [%0], [%1], 8, %2;" ::"r"(dst), "l"(src), "r"(bytes) : "memory");
}
__device__ __forceinline__ void copies_end() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void copies_wait() {
    asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}

template <bool BF16>
__device__ __forceinline__ void mma_k16(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
    if constexpr (BF16)
        asm("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
            : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
            : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
    else
        asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
            : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
            : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
__device__ __forceinline__ void mma_tf32(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
    asm("mma.sync.aligned.m16n8k8.row.col.f32.tf32.tf32.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

// x as two tf32 terms; infinities and NaN stay in the first
__device__ __forceinline__ void split_tf32(float x, uint32_t& hi, uint32_t& lo) {
    const bool fine = fabsf(x) < INFINITY;
    hi = fine ? __float_as_uint(x) & 0xffffe000u : __float_as_uint(x + x) & 0xffffe000u;
    lo = fine ? __float_as_uint(__fsub_rn(x, __uint_as_float(hi))) & 0xffffe000u : 0u;
}
// a pair as two bf16 terms
__device__ __forceinline__ void split_bf16(float a, float b, uint32_t& hi, uint32_t& lo) {
    const __nv_bfloat162 h = __floats2bfloat162_rn(a, b);
    const float ra = fabsf(a) < INFINITY ? a - __bfloat162float(h.x) : 0.0f, rb = fabsf(b) < INFINITY ? b - __bfloat162float(h.y) : 0.0f;
    const __nv_bfloat162 l = __floats2bfloat162_rn(ra, rb);
    hi = *reinterpret_cast<const uint32_t*>(&h);
    lo = *reinterpret_cast<const uint32_t*>(&l);
}

// A word of two 16-bit values (f16, or bf16) as tf32.
template <bool F16>
__device__ __forceinline__ void pair_tf32(uint32_t w, uint32_t& a, uint32_t& b) {
    if constexpr (F16) {
        const float2 v = __half22float2(*reinterpret_cast<const __half2*>(&w));
        a = __float_as_uint(v.x), b = __float_as_uint(v.y);
    } else {
        a = w << 16, b = w & 0xFFFF0000u;
    }
}
// Eight values of a bank row (1 f16, 2 bf16).
__device__ __forceinline__ void bank_tf32(uint4 u, int bank, uint32_t (&f)[8]) {
    const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        if (bank == 1) pair_tf32<true>(w[i], f[2 * i], f[2 * i + 1]);
        else pair_tf32<false>(w[i], f[2 * i], f[2 * i + 1]);
    }
}

// Eight values of a bank row of which the first `have` count: what stands behind a rank is no part of it.
__device__ __forceinline__ uint4 first_of(uint4 u, int have) {
    if (have >= 8) return u;
    uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) w[i] = 2 * i + 1 < have ? w[i] : 2 * i < have ? w[i] & 0xFFFFu : 0u;
    return make_uint4(w[0], w[1], w[2], w[3]);
}

// ---------------------------------------------------------------- shared memory

// Pitches (bytes) at which eight lanes of two neighbouring rows meet different banks.
template <typename T>
__host__ __device__ constexpr int row_pitch(int block) { return block * static_cast<int>(sizeof(T)) + (sizeof(T) == 4 ? 16 : 64); }
__host__ __device__ constexpr int bank_pitch(int bytes) { return (bytes + 63) / 128 * 128 + 64; }
__host__ __device__ constexpr int up32(int r) { return (r + 31) / 32 * 32; }

// Of WARPS warps, 16 MT rows and banks of R ranks:
//   sums [rows][up32(R) + 4]: this CTA's A x, which the others read;
//   t    [rows / 16][up32(R) / 8][32 lanes][4]: the whole A x in the order of the matrix instruction's operand;
//   part: sums of half of the parts of a block; ring: the blocks' copies, of the first product over part too.
template <typename T, int WARPS, int MT>
struct Plan {
    int sums, t, part, stage1, stage2;
    static constexpr int kParts = WARPS / MT, kBlock = 32 * kParts, kRows = 16 * MT;
    __host__ __device__ constexpr explicit Plan(int R) : sums(0), t(0), part(0), stage1(0), stage2(0) {
        sums = kRows * (up32(R) + 4) * 4;
        t = kRows * up32(R) * 4;
        part = kParts / 2 * sums;
        stage1 = kRows * row_pitch<T>(kBlock) + R * bank_pitch(2 * kBlock);
        stage2 = kRows * row_pitch<T>(kBlock) + kBlock * bank_pitch(2 * R);
    }
    __host__ __device__ constexpr int bytes(int stages) const {
        const int one = stages * stage1, two = part + stages * stage2;
        return sums + t + (one > two ? one : two);
    }
};

// ---------------------------------------------------------------- kernel

// NATIVE: rows and banks of one 16-bit type.  NT: 8-column tiles of the rank.  MT: tiles of 16 rows.
template <typename T, bool NATIVE, int NT, int WARPS, int MT>
__global__ void __launch_bounds__(32 * WARPS, NT > 8 ? 1 : 2) k_adapt(const __grid_constant__ AdaptParams p) {
    constexpr bool PAIRS = NATIVE && __is_same(T, __nv_bfloat16);
    using P = Plan<T, WARPS, MT>;
    constexpr int kStages = MT == 1 ? 2 : 3, kThreads = 32 * WARPS, kParts = P::kParts, kHalf = kParts / 2;
    constexpr int kBlock = P::kBlock, kRows = P::kRows, kPitch = row_pitch<T>(kBlock), kBankPitch = bank_pitch(2 * kBlock);
    pdl_launch_dependents();
    pdl_wait();
    extern __shared__ __align__(128) uint8_t smem[];
    __shared__ Group<kRows> sh;
    const int parts = static_cast<int>(cluster_size()), part = static_cast<int>(cluster_rank());
    find_group<WARPS>(p, sh, blockIdx.x / parts);
    const int rows = sh.rows, tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, g = lane >> 2, tq = lane & 3;
    if (rows == 0) return;  // of all the cluster's CTAs
    const T* const y = static_cast<const T*>(p.y);
    T* const out = static_cast<T*>(p.out);
    const int64_t n_step = ((p.N + 31) / 32 + parts - 1) / parts * 32, n0 = min(p.N, part * n_step), n1 = min(p.N, n0 + n_step);
    if (sh.adapter < 0) {
        if (p.out == p.y) return;
        for (int r = warp; r < rows; r += WARPS)
            for (int64_t n = n0 + lane; n < n1; n += 32) out[sh.row[r] * p.out_token + n] = y[sh.row[r] * p.y_token + n];
        return;
    }
    const int rank = p.ranks ? min(p.R, p.ranks[sh.adapter]) : p.R;
    const float scale = p.scales ? p.scales[sh.adapter] : 1.0f;
    const int k_step = ((p.K + 31) / 32 + parts - 1) / parts * 32, k0 = min(p.K, part * k_step), k1 = min(p.K, k0 + k_step);
    const uint16_t* const bank_a = static_cast<const uint16_t*>(p.a) + static_cast<int64_t>(sh.adapter) * p.R * p.K;
    const uint16_t* const bank_b = static_cast<const uint16_t*>(p.b) + static_cast<int64_t>(sh.adapter) * p.N * p.R;
    const P plan(p.R);
    const int wide = up32(p.R), pitch = wide + 4;  // floats of a row of the sums
    float* const sums = reinterpret_cast<float*>(smem);
    float* const t_frag = reinterpret_cast<float*>(smem + plan.sums);
    uint8_t* const ring1 = smem + plan.sums + plan.t;
    float* const parts_sums = reinterpret_cast<float*>(ring1);
    uint8_t* const ring2 = ring1 + plan.part;
    const int b_pitch = bank_pitch(2 * p.R);

    // rows' values [c0, c1) of a block that starts at column c: copies of 16 bytes, or of four 16-bit values
    const auto copy_rows = [&](const void* base, int64_t stride, bool wide16, int64_t c, int64_t c1, uint32_t to) {
        constexpr int kLog = kBlock == 64 ? 6 : kBlock == 128 ? 7 : 8;
        const int log_per = wide16 && sizeof(T) == 2 ? 3 : 2, per = 1 << log_per, log_chunks = kLog - log_per;
        for (int i = tid; i < kRows << log_chunks; i += kThreads) {
            const int r = i >> log_chunks, e = (i & ((1 << log_chunks) - 1)) << log_per;
            const int have = r < rows ? static_cast<int>(max(static_cast<int64_t>(0), min(static_cast<int64_t>(per), c1 - c - e))) : 0;
            const T* const src = have ? static_cast<const T*>(base) + sh.row[r] * stride + c + e : static_cast<const T*>(base);
            const uint32_t dst = to + r * kPitch + e * static_cast<int>(sizeof(T));
            if (per * sizeof(T) == 16) copy16(dst, src, have * static_cast<int>(sizeof(T)));
            else copy8(dst, src, have * static_cast<int>(sizeof(T)));
        }
    };
    const int blocks1 = (k1 - k0 + kBlock - 1) / kBlock, blocks2 = static_cast<int>((n1 - n0 + kBlock - 1) / kBlock);
    const auto load1 = [&](int b) {
        if (b < blocks1) {
            const uint32_t to = smem_addr(ring1 + (b % kStages) * plan.stage1), bank = to + kRows * kPitch;
            const int c = k0 + b * kBlock;
            copy_rows(p.x, p.x_token, p.x_whole, c, k1, to);
            constexpr int kChunks = kBlock / 8;
            for (int i = tid; i < (rank + 7) / 8 * 8 * kChunks; i += kThreads) {
                const int r = i / kChunks, k = c + i % kChunks * 8;
                const bool there = r < rank && k < k1;
                copy16(bank + r * kBankPitch + i % kChunks * 16, there ? bank_a + static_cast<int64_t>(r) * p.K + k : bank_a, there ? 16 : 0);
            }
        }
        copies_end();
    };
    const auto load2 = [&](int b) {
        if (b < blocks2) {
            const uint32_t to = smem_addr(ring2 + (b % kStages) * plan.stage2), bank = to + kRows * kPitch;
            const int64_t c = n0 + static_cast<int64_t>(b) * kBlock;
            if (p.y_whole) copy_rows(p.y, p.y_token, p.y_whole == 2, c, n1, to);
            const int chunks = (rank + 7) / 8, log_chunks = 32 - __clz(chunks - 1);  // (of a power of two)
            for (int i = tid; i < kBlock << log_chunks; i += kThreads) {
                const int r = i >> log_chunks, o = i & ((1 << log_chunks) - 1);
                if (o >= chunks) continue;
                const bool there = c + r < n1;
                copy16(bank + r * b_pitch + 16 * o, there ? bank_b + (c + r) * p.R + 8 * o : bank_b, there ? 16 : 0);
            }
        }
        copies_end();
    };

    const int m = warp % MT, sub = warp / MT, r_lo = 16 * m + g, r_hi = r_lo + 8;  // this warp's rows and part of a block
    const bool busy = 16 * m < rows;

    // A x of this CTA's inputs
    float acc[NT][4] = {};
    const int nt = (rank + 7) / 8;
#pragma unroll
    for (int b = 0; b < kStages - 1; ++b) load1(b);
    for (int b = 0; b < blocks1; ++b) {
        copies_wait<kStages - 2>();
        __syncthreads();
        load1(b + kStages - 1);
        if (!busy) continue;
        const uint8_t* const stage = ring1 + (b % kStages) * plan.stage1;
        const uint8_t* const bank = stage + kRows * kPitch + g * kBankPitch + 64 * sub + 16 * tq;
        const T* const x_lo = reinterpret_cast<const T*>(stage + r_lo * kPitch) + 32 * sub + 8 * tq;
        const T* const x_hi = reinterpret_cast<const T*>(stage + r_hi * kPitch) + 32 * sub + 8 * tq;
        if constexpr (NATIVE) {
            const uint4 lo = *reinterpret_cast<const uint4*>(x_lo), hi = *reinterpret_cast<const uint4*>(x_hi);
            const uint32_t f[2][4] = {{lo.x, hi.x, lo.y, hi.y}, {lo.z, hi.z, lo.w, hi.w}};
#pragma unroll
            for (int j = 0; j < NT; ++j) {
                if (j >= nt) break;
                const uint4 u = *reinterpret_cast<const uint4*>(bank + 8 * j * kBankPitch);
                mma_k16<PAIRS>(acc[j], f[0], u.x, u.y);
                mma_k16<PAIRS>(acc[j], f[1], u.z, u.w);
            }
        } else {
            constexpr int kTerms = sizeof(T) == 4 ? 2 : 1;
            uint32_t f[kTerms][4][4];  // [term][step][register]
#pragma unroll
            for (int r = 0; r < 2; ++r) {
                if constexpr (sizeof(T) == 4) {
                    float v[8];
                    const float4 a = ld4(r ? x_hi : x_lo), c = ld4((r ? x_hi : x_lo) + 4);
                    v[0] = a.x, v[1] = a.y, v[2] = a.z, v[3] = a.w, v[4] = c.x, v[5] = c.y, v[6] = c.z, v[7] = c.w;
#pragma unroll
                    for (int e = 0; e < 8; ++e) split_tf32(v[e], f[0][e >> 1][r + 2 * (e & 1)], f[1][e >> 1][r + 2 * (e & 1)]);
                } else {
                    const uint4 u = *reinterpret_cast<const uint4*>(r ? x_hi : x_lo);
                    const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
                    for (int q = 0; q < 4; ++q) pair_tf32<__is_same(T, __half)>(w[q], f[0][q][r], f[0][q][r + 2]);
                }
            }
#pragma unroll
            for (int j = 0; j < NT; ++j) {
                if (j >= nt) break;
                uint32_t u[8];
                bank_tf32(*reinterpret_cast<const uint4*>(bank + 8 * j * kBankPitch), p.bank, u);
#pragma unroll
                for (int term = 0; term < kTerms; ++term)
#pragma unroll
                    for (int q = 0; q < 4; ++q) mma_tf32(acc[j], f[term][q], u[2 * q], u[2 * q + 1]);
            }
        }
    }
    copies_wait<0>();
    __syncthreads();
    // the second product's first blocks come while the sums are joined
#pragma unroll
    for (int b = 0; b < kStages - 1; ++b) load2(b);
    {
        const auto put = [&](float* to, bool add) {
#pragma unroll
            for (int j = 0; j < NT; ++j) {
                if (j >= nt) break;
                float2* const lo = reinterpret_cast<float2*>(to + r_lo * pitch + 8 * j + 2 * tq);
                float2* const hi = reinterpret_cast<float2*>(to + r_hi * pitch + 8 * j + 2 * tq);
                if (add) {
                    const float2 a = *lo, b = *hi;
                    *lo = make_float2(a.x + acc[j][0], a.y + acc[j][1]), *hi = make_float2(b.x + acc[j][2], b.y + acc[j][3]);
                } else {
                    *lo = make_float2(acc[j][0], acc[j][1]), *hi = make_float2(acc[j][2], acc[j][3]);
                }
            }
        };
        // the parts of a block: by halves, then half of them together
        float* const mine = parts_sums + sub % kHalf * kRows * pitch;
        if (sub >= kHalf) put(mine, false);
        __syncthreads();
        if (sub < kHalf) put(mine, true);
        __syncthreads();
        for (int i = tid; i < kRows * nt * 8; i += kThreads) {
            const int at = i / (nt * 8) * pitch + i % (nt * 8);
            float v = parts_sums[at];
#pragma unroll
            for (int h = 1; h < kHalf; ++h) v += parts_sums[at + h * kRows * pitch];
            sums[at] = v;
        }
    }
    cluster_arrive();
    cluster_wait();
    // the sums of all CTAs, scaled, as the second product's operand
    for (int i = tid; i < kRows * (wide / 8); i += kThreads) {
        const int r = i / (wide / 8), o = i - r * (wide / 8);  // eight ranks of a row
        float t[8] = {};
        if (8 * o < rank && r < rows) {
#pragma unroll 4
            for (int c = 0; c < parts; ++c) {
                const uint32_t at = cluster_addr(sums + r * pitch + 8 * o, c);
                float v[8];
#pragma unroll
                for (int q = 0; q < 2; ++q)
                    asm volatile("ld.shared::cluster.v4.f32 {%0,%1,%2,%3}, [%4];"
                                 : "=f"(v[4 * q]), "=f"(v[4 * q + 1]), "=f"(v[4 * q + 2]), "=f"(v[4 * q + 3])
                                 : "r"(at + 16 * q));
#pragma unroll
                for (int e = 0; e < 8; ++e) t[e] += v[e];
            }
        }
        // element e of the eight is lane 4 (r % 8) + o % 4's, register (r / 8) % 2 + 2 (e % 2) of step e / 2
        float* const to = t_frag + (((r >> 4) * (wide / 8) + (o >> 2) * 4) * 32 + (r & 7) * 4 + (o & 3)) * 4 + ((r >> 3) & 1);
#pragma unroll
        for (int e = 0; e < 8; ++e) to[(e >> 1) * 128 + 2 * (e & 1)] = 8 * o + e < rank ? t[e] * scale : 0.0f;
    }
    cluster_arrive();  // nobody leaves before its sums are read

    // out = y + (A x) B^T
    const float4* const t_mine = reinterpret_cast<const float4*>(t_frag) + m * (wide / 8) * 32 + lane;
    for (int b = 0; b < blocks2; ++b) {
        copies_wait<kStages - 2>();
        __syncthreads();
        load2(b + kStages - 1);
        if (!busy) continue;
        const uint8_t* const stage = ring2 + (b % kStages) * plan.stage2;
        const uint8_t* const bank = stage + kRows * kPitch + (32 * sub + 8 * (g >> 1) + (g & 1)) * b_pitch + 16 * tq;
        const int64_t n = n0 + static_cast<int64_t>(b) * kBlock + 32 * sub + 8 * tq;  // this lane's eight outputs
        float o[4][4] = {};
        for (int s0 = 0; 32 * s0 < rank; ++s0) {
            const int have = rank - 32 * s0 - 8 * tq;
            uint4 u[4];
#pragma unroll
            for (int j = 0; j < 4; ++j)
                u[j] = have > 0 ? first_of(*reinterpret_cast<const uint4*>(bank + 2 * j * b_pitch + 64 * s0), have) : make_uint4(0, 0, 0, 0);
            if constexpr (PAIRS) {
#pragma unroll
                for (int q = 0; q < 2; ++q) {
                    const float4 a = t_mine[(4 * s0 + 2 * q) * 32], c = t_mine[(4 * s0 + 2 * q + 1) * 32];
                    uint32_t f[2][4];
                    split_bf16(a.x, a.z, f[0][0], f[1][0]);
                    split_bf16(a.y, a.w, f[0][1], f[1][1]);
                    split_bf16(c.x, c.z, f[0][2], f[1][2]);
                    split_bf16(c.y, c.w, f[0][3], f[1][3]);
#pragma unroll
                    for (int term = 0; term < 2; ++term)
#pragma unroll
                        for (int j = 0; j < 4; ++j) mma_k16<true>(o[j], f[term], q ? u[j].z : u[j].x, q ? u[j].w : u[j].y);
                }
            } else {
                uint32_t w[4][8];
#pragma unroll
                for (int j = 0; j < 4; ++j) bank_tf32(u[j], p.bank, w[j]);
#pragma unroll
                for (int q = 0; q < 4; ++q) {
                    const float4 a = t_mine[(4 * s0 + q) * 32];
                    uint32_t f[2][4];
                    split_tf32(a.x, f[0][0], f[1][0]);
                    split_tf32(a.y, f[0][1], f[1][1]);
                    split_tf32(a.z, f[0][2], f[1][2]);
                    split_tf32(a.w, f[0][3], f[1][3]);
#pragma unroll
                    for (int term = 0; term < 2; ++term)
#pragma unroll
                        for (int j = 0; j < 4; ++j) mma_tf32(o[j], f[term], w[j][2 * q], w[j][2 * q + 1]);
                }
            }
        }
#pragma unroll
        for (int r = 0; r < 2; ++r) {
            const int at = r ? r_hi : r_lo;
            if (at >= rows || n >= n1) continue;
            T* const to = out + sh.row[at] * p.out_token + n;
            float v[8];
            if (p.y_whole) {
                const T* const from = reinterpret_cast<const T*>(stage + at * kPitch) + 32 * sub + 8 * tq;
                const float4 a = ld4(from), c = ld4(from + 4);
                v[0] = a.x, v[1] = a.y, v[2] = a.z, v[3] = a.w, v[4] = c.x, v[5] = c.y, v[6] = c.z, v[7] = c.w;
            } else {
                const T* const from = y + sh.row[at] * p.y_token + n;
#pragma unroll
                for (int e = 0; e < 8; ++e) v[e] = n + e < n1 ? ld1(from + e) : 0.0f;
            }
#pragma unroll
            for (int j = 0; j < 4; ++j)
#pragma unroll
                for (int e = 0; e < 2; ++e) v[2 * j + e] += o[j][2 * r + e];
            if (p.out_whole && n + 8 <= n1) {
                st4(to, make_float4(v[0], v[1], v[2], v[3]));
                st4(to + 4, make_float4(v[4], v[5], v[6], v[7]));
            } else {
#pragma unroll
                for (int e = 0; e < 8; ++e)
                    if (n + e < n1) st1(to + e, v[e]);
            }
        }
    }
    cluster_wait();
}

template <typename T, bool NATIVE, int NT, int WARPS, int MT>
cudaError_t launch(const AdaptParams& p, int64_t groups, int parts, cudaStream_t s) {
    using P = Plan<T, WARPS, MT>;
    constexpr int kStages = MT == 1 ? 2 : 3, kMost = P(8 * NT).bytes(kStages);
    static_assert(kMost + 768 <= kSmemLimit, "ring, operand and sums of the largest rank in a CTA's shared memory");
    static thread_local bool done[kMaxDevices] = {};
    const auto kernel = k_adapt<T, NATIVE, NT, WARPS, MT>;
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e == cudaSuccess && (dev >= kMaxDevices || !done[dev])) {
        e = cudaFuncSetAttribute(kernel, cudaFuncAttributeNonPortableClusterSizeAllowed, 1);
        if (e == cudaSuccess) e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, kMost);
        if (e == cudaSuccess && dev < kMaxDevices) done[dev] = true;
    }
    if (e != cudaSuccess) return e;
    return launch_cluster(kernel, dim3(static_cast<unsigned>(groups * parts)), dim3(32 * WARPS), P(p.R).bytes(kStages), parts, s, p);
}

template <typename T, bool NATIVE>
cudaError_t launch_type(const AdaptParams& p, cudaStream_t s) {
    const int64_t rows = p.q_start && p.T > 8 * p.seqs && p.R <= 128 ? 64 : 16;
    const int64_t groups = p.q_start ? p.T / rows + std::min(p.seqs, p.T) : p.seqs;
    if (rows == 64) {  // more than eight rows a sequence
        const int parts = groups <= 38 ? 8 : 4;
        if (p.R <= 64) return launch<T, NATIVE, 8, 8, 4>(p, groups, parts, s);
        return launch<T, NATIVE, 16, 8, 4>(p, groups, parts, s);
    }
    const int parts = groups <= 18 ? 16 : groups <= 304 ? 8 : 4;
    if (p.R <= 64) return launch<T, NATIVE, 8, 8, 1>(p, groups, parts, s);
    // (wide blocks of high ranks do not fit a CTA)
    if (p.R <= 128) return launch<T, NATIVE, 16, 4, 1>(p, groups, parts, s);
    return launch<T, NATIVE, 32, 4, 1>(p, groups, parts, s);
}

}  // namespace

cudaError_t launch_adapt(const AdaptParams& given, int dtype, cudaStream_t s) {
    AdaptParams p = given;
    if (p.T == 0 || p.seqs == 0 || p.N == 0) return cudaSuccess;
    // rows at multiples of four elements, and of 16 bytes
    const int size = dtype == 0 ? 4 : 2;
    const auto whole = [&](const void* at, int64_t stride, int64_t bytes) {
        return aligned_to(at, bytes) && (p.T < 2 || stride * size % bytes == 0);
    };
    p.x_whole = whole(p.x, p.x_token, 16);
    p.y_whole = whole(p.y, p.y_token, 16) ? 2 : whole(p.y, p.y_token, 4 * size) ? 1 : 0;
    p.out_whole = whole(p.out, p.out_token, 4 * size);
    if (dtype == 0) return launch_type<float, false>(p, s);
    if (dtype == 1) return p.bank == 1 ? launch_type<__half, true>(p, s) : launch_type<__half, false>(p, s);
    return p.bank == 2 ? launch_type<__nv_bfloat16, true>(p, s) : launch_type<__nv_bfloat16, false>(p, s);
}

}  // namespace ggq
