// ggq_adapt.cu -- low-rank adapters of many requests beside a shared projection.
//
// Mathematics: out[t] = y[t] + s_a B_a (A_a x[t]) with the adapter a of row t's sequence.  What has to move
// is x, y and out once and the banks of the adapters in use, 2 rank (K + N) bytes each; products are few.
//
// One launch: a cluster of CTAs takes a group of rows of one adapter.  Its CTAs share the inputs: each multiplies
// its part of K, the partial A x (rows x rank, fp32) meet through distributed shared memory, summed in the order
// of the CTAs, and each CTA then takes its part of the N outputs.  So one row's banks are read by up to 16 SMs,
// with no scratch and no second launch.  Groups are 32 rows of a sequence (long prompts) or 16: of a sequence, or of
// single tokens of one adapter, so that a bank is read once for 16 rows whatever the order of the ids is: each cluster
// counts through the ids and takes its group (64 rows of 24 adapters to 6144 outputs, bf16, rank 64: 11.9 us, where a
// cluster a row, of which those work whose row is the first, 17th, ... of its adapter, took 14.7).  So go more than 256 rows,
// each of whose clusters counts up to its own: the time grows with their square (24 adapters of rank 64, bf16: 18 us for
// 256 rows, 41 for 512, 73 for 1024, 0.47 ms for 4096).
//
// Inside a CTA, blocks of x and bank (then of y and bank) come through a ring of shared memory by asynchronous
// copies; memory is the bound, so what counts is bytes in flight: 50 to 100 KB an SM.  Four warps are 2 tiles of
// 16 rows times 2 parts of a block of 64 channels (outputs), or 1 times 4 parts of 128 (eight: 256).  The order of the summed
// index is free as long as both operands of the matrix instruction share it, so a lane takes eight neighbouring
// values as its elements of four k = 8 steps; the order of the outputs is free too: a lane's columns of four
// 8-column tiles are eight neighbouring outputs, so y moves in whole vectors.
//
// Operands of the matrix instruction (m16n8k16) are bf16 terms: an fp32 value is three of 8 bits each, an f16 value
// two, exactly, and products of terms that lie below the last bit of the whole are left out.  f16 rows with f16 banks
// enter as they are.  A x, fp32, is an operand of three terms for fp32 rows and of two for 16-bit ones (2.5e-6 of the
// result, where the rounding of fp16 outputs is 2.1e-4 and of bf16 ones 1.7e-3).  A value that rounds to an infinity as bf16 gives NaN.  (tf32 instructions, of which an fp32 value takes two, run at a third of the
// rate a product on this part.)
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
constexpr int kAdaptSorted = 256;  // single tokens of a call whose ids every cluster looks at

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

// An adapter id that counts: -1 for none or one outside the adapters.
__device__ __forceinline__ int adapter_of(const AdaptParams& p, int64_t seq) {
    const int a = p.ids[seq];
    if (a >= p.n) set_error(p.err, DEV_ERR_BAD_ADAPTER);
    return a < 0 || a >= p.n ? -1 : a;
}

// Finds the rows of cluster `c`: sh.rows of them (0: none) of adapter sh.adapter (-1: rows that stay as they are).
// scratch: kAdaptSorted words of shared memory.
template <int WARPS, int ROWS>
__device__ __forceinline__ void find_group(const AdaptParams& p, Group<ROWS>& sh, int* scratch, int64_t c) {
    constexpr int kThreads = 32 * WARPS;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    if (tid == 0) sh.rows = 0;
    if (!p.q_start && p.seqs <= kAdaptSorted) {
        // every row's place among its adapter's (-1: rows without one); every ROWS-th begins a group
        constexpr int kEach = kAdaptSorted / kThreads;  // rows a thread
        const int seqs = static_cast<int>(p.seqs);
        int id[kEach], place[kEach];
#pragma unroll
        for (int k = 0; k < kEach; ++k) {
            const int j = k * kThreads + tid;
            id[k] = -1, place[k] = 0;
            if (j < seqs) id[k] = adapter_of(p, j);
            scratch[j] = id[k];
        }
        if (tid == 0) sh.adapter = -2;
        __syncthreads();
        bool begins[kEach];
#pragma unroll
        for (int k = 0; k < kEach; ++k) {
            const int j = k * kThreads + tid;
            if (j < seqs)
                for (int i = 0; i < j; i += 4) {
                    const int4 a = *reinterpret_cast<const int4*>(scratch + i);
                    place[k] += (a.x == id[k]) + (i + 1 < j && a.y == id[k]) + (i + 2 < j && a.z == id[k]) + (i + 3 < j && a.w == id[k]);
                }
            begins[k] = j < seqs && place[k] % ROWS == 0;
            const unsigned there = __ballot_sync(kFull, begins[k]);
            if (lane == 0) sh.count[k * WARPS + warp] = __popc(there);
        }
        __syncthreads();
#pragma unroll
        for (int k = 0; k < kEach; ++k) {
            int at = __popc(__ballot_sync(kFull, begins[k]) & ((1u << lane) - 1));
#pragma unroll
            for (int w = 0; w < kEach * WARPS; ++w) at += w < k * WARPS + warp ? sh.count[w] : 0;
            if (begins[k] && at == c) sh.adapter = id[k], sh.first = place[k];
        }
        __syncthreads();
        int rows = 0;
        if (sh.adapter > -2) {
#pragma unroll
            for (int k = 0; k < kEach; ++k) {
                const int64_t at = place[k] - sh.first;
                const bool mine = k * kThreads + tid < seqs && id[k] == sh.adapter && at >= 0 && at < ROWS;
                if (mine) sh.row[at] = k * kThreads + tid;
                rows += __syncthreads_count(mine);
            }
        }
        if (tid == 0) sh.rows = rows;
        __syncthreads();
        return;
    }
    if (!p.q_start) {
        const int id = p.ids[c];
        int next = tid < p.seqs ? p.ids[tid] : -1;
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
            const bool mine = next == id;
            next = j + kThreads < p.seqs ? p.ids[j + kThreads] : -1;
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
// Waits until at most n groups of copies (0 .. 2) are under way.
__device__ __forceinline__ void copies_wait(int n) {
    if (n == 0) asm volatile("cp.async.wait_group 0;" ::: "memory");
    else if (n == 1) asm volatile("cp.async.wait_group 1;" ::: "memory");
    else asm volatile("cp.async.wait_group 2;" ::: "memory");
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
// A pair of values as N pairs of bf16 terms.  What is not finite gives NaN.
template <int N>
__device__ __forceinline__ void split(float a, float b, uint32_t (&t)[N]) {
#pragma unroll
    for (int i = 0; i < N; ++i) {
        const __nv_bfloat162 h = __floats2bfloat162_rn(a, b);
        t[i] = *reinterpret_cast<const uint32_t*>(&h);
        a = __fsub_rn(a, __uint_as_float(t[i] << 16)), b = __fsub_rn(b, __uint_as_float(t[i] & 0xFFFF0000u));
    }
}
// Eight 16-bit values as N terms: bf16 ones as they are, f16 ones (F16) as two.
template <bool F16, int N>
__device__ __forceinline__ void terms_of(uint4 u, uint32_t (&f)[N][4]) {
    const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        if constexpr (F16 && N > 1) {
            const float2 v = __half22float2(*reinterpret_cast<const __half2*>(&w[i]));
            uint32_t t[N];
            split(v.x, v.y, t);
#pragma unroll
            for (int k = 0; k < N; ++k) f[k][i] = t[k];
        } else {
            f[0][i] = w[i];
        }
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
//   t    the whole A x as the matrix instruction's operand: [rows / 16][steps of 16][term][32 lanes][4 words],
//        and before it the sums of half of the parts of a block;
//   ring: the blocks' copies; those of the first product over t too.
template <typename T, int NT, int WARPS, int MT>
struct Plan {
    int sums, t, stage1, stage2, stages1, stages2, ctas;
    static constexpr int kTerms = sizeof(T) == 4 ? 3 : 2;  // of A x
    static constexpr int kParts = WARPS / MT, kBlock = 32 * kParts, kRows = 16 * MT;
    __host__ __device__ constexpr explicit Plan(int R, bool alone = false) : sums(0), t(0), stage1(0), stage2(0), stages1(0), stages2(0), ctas(1) {
        sums = kRows * (up32(R) + 4) * 4;
        t = kRows * up32(R) * 2 * kTerms;
        if (t < kParts / 2 * sums) t = kParts / 2 * sums;
        stage1 = kRows * row_pitch<T>(kBlock) + up32(R) * bank_pitch(2 * kBlock);
        stage2 = kRows * row_pitch<T>(kBlock) + kBlock * bank_pitch(2 * R);
        // two to four blocks at once, of as many CTAs an SM as have registers if they fit (unless they all run `alone`)
        ctas = alone ? 1 : WARPS == 8 ? 2 : NT > 8 ? 3 : 4;
        while (ctas > 1 && bytes(2, 2) > kSmemLimit / ctas - 2048) --ctas;
        const int room = kSmemLimit / ctas - 2048;
        for (stages1 = 2; stages1 < 4 && bytes(stages1 + 1, 2) <= room;) ++stages1;
        for (stages2 = 2; stages2 < 4 && bytes(2, stages2 + 1) <= room;) ++stages2;
    }
    __host__ __device__ constexpr int bytes(int s1, int s2) const {
        const int one = s1 * stage1, two = t + s2 * stage2;
        return sums + (one > two ? one : two);
    }
    __host__ __device__ constexpr int bytes() const { return bytes(stages1, stages2); }
};

// ---------------------------------------------------------------- kernel

// BF: banks of bf16, else f16.  NT: 8-column tiles of the rank.  MT: tiles of 16 rows.
template <typename T, bool BF, int NT, int WARPS, int MT>
__global__ void __launch_bounds__(32 * WARPS, NT > 16 ? 1 : WARPS == 8 ? 2 : NT > 8 ? 3 : 4) k_adapt(const __grid_constant__ AdaptParams p) {
    using P = Plan<T, NT, WARPS, MT>;
    // terms: of x and A's bank, of A x and B's bank
    constexpr bool F16 = __is_same(T, __half) && !BF;
    constexpr int kX = sizeof(T) == 4 ? 3 : __is_same(T, __half) && BF ? 2 : 1, kA = BF || F16 ? 1 : 2, kT = P::kTerms, kB = BF ? 1 : 2;
    constexpr int kThreads = 32 * WARPS, kParts = P::kParts, kHalf = kParts / 2;
    constexpr int kBlock = P::kBlock, kRows = P::kRows, kPitch = row_pitch<T>(kBlock), kBankPitch = bank_pitch(2 * kBlock);
    pdl_launch_dependents();
    pdl_wait();
    extern __shared__ __align__(128) uint8_t smem[];
    __shared__ Group<kRows> sh;
    const int parts = static_cast<int>(cluster_size()), part = static_cast<int>(cluster_rank());
    find_group<WARPS>(p, sh, reinterpret_cast<int*>(smem), blockIdx.x / parts);
    const int rows = sh.rows, tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, g = lane >> 2, tq = lane & 3;
    if (rows == 0) return;  // of all the cluster's CTAs
    const T* const y = static_cast<const T*>(p.y);
    T* const out = static_cast<T*>(p.out);
    const int64_t n_step = ((p.N + 31) / 32 + parts - 1) / parts * 32, n0 = min(p.N, part * n_step), n1 = min(p.N, n0 + n_step);
    const int rank = sh.adapter < 0 ? 0 : p.ranks ? min(p.R, p.ranks[sh.adapter]) : p.R;
    if (rank <= 0) {
        if (p.out == p.y) return;
        constexpr int kEach = 16 / sizeof(T);
        const bool wide = p.y_whole == 2 && p.out_whole == 2;
        const int count = static_cast<int>(n1 - n0), each = wide ? kEach : 1, chunks = (count + each - 1) / each;
        for (int64_t i = tid; i < static_cast<int64_t>(rows) * chunks; i += kThreads) {
            const int r = static_cast<int>(i / chunks), n = static_cast<int>(i - static_cast<int64_t>(r) * chunks) * each;
            const T* const from = y + sh.row[r] * p.y_token + n0 + n;
            T* const to = out + sh.row[r] * p.out_token + n0 + n;
            if (wide && n + each <= count) {
                *reinterpret_cast<uint4*>(to) = *reinterpret_cast<const uint4*>(from);
            } else {
                for (int e = 0; e < each && n + e < count; ++e) to[e] = from[e];
            }
        }
        return;
    }
    const float scale = p.scales ? p.scales[sh.adapter] : 1.0f;
    const int k_step = ((p.K + 31) / 32 + parts - 1) / parts * 32, k0 = min(p.K, part * k_step), k1 = min(p.K, k0 + k_step);
    const uint16_t* const bank_a = static_cast<const uint16_t*>(p.a) + static_cast<int64_t>(sh.adapter) * p.R * p.K;
    const uint16_t* const bank_b = static_cast<const uint16_t*>(p.b) + static_cast<int64_t>(sh.adapter) * p.N * p.R;
    const P plan(p.R);
    const int wide = up32(p.R), pitch = wide + 4;  // floats of a row of the sums
    float* const sums = reinterpret_cast<float*>(smem);
    uint32_t* const t_words = reinterpret_cast<uint32_t*>(smem + plan.sums);
    float* const parts_sums = reinterpret_cast<float*>(smem + plan.sums);
    uint8_t* const ring1 = smem + plan.sums;
    uint8_t* const ring2 = ring1 + plan.t;
    const int b_pitch = bank_pitch(2 * p.R), stages1 = p.stages1, stages2 = p.stages2;

    // A thread's share of the copies of a block of rows: the same places of every block.  16 bytes, or four 16-bit values.
    struct Share {
        const T* at[4];  // null: no row
        int column, per, step;
        uint32_t to;
    };
    const auto share_of = [&](const void* base, int64_t stride, bool wide16, int64_t c0) {
        constexpr int kLog = kBlock == 64 ? 6 : kBlock == 128 ? 7 : 8;
        const int log_per = wide16 && sizeof(T) == 2 ? 3 : 2, log_chunks = kLog - log_per, r0 = tid >> log_chunks;
        Share h;
        h.per = 1 << log_per, h.step = kThreads >> log_chunks, h.column = (tid & ((1 << log_chunks) - 1)) << log_per;
        h.to = r0 * kPitch + h.column * static_cast<int>(sizeof(T));
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const int r = r0 + i * h.step;
            h.at[i] = r < rows ? static_cast<const T*>(base) + sh.row[r] * stride + c0 + h.column : nullptr;
        }
        return h;
    };
    // Its copies of the block of columns b kBlock .. of `count` columns.  A copy of no bytes names an address all the same, which
    // has to be a multiple of 16 bytes as every other one: the bank's, since rows of x may start at 8.
    const auto copy_rows = [&](const Share& h, int b, int count, uint32_t to) {
        const int have = max(0, min(h.per, count - b * kBlock - h.column));
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            if (i * h.step >= kRows) break;
            if (!h.at[i]) continue;  // (what stands in the place of a row that is not there stays in that row)
            const void* const src = have ? static_cast<const void*>(h.at[i] + b * kBlock) : p.a;
            const uint32_t dst = to + h.to + i * h.step * kPitch;
            if (sizeof(T) == 4 || h.per == 8) copy16(dst, src, have * static_cast<int>(sizeof(T)));
            else copy8(dst, src, have * static_cast<int>(sizeof(T)));
        }
    };
    const int inputs = k1 - k0, outputs = static_cast<int>(n1 - n0);
    const int blocks1 = (inputs + kBlock - 1) / kBlock, blocks2 = (outputs + kBlock - 1) / kBlock;

    const int m = warp % MT, sub = warp / MT, r_lo = 16 * m + g, r_hi = r_lo + 8;  // this warp's rows and part of a block
    const bool busy = 16 * m < rows;

    // A x of this CTA's inputs
    float acc[NT][4] = {};
    const int nt = (rank + 7) / 8;
    {
        const Share h = share_of(p.x, p.x_token, p.x_whole, k0);
        constexpr int kChunks = kBlock / 8, kStep = kThreads / kChunks;
        const int row = tid / kChunks, column = tid % kChunks * 8;
        const uint16_t* const mine = bank_a + static_cast<int64_t>(row) * p.K + k0 + column;
        const auto load = [&](int b, int slot) {
            if (b < blocks1) {
                const uint32_t to = smem_addr(ring1 + slot * plan.stage1);
                copy_rows(h, b, inputs, to);
                const bool in = b * kBlock + column < inputs;
                const uint16_t* src = mine + b * kBlock;
                uint32_t dst = to + kRows * kPitch + row * kBankPitch + 2 * column;
                for (int r = row; r < rank; r += kStep, src += static_cast<int64_t>(kStep) * p.K, dst += kStep * kBankPitch)
                    copy16(dst, in ? src : bank_a, in ? 16 : 0);
            }
            copies_end();
        };
        for (int b = 0; b < stages1 - 1; ++b) load(b, b);
        for (int b = 0, slot = 0, next = stages1 - 1; b < blocks1; ++b) {
            copies_wait(stages1 - 2);
            __syncthreads();
            load(b + stages1 - 1, next);
            const uint8_t* const stage = ring1 + slot * plan.stage1;
            slot = slot + 1 == stages1 ? 0 : slot + 1, next = next + 1 == stages1 ? 0 : next + 1;
            if (!busy) continue;
            const uint8_t* const bank = stage + kRows * kPitch + g * kBankPitch + 64 * sub + 16 * tq;
            const T* const x_lo = reinterpret_cast<const T*>(stage + r_lo * kPitch) + 32 * sub + 8 * tq;
            const T* const x_hi = reinterpret_cast<const T*>(stage + r_hi * kPitch) + 32 * sub + 8 * tq;
            uint32_t f[kX][2][4];  // [term][step][register]
#pragma unroll
            for (int r = 0; r < 2; ++r) {
                uint32_t v[kX][4];
                if constexpr (sizeof(T) == 4) {
                    const float4 a = ld4(r ? x_hi : x_lo), c = ld4((r ? x_hi : x_lo) + 4);
                    const float e[8] = {a.x, a.y, a.z, a.w, c.x, c.y, c.z, c.w};
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        uint32_t t[kX];
                        split(e[2 * i], e[2 * i + 1], t);
#pragma unroll
                        for (int k = 0; k < kX; ++k) v[k][i] = t[k];
                    }
                } else {
                    terms_of<__is_same(T, __half) && !F16>(*reinterpret_cast<const uint4*>(r ? x_hi : x_lo), v);
                }
#pragma unroll
                for (int k = 0; k < kX; ++k)
#pragma unroll
                    for (int i = 0; i < 4; ++i) f[k][i >> 1][r + 2 * (i & 1)] = v[k][i];
            }
            // four tiles at once: four chains of dependent instructions (columns behind the rank are not looked at)
#pragma unroll
            for (int j0 = 0; j0 < NT; j0 += 4) {
                if (j0 >= nt) break;
                uint32_t u[4][kA][4];
#pragma unroll
                for (int j = 0; j < 4; ++j) terms_of<!BF && !F16>(*reinterpret_cast<const uint4*>(bank + 8 * (j0 + j) * kBankPitch), u[j]);
                // (of fp32 rows a block at a time: the instruction's own additions cut off what they do not hold, which
                // over 4096 inputs showed, 1.1e-6 of the result; 16-bit rows leave that to the instruction, since their output's
                // rounding is 200 times as much)
                constexpr bool ALONE = sizeof(T) == 4;
                float block[4][4] = {};
#pragma unroll
                for (int i = kX - 1; i >= 0; --i)
#pragma unroll
                    for (int k = kA - 1; k >= 0; --k) {
                        if (i + k >= (kX > kA ? kX : kA)) continue;  // below the last bit
#pragma unroll
                        for (int q = 0; q < 2; ++q)
#pragma unroll
                            for (int j = 0; j < 4; ++j)
                                mma_k16<!F16>(ALONE ? block[j] : acc[j0 + j], f[i][q], u[j][k][2 * q], u[j][k][2 * q + 1]);
                    }
                if constexpr (ALONE)
#pragma unroll
                    for (int j = 0; j < 4; ++j)
#pragma unroll
                        for (int e = 0; e < 4; ++e) acc[j0 + j][e] += block[j][e];
            }
        }
    }
    copies_wait(0);
    __syncthreads();

    // the second product's first blocks come while the sums are joined
    const Share h = share_of(p.y, p.y_token, p.y_whole == 2, n0);
    const int chunks = nt, log_chunks = 32 - __clz(chunks - 1), b_row = tid >> log_chunks, b_chunk = tid & ((1 << log_chunks) - 1);
    const uint16_t* const b_mine = bank_b + (n0 + b_row) * p.R + 8 * b_chunk;
    const auto load2 = [&](int b, int slot) {
        if (b < blocks2) {
            const uint32_t to = smem_addr(ring2 + slot * plan.stage2);
            if (p.y_whole) copy_rows(h, b, outputs, to);
            if (b_chunk < chunks) {
                const int step = kThreads >> log_chunks, left = outputs - b * kBlock;
                const uint16_t* src = b_mine + static_cast<int64_t>(b * kBlock) * p.R;
                uint32_t dst = to + kRows * kPitch + b_row * b_pitch + 16 * b_chunk;
                for (int r = b_row; r < kBlock; r += step, src += step * p.R, dst += step * b_pitch) copy16(dst, r < left ? src : bank_b, r < left ? 16 : 0);
            }
        }
        copies_end();
    };
    for (int b = 0; b < stages2 - 1; ++b) load2(b, b);
    // zeros in the places behind the rank, up to 32
    for (int i = tid; i < stages2 * kBlock; i += kThreads)
        for (int o = nt; o < (rank + 31) / 32 * 4; ++o)
            *reinterpret_cast<uint4*>(ring2 + i / kBlock * plan.stage2 + kRows * kPitch + i % kBlock * b_pitch + 16 * o) = make_uint4(0, 0, 0, 0);
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
        constexpr int kLanes = kThreads / kRows;  // of a row
        for (int i = tid % kLanes * 4; i < nt * 8; i += 4 * kLanes) {
            const int at = tid / kLanes * pitch + i;
            float4 v = ld4(parts_sums + at);
#pragma unroll
            for (int h = 1; h < kHalf; ++h) {
                const float4 w = ld4(parts_sums + at + h * kRows * pitch);
                v = make_float4(v.x + w.x, v.y + w.y, v.z + w.z, v.w + w.w);
            }
            st4(sums + at, v);
        }
    }
    cluster_arrive();
    cluster_wait();
    // the sums of all CTAs, scaled, as the second product's operand
    // Eight ranks of a row at a time, by four lanes that add up a quarter of the CTAs each; a thread has kAtOnce of them
    // under way.
    const int eights = (rank + 31) / 32 * 4, items = kRows * eights;
    constexpr int kAtOnce = MT == 1 ? 1 : 2;
    for (int i0 = tid >> 2; i0 < items; i0 += kAtOnce * (kThreads / 4)) {
        const int quarter = tid & 3;
        float t[kAtOnce][8] = {};
        for (int c = quarter * parts / 4; c < (quarter + 1) * parts / 4; ++c)
#pragma unroll
            for (int n = 0; n < kAtOnce; ++n) {
                const int i = i0 + n * (kThreads / 4), r = i / eights, o = i - r * eights;
                if (i >= items || r >= rows || 8 * o >= rank) continue;
                const uint32_t at = cluster_addr(sums + r * pitch + 8 * o, c);
                float v[8];
#pragma unroll
                for (int q = 0; q < 2; ++q)
                    asm volatile("ld.shared::cluster.v4.f32 {%0,%1,%2,%3}, [%4];"
                                 : "=f"(v[4 * q]), "=f"(v[4 * q + 1]), "=f"(v[4 * q + 2]), "=f"(v[4 * q + 3])
                                 : "r"(at + 16 * q));
#pragma unroll
                for (int e = 0; e < 8; ++e) t[n][e] += v[e];
            }
#pragma unroll
        for (int n = 0; n < kAtOnce; ++n) {
            const int i = i0 + n * (kThreads / 4), r = i / eights, o = i - r * eights;
#pragma unroll
            for (int d = 1; d < 4; d <<= 1)
#pragma unroll
                for (int e = 0; e < 8; ++e) t[n][e] += __shfl_xor_sync(kFull, t[n][e], d);
            if (i >= items) continue;
            // this lane's pair of the eight is lane 4 (r % 8) + o % 4's, registers (r / 8) % 2 and that + 2 of a step of 16
            uint32_t* const to = t_words + ((r >> 4) * (wide / 16) + (o >> 2) * 2) * kT * 128 + ((r & 7) * 4 + (o & 3)) * 4 + ((r >> 3) & 1);
#pragma unroll
            for (int q = 0; q < 4; ++q) {
                if (q != quarter) continue;
                const int e = 8 * o + 2 * q;
                uint32_t v[kT];
                split(e < rank ? t[n][2 * q] * scale : 0.0f, e + 1 < rank ? t[n][2 * q + 1] * scale : 0.0f, v);
#pragma unroll
                for (int k = 0; k < kT; ++k) to[((q >> 1) * kT + k) * 128 + 2 * (q & 1)] = v[k];
            }
        }
    }
    cluster_arrive();  // nobody leaves before its sums are read

    // out = y + (A x) B^T
    const uint4* const t_mine = reinterpret_cast<const uint4*>(t_words) + m * (wide / 16) * kT * 32 + lane;
    T* const out_lo = out + (r_lo < rows ? sh.row[r_lo] * p.out_token : 0) + n0 + 32 * sub + 8 * tq;
    T* const out_hi = out + (r_hi < rows ? sh.row[r_hi] * p.out_token : 0) + n0 + 32 * sub + 8 * tq;
    for (int b = 0, slot = 0, next = stages2 - 1; b < blocks2; ++b) {
        copies_wait(stages2 - 2);
        __syncthreads();
        load2(b + stages2 - 1, next);
        const uint8_t* const stage = ring2 + slot * plan.stage2;
        slot = slot + 1 == stages2 ? 0 : slot + 1, next = next + 1 == stages2 ? 0 : next + 1;
        if (!busy) continue;
        const uint8_t* const bank = stage + kRows * kPitch + (32 * sub + 8 * (g >> 1) + (g & 1)) * b_pitch + 16 * tq;
        const int n = b * kBlock + 32 * sub + 8 * tq;  // this lane's eight outputs, from n0
        // (of fp32 rows 32 ranks at a time, as above: 256 ranks of f16 banks 1.5e-6 of the result otherwise, 3.1e-7 so)
        constexpr bool ALONE = sizeof(T) == 4;
        float o[4][4] = {};
        for (int s0 = 0; 32 * s0 < rank; ++s0) {
            float block[4][4] = {};
            uint4 u[4];
#pragma unroll
            for (int j = 0; j < 4; ++j) u[j] = *reinterpret_cast<const uint4*>(bank + 2 * j * b_pitch + 64 * s0);
            if (rank & 7) {
                const int have = max(0, rank - 32 * s0 - 8 * tq);
#pragma unroll
                for (int j = 0; j < 4; ++j) u[j] = first_of(u[j], have);
            }
            uint32_t w[4][kB][4];
#pragma unroll
            for (int j = 0; j < 4; ++j) terms_of<!BF>(u[j], w[j]);
#pragma unroll
            for (int q = 0; q < 2; ++q)
#pragma unroll
                for (int i = 0; i < kT; ++i) {
                    const uint4 f4 = t_mine[((2 * s0 + q) * kT + i) * 32];
                    const uint32_t f[4] = {f4.x, f4.y, f4.z, f4.w};
#pragma unroll
                    for (int k = 0; k < kB; ++k) {
                        if (i + k >= kT) continue;  // below the last bit
#pragma unroll
                        for (int j = 0; j < 4; ++j) mma_k16<true>(ALONE ? block[j] : o[j], f, w[j][k][2 * q], w[j][k][2 * q + 1]);
                    }
                }
            if constexpr (ALONE)
#pragma unroll
                for (int j = 0; j < 4; ++j)
#pragma unroll
                    for (int e = 0; e < 4; ++e) o[j][e] += block[j][e];
        }
#pragma unroll
        for (int r = 0; r < 2; ++r) {
            const int at = r ? r_hi : r_lo;
            if (at >= rows || n >= outputs) continue;
            T* const to = (r ? out_hi : out_lo) + b * kBlock;
            float v[8];
            if (p.y_whole) {
                ld8(reinterpret_cast<const T*>(stage + at * kPitch) + 32 * sub + 8 * tq, v);
            } else {
                const T* const from = y + sh.row[at] * p.y_token + n0 + n;
#pragma unroll
                for (int e = 0; e < 8; ++e) v[e] = n + e < outputs ? ld1(from + e) : 0.0f;
            }
#pragma unroll
            for (int j = 0; j < 4; ++j)
#pragma unroll
                for (int e = 0; e < 2; ++e) v[2 * j + e] += o[j][2 * r + e];
            if (p.out_whole == 2 && n + 8 <= outputs) {
                st8(to, v);
            } else if (p.out_whole && n + 8 <= outputs) {
                st4(to, make_float4(v[0], v[1], v[2], v[3]));
                st4(to + 4, make_float4(v[4], v[5], v[6], v[7]));
            } else {
#pragma unroll
                for (int e = 0; e < 8; ++e)
                    if (n + e < outputs) st1(to + e, v[e]);
            }
        }
    }
    cluster_wait();
}

// Clusters of so many CTAs, one an SM, that this part holds at once (its clusters of SMs differ in size).
constexpr int at_once(int parts) { return parts > 8 ? 7 : parts > 4 ? 15 : 36; }

// groups: of the grid; working: at most so many of them have rows of an adapter.
template <typename T, bool BF, int NT, int WARPS, int MT>
cudaError_t launch(AdaptParams p, int64_t groups, int64_t working, int parts, cudaStream_t s) {
    using P = Plan<T, NT, WARPS, MT>;
    static_assert(P(8 * NT).bytes() + 1024 <= kSmemLimit, "ring, operand and sums of the largest rank in a CTA's shared memory");
    const P plan(p.R, working <= at_once(parts));
    p.stages1 = plan.stages1, p.stages2 = plan.stages2;
    static thread_local bool done[kMaxDevices] = {};
    const auto kernel = k_adapt<T, BF, NT, WARPS, MT>;
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e == cudaSuccess && (dev >= kMaxDevices || !done[dev])) {
        e = cudaFuncSetAttribute(kernel, cudaFuncAttributeNonPortableClusterSizeAllowed, 1);
        if (e == cudaSuccess) e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, kSmemLimit - 1024);
        if (e == cudaSuccess && dev < kMaxDevices) done[dev] = true;
    }
    if (e != cudaSuccess) return e;
    return launch_cluster(kernel, dim3(static_cast<unsigned>(groups * parts)), dim3(32 * WARPS), plan.bytes(), parts, s, p);
}

// What counts is that all working clusters are in flight at once, each of as many CTAs as that leaves (4096 to 4096, bf16
// banks).  Of single tokens at most one group an adapter, and one more for each 16 rows, works.
template <typename T, bool BF>
cudaError_t launch_type(const AdaptParams& p, cudaStream_t s) {
    const int64_t seqs = std::min(p.seqs, p.T);
    const int64_t groups = p.q_start ? p.T / 16 + seqs : p.seqs <= kAdaptSorted ? std::min(p.seqs, p.n + 1 + p.seqs / 16) : p.seqs;
    const int64_t working = p.q_start ? groups : std::min(p.seqs, p.n + p.seqs / 16);
    if (p.q_start && p.T > 8 * p.seqs && p.R <= 128 && working > (p.R <= 64 ? 74 : at_once(4))) {
        // Prompts whose groups of 16 rows do not fit: tiles of 32 rows, and so many CTAs of a tile that those which fit the
        // SMs at once are in flight (five prompts of 150 to 1000 rows, 92 tiles, fp32, rank 32: 49.5 us with 4, 40.1 with 6,
        // 61.7 with 8; one of 2048, fp32, rank 64: 43.3 us, 63.6 in groups; one of 1024: 37.7, 33.1 in groups).
        const int64_t tiles = p.T / 32 + seqs;
        const auto parts = [&](int ctas) { return std::max<int>(4, std::min<int>(8, 145 * ctas / tiles)); };
        if (p.R <= 64) return launch<T, BF, 8, 4, 2>(p, tiles, tiles, parts(Plan<T, 8, 4, 2>(p.R).ctas), s);
        return launch<T, BF, 16, 4, 2>(p, tiles, tiles, parts(Plan<T, 16, 4, 2>(p.R).ctas), s);
    }
    // Many groups of low ranks: small CTAs, four an SM (192 rows of 64 adapters, fp32, rank 64, a cluster a row: 30.2 us, 37.8
    // with 4 of eight warps; 96 of 32: 15.8 and 14.6; a cluster a group takes 23.9 and 14.8).
    if (p.R <= 64 && working > 74) return launch<T, BF, 8, 4, 1>(p, groups, working, 8, s);
    // 16 CTAs of a group, 8 or 4, as many as fit (a prompt of 64 rows, fp32, rank 16: 9.2 us, 9.9 with 8; one of 128: 11.7 and
    // 10.2; one of 256, rank 64: 23.6 with 8, 16.1 with 4).  Two CTAs of low ranks fit an SM; of single tokens, half of the
    // adapters are taken to be in use (64 rows, 8 of 24 adapters, rank 64: 12.6 us with 8, 15.0 with 4).
    const int most = at_once(8) * (p.R <= 32 ? 2 : 1) * (p.q_start ? 1 : 2);
    const int parts = working <= at_once(16) ? 16 : working <= most ? 8 : 4;
    if (p.R <= 64) return launch<T, BF, 8, 8, 1>(p, groups, working, parts, s);
    // (wide blocks of high ranks do not fit a CTA)
    if (p.R <= 128) return launch<T, BF, 16, 4, 1>(p, groups, working, parts, s);
    return launch<T, BF, 32, 4, 1>(p, groups, working, parts, s);
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
    p.out_whole = whole(p.out, p.out_token, 16) ? 2 : whole(p.out, p.out_token, 4 * size) ? 1 : 0;
    const bool bf = p.bank == 2;
    if (dtype == 0) return bf ? launch_type<float, true>(p, s) : launch_type<float, false>(p, s);
    if (dtype == 1) return bf ? launch_type<__half, true>(p, s) : launch_type<__half, false>(p, s);
    return bf ? launch_type<__nv_bfloat16, true>(p, s) : launch_type<__nv_bfloat16, false>(p, s);
}

}  // namespace ggq
