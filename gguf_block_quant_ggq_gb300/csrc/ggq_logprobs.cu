// ggq_logprobs.cu -- log probabilities of given tokens, entropy and the best alternatives.
//
// Mathematics, with m the largest logit and a_i = (x_i - m) scale log2(e): s = sum 2^a, w = sum 2^a a,
// log p_i = (x_i - m) scale - log s, entropy = log s - ln 2 w / s.  One pass: every thread keeps the
// largest logit, s and w of its part in fp32; parts are joined in a fixed order.
//
// A row is a cluster's: its CTAs take neighbouring parts and the first one joins them through
// distributed shared memory, so few rows use many SMs without scratch or a second launch.
//
// The best: in the pass nothing but the largest logit of each thread is kept.  Of the CTA's groups of
// eight lanes (64, or 32 of a CTA of 256 threads) the `top`-th largest maximum is a bound that at least `top` logits reach; threads whose maximum
// reaches it (a handful) have their part read again, by all, and what reaches the bound goes to a pool, whose
// entries find their places by counting those before them (value, then id), so the order in which
// they arrive does not show.  Where ties overflow the pool the places are found one after another, by `top` passes over
// the part: so in a CTA of whose groups fewer than `top` hold a value that its mask leaves (2048 rows of 100003 bf16
// logits, 8 and 20 best: 80 and 96 us, 0.19 and 0.20 ms with 50 values left in a row, 1.4 and 3.3 ms with 5; one row of 131072
// fp32 5.3 and 6.5 us, 25 and 53 with 50 or 5).
//
// Sums of 16-bit logits take five instructions a value, so that memory is the bound: masked
// values are raised to one that weighs 0 while they are packed, pairs are multiplied and added at once.
// Where that value would not weigh 0 (a row whose maximum is near it), the sums are done again
// with every value looked at.
#include "ggq_cluster.cuh"
#include "ggq_device.cuh"
#include "ggq_internal.h"
#include "ggq_kv.cuh"
#include "ggq_logprobs.cuh"
#include "ggq_tcgen05.cuh"

namespace ggq {

namespace {

constexpr uint32_t kFull = 0xffffffffu;
constexpr int kMaxWarps = 16;
constexpr int kMaxParts = 8;  // CTAs a row
constexpr int kPool = 512;
constexpr int kNone = INT32_MAX;
constexpr float kLog2e = 1.4426950408889634f, kLn2 = 0.6931471805599453f;
constexpr float kGone = -150.0f;  // 2^a from here down is no part of a sum in fp32 whose largest term is 1

struct Sums {
    float m, s, w;  // largest logit (-inf without one), sums about it
};
__device__ __forceinline__ float pow2(float a) {
    float r;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(a));
    return r;
}
// Sums about the larger logit m.  (Differences of infinities are NaN, which the maximum leaves out.)
__device__ __forceinline__ void raise(Sums& v, float m, float c) {
    const float a = fmaxf((v.m - m) * c, -1000.0f), f = pow2(a);
    v.w = f * fmaf(a, v.s, v.w);
    v.s *= f;
    v.m = m;
}
__device__ __forceinline__ Sums join(Sums a, Sums b, float c) {
    const float m = fmaxf(a.m, b.m);
    raise(a, m, c);
    raise(b, m, c);
    return {m, a.s + b.s, a.w + b.w};
}
__device__ __forceinline__ Sums warp_join(Sums v, float c) {
#pragma unroll
    for (int d = 16; d >= 1; d >>= 1)
        v = join(v, Sums{__shfl_xor_sync(kFull, v.m, d), __shfl_xor_sync(kFull, v.s, d), __shfl_xor_sync(kFull, v.w, d)}, c);
    return v;
}
__device__ __forceinline__ Sums no_sums() { return {-INFINITY, 0.0f, 0.0f}; }

// One value, whatever it is (NaN and -inf weigh 0).
__device__ __forceinline__ void add_one(Sums& v, float x, float c) {
    if (!(x > -INFINITY)) return;
    if (x > v.m) raise(v, x, c);
    const float a = fmaxf((x - v.m) * c, -1000.0f), e = pow2(a);
    v.s += e;
    v.w = fmaf(e, a, v.w);
}

// Two sums and two products at once
__device__ __forceinline__ void add2(float& d0, float& d1, float a0, float a1, float b0, float b1) {
    asm("{\n\t.reg .b64 ra, rb, rd;\n\tmov.b64 ra, {%2, %3};\n\tmov.b64 rb, {%4, %5};\n\tadd.rn.f32x2 rd, ra, rb;\n\t"
        "mov.b64 {%0, %1}, rd;\n\t}" : "=f"(d0), "=f"(d1) : "f"(a0), "f"(a1), "f"(b0), "f"(b1));
}
__device__ __forceinline__ void mul2(float& d0, float& d1, float a0, float a1, float b) {
    asm("{\n\t.reg .b64 ra, rb, rd;\n\tmov.b64 ra, {%2, %3};\n\tmov.b64 rb, {%4, %4};\n\tmul.rn.f32x2 rd, ra, rb;\n\t"
        "mov.b64 {%0, %1}, rd;\n\t}" : "=f"(d0), "=f"(d1) : "f"(a0), "f"(a1), "f"(b));
}

// Whether (x, i) stands before (y, j)
__device__ __forceinline__ bool before(float x, int i, float y, int j) { return x > y || (x == y && i < j); }

struct Shared {
    Sums sums[kMaxWarps];
    float group[4 * kMaxWarps];
    float bound;
    int count, hots;
    int16_t hot[32 * kMaxWarps];
    float pool_x[kPool];
    int pool_id[kPool];
    float best_x[kLogprobsMaxTop];
    int best_id[kLogprobsMaxTop];
    float pick_x[kMaxWarps];
    int pick_id[kMaxWarps];
    // of the cluster's CTAs, in the first one
    Sums part[kMaxParts];
    float part_x[kMaxParts * kLogprobsMaxTop];
    int part_id[kMaxParts * kLogprobsMaxTop];
};

// The entries of (x, id)[n] that come first, in order, to best_x, best_id (entries without an id come nowhere).  As many
// neighbouring lanes an entry as there are threads for count those before it.
template <int kRowThreads>
__device__ __forceinline__ void rank_entries(const float* x, const int* id, int n, int top, float* best_x, int* best_id) {
    int log_lanes = 5;
    while (log_lanes > 0 && n << log_lanes > kRowThreads) --log_lanes;
    const int lanes = 1 << log_lanes, mine = threadIdx.x & (lanes - 1), step = kRowThreads >> log_lanes;
    for (int i0 = 0; i0 < n; i0 += step) {
        const int i = i0 + (static_cast<int>(threadIdx.x) >> log_lanes);
        const float mx = i < n ? x[i] : 0.0f;
        const int mi = i < n ? id[i] : kNone;
        int at = 0;
        for (int j = mine; j < n; j += lanes) at += before(x[j], id[j], mx, mi) ? 1 : 0;
        for (int d = 1; d < lanes; d <<= 1) at += __shfl_xor_sync(kFull, at, d);
        if (mine == 0 && mi != kNone && at < top) best_x[at] = mx, best_id[at] = mi;
    }
}

// The same of `parts` lists of `top` entries in order each: a place in a list is found by halving it.
template <int kRowThreads>
__device__ __forceinline__ void rank_lists(const float* x, const int* id, int parts, int top, float* best_x, int* best_id) {
    const int n = parts * top;
    int log_lanes = 3;  // lanes an entry, each with its share of the lists
    while (log_lanes > 0 && n << log_lanes > kRowThreads) --log_lanes;
    const int lanes = 1 << log_lanes, mine = threadIdx.x & (lanes - 1), step = kRowThreads >> log_lanes;
    for (int i0 = 0; i0 < n; i0 += step) {
        const int i = i0 + (static_cast<int>(threadIdx.x) >> log_lanes);
        const float mx = i < n ? x[i] : 0.0f;
        const int mi = i < n ? id[i] : kNone;
        int at = 0;
        for (int c = mine; c < parts; c += lanes) {
            int lo = 0, hi = top;  // entries of list c before this one
            while (lo < hi) {
                const int j = (lo + hi) >> 1;
                if (before(x[c * top + j], id[c * top + j], mx, mi)) lo = j + 1;
                else hi = j;
            }
            at += lo;
        }
        for (int d = 1; d < lanes; d <<= 1) at += __shfl_xor_sync(kFull, at, d);
        if (mine == 0 && mi != kNone && at < top) best_x[at] = mx, best_id[at] = mi;
    }
}

// A thread's 16 bytes of logits.
template <typename T>
struct Vec {
    static constexpr int kN = 16 / sizeof(T);
    static __device__ __forceinline__ void unpack(uint4 u, float (&x)[kN]) {
        const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            if constexpr (sizeof(T) == 4) {
                x[i] = __uint_as_float(w[i]);
            } else if constexpr (__is_same(T, __half)) {
                const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&w[i]));
                x[2 * i] = f.x, x[2 * i + 1] = f.y;
            } else {
                x[2 * i] = __uint_as_float(w[i] << 16), x[2 * i + 1] = __uint_as_float(w[i] & 0xFFFF0000u);
            }
        }
    }
    // values that masks leave out, raised to low()
    static __device__ __forceinline__ float low() { return __is_same(T, __half) ? -65504.0f : -0x1p100f; }
    static __device__ __forceinline__ uint32_t max2(uint32_t a, uint32_t b) {
        uint32_t r;
        if constexpr (__is_same(T, __half)) asm("max.f16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
        else asm("max.bf16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
        return r;
    }
    static __device__ __forceinline__ uint4 raised(uint4 u) {
        if constexpr (sizeof(T) == 4) {
            const auto up = [](uint32_t w) { return __float_as_uint(fmaxf(__uint_as_float(w), -0x1p100f)); };
            return make_uint4(up(u.x), up(u.y), up(u.z), up(u.w));
        } else {
            const uint32_t l = __is_same(T, __half) ? 0xfbfffbffu : 0xf180f180u;  // -65504, -2^100
            return make_uint4(max2(u.x, l), max2(u.y, l), max2(u.z, l), max2(u.w, l));
        }
    }
    // the largest of raised values
    template <int N>
    static __device__ __forceinline__ float largest(const uint4 (&u)[N]) {
        if constexpr (sizeof(T) == 4) {
            float m = -INFINITY;
#pragma unroll
            for (int k = 0; k < N; ++k)
                m = fmaxf(m, fmaxf(fmaxf(__uint_as_float(u[k].x), __uint_as_float(u[k].y)), fmaxf(__uint_as_float(u[k].z), __uint_as_float(u[k].w))));
            return m;
        } else {
            uint32_t m = max2(max2(u[0].x, u[0].y), max2(u[0].z, u[0].w));
#pragma unroll
            for (int k = 1; k < N; ++k) m = max2(m, max2(max2(u[k].x, u[k].y), max2(u[k].z, u[k].w)));
            float x[kN];
            unpack(make_uint4(m, m, m, m), x);
            return fmaxf(x[0], x[1]);
        }
    }
    static __device__ __forceinline__ uint4 none() {
        const uint32_t l = sizeof(T) == 4 ? 0xff800000u : __is_same(T, __half) ? 0xfc00fc00u : 0xff80ff80u;  // -inf
        return make_uint4(l, l, l, l);
    }
};

// TOP: whether alternatives are asked for
template <typename T, bool TOP, int kRowThreads>
__global__ void __launch_bounds__(kRowThreads, 1024 / kRowThreads) k_logprobs(const __grid_constant__ LogprobsParams p) {
    pdl_launch_dependents();
    pdl_wait();
    using V = Vec<T>;
    constexpr int kN = V::kN, kLoads = 4, kWarps = kRowThreads / 32, kGroups = kRowThreads / 8;
    static_assert(kGroups >= kLogprobsMaxTop && 2 * 16 <= kRowThreads, "the bound and the row's ends");
    __shared__ Shared sh;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int rank = static_cast<int>(cluster_rank()), parts = static_cast<int>(cluster_size());
    if (parts > 1) cluster_arrive();  // every CTA runs before one writes to another
    const int64_t t = blockIdx.x / parts;
    const T* const row = static_cast<const T*>(p.logits) + t * p.row;
    const float c = fminf(p.scale * kLog2e, 0x1.fffffep127f);  // (0 times infinity is no weight)
    if (TOP && tid == 0) sh.count = 0, sh.hots = 0;

    // the row's first value at 16 bytes, and whole vectors from there; the ends are the first CTA's, one a thread
    const int skew = static_cast<int>((reinterpret_cast<uintptr_t>(row) & 15) / sizeof(T));
    const int head = min(p.V, skew ? kN - skew : 0), vectors = (p.V - head) / kN, tail = p.V - head - vectors * kN;
    const int per = (vectors + parts - 1) / parts, v0 = min(vectors, rank * per), v1 = min(vectors, v0 + per);
    const uint4* const body = reinterpret_cast<const uint4*>(row + head);
    const int end_id = rank ? kNone : tid < head ? tid : tid >= 16 && tid < 16 + tail ? p.V - tail + tid - 16 : kNone;
    const float end_x = end_id != kNone ? ld1(row + end_id) : -INFINITY;

    // the first given tokens' logits
    int given_id = -1;
    float given_x = 0.0f;
    if (rank == 0 && tid < min(32, p.given)) {
        given_id = p.tokens[t * p.given + tid];
        if (given_id >= 0 && given_id < p.V) given_x = ld1(row + given_id);
    }

    Sums v = no_sums();
    uint4 u[kLoads];
    const auto load = [&](int at, uint4 (&u)[kLoads]) {
#pragma unroll
        for (int k = 0; k < kLoads; ++k) u[k] = at + kRowThreads * k < v1 ? body[at + kRowThreads * k] : V::none();
    };
    {
        float s0 = 0.0f, s1 = 0.0f, w0 = 0.0f, w1 = 0.0f;
        uint4 next[kLoads];
        load(v0 + tid, next);
        for (int at = v0 + tid; at < v1; at += kRowThreads * kLoads) {
#pragma unroll
            for (int k = 0; k < kLoads; ++k) u[k] = V::raised(next[k]);
            load(at + kRowThreads * kLoads, next);
            const float m = V::largest(u);
            if (m > v.m) {
                const float a = fmaxf((v.m - m) * c, -1000.0f), f = pow2(a);
                w0 = f * fmaf(a, s0, w0), w1 = f * fmaf(a, s1, w1);
                s0 *= f, s1 *= f;
                v.m = m;
            }
#pragma unroll
            for (int k = 0; k < kLoads; ++k) {
                float x[kN];
                V::unpack(u[k], x);
#pragma unroll
                for (int i = 0; i < kN; i += 2) {
                    float a0, a1;
                    add2(a0, a1, x[i], x[i + 1], -v.m, -v.m);
                    mul2(a0, a1, a0, a1, c);
                    const float e0 = pow2(a0), e1 = pow2(a1);
                    ffma2p(w0, w1, e0, e1, a0, a1, w0, w1);
                    add2(s0, s1, e0, e1, s0, s1);
                }
            }
        }
        v.s = s0 + s1, v.w = w0 + w1;
    }
    // the smallest values weigh 0 beside the thread's largest one, or every value is looked at
    const float least = (V::low() - v.m) * c;
    const bool plain = v.m < INFINITY && least <= kGone && least > -INFINITY;
    if (v0 + tid < v1 && !plain) {
        v = no_sums();
        for (int at = v0 + tid; at < v1; at += kRowThreads) {
            float x[kN];
            V::unpack(body[at], x);
#pragma unroll
            for (int i = 0; i < kN; ++i) add_one(v, x[i], c);
        }
    }
    if (end_id != kNone) add_one(v, end_x, c);
    const float mine = v.m;

    // the bound
    if constexpr (TOP) {
        float g = mine;
#pragma unroll
        for (int d = 4; d >= 1; d >>= 1) g = fmaxf(g, __shfl_xor_sync(kFull, g, d));
        if ((lane & 7) == 0) sh.group[tid >> 3] = g;
    }
    v = warp_join(v, c);
    if (lane == 0) sh.sums[warp] = v;
    __syncthreads();
    if constexpr (TOP) {
        {
            // eight lanes a group count those before it
            const float g = sh.group[tid >> 3];
            int at = 0;
#pragma unroll
            for (int j = tid & 7; j < kGroups; j += 8) at += before(sh.group[j], j, g, tid >> 3) ? 1 : 0;
#pragma unroll
            for (int d = 1; d < 8; d <<= 1) at += __shfl_xor_sync(kFull, at, d);
            if ((tid & 7) == 0 && at == p.top - 1) sh.bound = g;
        }
        __syncthreads();
        const float bound = sh.bound;
        const auto offer = [&](float x, int id) {
            if (x != x) x = -INFINITY;
            if (!(x >= bound)) return;
            const int at = atomicAdd(&sh.count, 1);
            if (at < kPool) sh.pool_x[at] = x, sh.pool_id[at] = id;
        };
        if (end_id != kNone) offer(end_x, end_id);
        const bool once = v1 - v0 <= kRowThreads * kLoads;
        if (once && bound > V::low()) {
            // the values are still here
            if (v0 + tid < v1 && mine >= bound)
#pragma unroll
                for (int k = 0; k < kLoads; ++k) {
                    float x[kN];
                    V::unpack(u[k], x);
#pragma unroll
                    for (int i = 0; i < kN; ++i) offer(x[i], head + (v0 + tid + kRowThreads * k) * kN + i);
                }
        } else {
            // the parts of the threads whose values reach the bound are read again, by all
            if (v0 + tid < v1 && mine >= bound) sh.hot[atomicAdd(&sh.hots, 1)] = static_cast<int16_t>(tid);
            __syncthreads();
            const int each = (v1 - v0 + kRowThreads - 1) / kRowThreads, items = sh.hots * each;
            for (int i = tid; i < items; i += kRowThreads) {
                const int h = i / each, at = v0 + sh.hot[h] + kRowThreads * (i - h * each);
                if (at >= v1 || *static_cast<volatile int*>(&sh.count) > kPool) continue;
                float x[kN];
                V::unpack(body[at], x);
#pragma unroll
                for (int i = 0; i < kN; ++i) offer(x[i], head + at * kN + i);
            }
        }
        if (tid < p.top) sh.best_x[tid] = -INFINITY, sh.best_id[tid] = kNone;
        __syncthreads();
        const int n = sh.count;
        if (n <= kPool) {
            rank_entries<kRowThreads>(sh.pool_x, sh.pool_id, n, p.top, sh.best_x, sh.best_id);
            __syncthreads();
        } else {
            // place by place: the first value behind the last one taken
            float last_x = INFINITY;
            int last_id = -1;
            for (int j = 0; j < p.top; ++j) {
                float bx = -INFINITY;
                int bi = kNone;
                const auto look = [&](float x, int id) {
                    if (x != x) x = -INFINITY;
                    if (before(last_x, last_id, x, id) && before(x, id, bx, bi)) bx = x, bi = id;
                };
                if (end_id != kNone) look(end_x, end_id);
                for (int at = v0 + tid; at < v1; at += kRowThreads) {
                    float x[kN];
                    V::unpack(body[at], x);
#pragma unroll
                    for (int i = 0; i < kN; ++i) look(x[i], head + at * kN + i);
                }
#pragma unroll
                for (int d = 16; d >= 1; d >>= 1) {
                    const float ox = __shfl_xor_sync(kFull, bx, d);
                    const int oi = __shfl_xor_sync(kFull, bi, d);
                    if (before(ox, oi, bx, bi)) bx = ox, bi = oi;
                }
                if (lane == 0) sh.pick_x[warp] = bx, sh.pick_id[warp] = bi;
                __syncthreads();
                for (int w = 0; w < kWarps; ++w)
                    if (w == 0 || before(sh.pick_x[w], sh.pick_id[w], bx, bi)) bx = sh.pick_x[w], bi = sh.pick_id[w];
                last_x = bx, last_id = bi;
                if (tid == 0) sh.best_x[j] = bx, sh.best_id[j] = bi;
                __syncthreads();
                if (bi == kNone) break;
            }
        }
    }

    // the CTA, the cluster
    if (warp == 0) v = warp_join(lane < kWarps ? sh.sums[lane] : no_sums(), c);
    if (parts > 1) {
        cluster_wait();
        if (warp == 0) {
            if (lane == 0) {
                const uint32_t to = cluster_addr(&sh.part[rank], 0);
                st_cluster(to, __float_as_uint(v.m));
                st_cluster(to + 4, __float_as_uint(v.s));
                st_cluster(to + 8, __float_as_uint(v.w));
            }
            if (TOP && lane < p.top) {
                st_cluster(cluster_addr(&sh.part_x[rank * p.top + lane], 0), __float_as_uint(sh.best_x[lane]));
                st_cluster(cluster_addr(&sh.part_id[rank * p.top + lane], 0), static_cast<uint32_t>(sh.best_id[lane]));
            }
            __syncwarp();
        }
        cluster_arrive();
        cluster_wait();
        if (rank != 0) return;
        if (warp == 0) v = warp_join(lane < parts ? sh.part[lane] : no_sums(), c);
        if constexpr (TOP) {
            rank_lists<kRowThreads>(sh.part_x, sh.part_id, parts, p.top, sh.best_x, sh.best_id);
            __syncthreads();
        }
    }
    if (warp != 0) return;
    const float log_sum = logf(v.s);
    const bool nothing = v.m == -INFINITY;  // a mask over the whole row
    const auto logprob = [&](float x) {
        if (v.m == INFINITY) return NAN;
        if (!(x > -INFINITY)) return -INFINITY;
        return (x - v.m) * p.scale - log_sum;
    };
    if (p.entropy && lane == 0) p.entropy[t] = nothing ? 0.0f : v.m == INFINITY ? NAN : fmaxf(0.0f, log_sum - kLn2 * (v.w / v.s));
    for (int j = lane; j < p.given; j += 32) {
        if (j >= 32) {
            given_id = p.tokens[t * p.given + j];
            if (given_id >= 0 && given_id < p.V) given_x = ld1(row + given_id);
        }
        if (given_id >= p.V) set_error(p.err, DEV_ERR_BAD_TOKEN);
        p.logprobs[t * p.given + j] = given_id < 0 || given_id >= p.V ? 0.0f : logprob(given_x);
    }
    if (TOP && lane < p.top) {
        p.ids[t * p.top + lane] = sh.best_id[lane];
        p.best[t * p.top + lane] = logprob(sh.best_x[lane]);
    }
}

template <typename T, bool TOP>
cudaError_t launch(const LogprobsParams& p, cudaStream_t s) {
    // CTAs a row: a cluster costs 1 us and pays from some 16 thousand logits a CTA on, as long as each has an SM, or two half
    // of one (top 8, us with 1 / 2 / 4 / 8 / 16 CTAs: one row of 131072 fp32 8.9 / 7.4 / 6.0 / 5.5 / 6.0, of 32000 bf16 5.0 / 5.7 /
    // 5.7 / 5.8 / 6.3; 19 rows of 262144 bf16 13.8 / 10.0 / 9.4 / 8.5 / 12.1; 76 17.6 / 13.2 / 18.2 / 22.4 / 34.9)
    int parts = 1;
    while (parts < kMaxParts && p.T * parts * 2 <= (parts == 1 ? 304 : 152) && p.V / (2 * parts) >= 16384) parts *= 2;
    // Smaller CTAs for short rows, and for more rows than SMs hold of the large ones, so that an SM sums some while it ranks
    // others (bf16, us with 256 / 512 threads: 500 rows of 32000 10.1 / 13.7, 2048 of 100003 79 / 88); but not of rows above
    // 256 KB, whose reading outweighs that (200064 logits, fp32: 620 rows 115 / 94, 2048 286 / 253, 4096 545 / 499; bf16: 62 / 55,
    // 151 / 143, 281 / 273; at the border, 131072 bf16: 620 rows 41 / 38, 2048 98 / 98, 8192 348 / 354).  Up to 608 rows the
    // larger CTAs do not fill the SMs twice and the two differ little (500 rows of 131072, fp32 47.5 / 46.1, bf16 29.0 / 29.5).
    const bool lengthy = static_cast<int64_t>(p.V) * sizeof(T) > 256 * 1024 && p.T > 608;
    if (parts == 1 && (p.V <= 16384 || (p.T > 304 && !lengthy)))
        return launch_cluster(k_logprobs<T, TOP, 256>, dim3(static_cast<unsigned>(p.T)), dim3(256), 0, 1, s, p);
    return launch_cluster(k_logprobs<T, TOP, 512>, dim3(static_cast<unsigned>(p.T * parts)), dim3(512), 0, parts, s, p);
}

template <typename T>
cudaError_t launch_type(const LogprobsParams& p, cudaStream_t s) {
    return p.top ? launch<T, true>(p, s) : launch<T, false>(p, s);
}

}  // namespace

cudaError_t launch_logprobs(const LogprobsParams& p, int dtype, cudaStream_t s) {
    if (p.T == 0) return cudaSuccess;
    if (dtype == 0) return launch_type<float>(p, s);
    if (dtype == 1) return launch_type<__half>(p, s);
    return launch_type<__nv_bfloat16>(p, s);
}

}  // namespace ggq
