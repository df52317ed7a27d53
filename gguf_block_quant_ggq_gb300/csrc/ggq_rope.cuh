// ggq_rope.cuh -- the rotation of positions: parameters, and the device code that the
// rotation alone (ggq_rope.cu) and the cache's writer (ggq_kv.cu) share.
//
// Mathematics: pair j of a head's turned channels, (a, b), becomes (a c - b s, a s + b c) with
// (c, s) the table's entry of the token's position and j.  Products and their sum are rounded
// one by one in fp32, so that the result is the same wherever it is computed.
#pragma once
#include <stdint.h>

#include <type_traits>

#include "ggq_device.cuh"
#include "ggq_kv.cuh"

namespace ggq {

constexpr int kRotaryMaxDim = 1024;

struct Rotary {
    const float2* table;  // [n_positions][half]
    int64_t n_positions;
    const int32_t* positions;  // one a token
    int half;   // pairs of a head
    int first;  // first turned channel
    int pairs;  // 1: neighbours (2 j, 2 j + 1), 0: halves (j, j + half)
    int whole;  // 4, 8: half and first are multiples of it and the table starts at 16 bytes (cache writer)
};

// Queries and keys outside the cache that are turned: rows, heads, strides in elements.
struct RotateParams {
    Rotary r;
    const void* x;
    void* out;
    int64_t x_token, x_head, out_token, out_head;
    const int64_t* slots;  // or null; a token with a negative slot has no position to report
    int64_t T;
    int H, D;
    int units;     // units of 2 V channels of a head: first the turned ones, then those that stay
    int in_place;  // x and out are the same rows
    int heads_at_once, rows_at_once;
    int* err;
};

// The table's row of a token: null for a position outside the table, which turns nothing.
__device__ __forceinline__ const float2* rotary_row(const Rotary& r, int64_t token) {
    const int64_t pos = r.positions[token];
    return pos >= 0 && pos < r.n_positions ? r.table + pos * r.half : nullptr;
}

__device__ __forceinline__ float turned_a(float a, float b, float2 cs) { return __fsub_rn(__fmul_rn(a, cs.x), __fmul_rn(b, cs.y)); }
__device__ __forceinline__ float turned_b(float a, float b, float2 cs) { return __fadd_rn(__fmul_rn(a, cs.y), __fmul_rn(b, cs.x)); }

// V consecutive elements of a row, as they come from memory
template <int V, typename T>
struct RawV {
    static constexpr int kBytes = V * static_cast<int>(sizeof(T));
    using Word = typename std::conditional<kBytes == 16, uint4, typename std::conditional<kBytes == 8, uint2, T>::type>::type;
    Word w;
    __device__ __forceinline__ void load(const T* p) { w = *reinterpret_cast<const Word*>(p); }
    __device__ __forceinline__ void to(float (&x)[V]) const {
        if constexpr (V == 1) {
            x[0] = ld1(&w);
        } else if constexpr (V == 4) {
            const float4 f = ld4(reinterpret_cast<const T*>(&w));
            x[0] = f.x, x[1] = f.y, x[2] = f.z, x[3] = f.w;
        } else {
            const uint32_t u[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                if constexpr (__is_same(T, __half)) {
                    const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&u[i]));
                    x[2 * i] = f.x, x[2 * i + 1] = f.y;
                } else {
                    x[2 * i] = __uint_as_float(u[i] << 16), x[2 * i + 1] = __uint_as_float(u[i] & 0xFFFF0000u);
                }
            }
        }
    }
};
template <int V>
__device__ __forceinline__ void stv(float* p, const float (&x)[V]) {
    if constexpr (V == 1) *p = x[0];
    else
#pragma unroll
        for (int i = 0; i < V; i += 4) st4(p + i, make_float4(x[i], x[i + 1], x[i + 2], x[i + 3]));
}
template <int V, typename T>
__device__ __forceinline__ void stv(T* p, const float (&x)[V]) {
    if constexpr (V == 1) {
        st1(p, x[0]);
    } else if constexpr (V == 4) {
        st4(p, make_float4(x[0], x[1], x[2], x[3]));
    } else {
        uint32_t w[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            if constexpr (__is_same(T, __half)) {
                const __half2 h = __floats2half2_rn(x[2 * i], x[2 * i + 1]);
                w[i] = *reinterpret_cast<const uint32_t*>(&h);
            } else {
                const __nv_bfloat162 h = __floats2bfloat162_rn(x[2 * i], x[2 * i + 1]);
                w[i] = *reinterpret_cast<const uint32_t*>(&h);
            }
        }
        *reinterpret_cast<uint4*>(p) = make_uint4(w[0], w[1], w[2], w[3]);
    }
}

// Turns the heads h0 .. h1 - 1 of the rows r0 .. r1 - 1.  A thread has one unit of a row, 2 V
// channels, and takes it through the heads, four at a time, with its table entries in registers.
template <int V, typename T>
__device__ __forceinline__ void rotate_tile(const RotateParams& p, int64_t r0, int64_t r1, int h0, int h1) {
    const int turned = p.r.half / V, items = static_cast<int>(r1 - r0) * p.units;
    for (int item = threadIdx.x; item < items; item += blockDim.x) {
        const int row = item / p.units, u = item - row * p.units;
        const int64_t t = r0 + row;
        bool turn = u < turned;
        int ca, cb;  // first channels of the unit's two vectors
        bool two = true;
        float2 cs[V];
        if (turn) {
            ca = p.r.first + u * V * (p.r.pairs ? 2 : 1);
            cb = ca + (p.r.pairs ? V : p.r.half);
            const float2* const entry = rotary_row(p.r, t);
            if (entry) {
                if constexpr (V == 1) {
                    cs[0] = entry[u];
                } else {
#pragma unroll
                    for (int i = 0; i < V; i += 2) {
                        const float4 f = *reinterpret_cast<const float4*>(entry + u * V + i);
                        cs[i] = make_float2(f.x, f.y), cs[i + 1] = make_float2(f.z, f.w);
                    }
                }
            } else {
                // as they are (0 times what is not finite is NaN)
                if (!p.slots || p.slots[t] >= 0) set_error(p.err, DEV_ERR_BAD_POSITION);
                if (p.in_place) continue;
                turn = false;
            }
        } else {
            if (p.in_place) continue;
            // channels before and behind the turned ones, in order
            const int k = 2 * (u - turned) * V;
            ca = k < p.r.first ? k : k + 2 * p.r.half;
            cb = k + V < p.r.first ? k + V : k + V + 2 * p.r.half;
            two = cb < p.D;
        }
        const T* const src = static_cast<const T*>(p.x) + t * p.x_token;
        T* const dst = static_cast<T*>(p.out) + t * p.out_token;
        const auto one = [&](T* to, const RawV<V, T>& ra, const RawV<V, T>& rb) {
            float a[V], b[V];
            ra.to(a);
            rb.to(b);
            if (!turn) {
                stv<V>(to + ca, a);
                if (two) stv<V>(to + cb, b);
                return;
            }
            float ya[V], yb[V];
            if (V > 1 && p.r.pairs) {
#pragma unroll
                for (int i = 0; i < V; ++i) {  // pair i: elements 2 i and 2 i + 1 of the two vectors together
                    const float e = 2 * i < V ? a[2 * i % V] : b[2 * i % V], o = 2 * i < V ? a[(2 * i + 1) % V] : b[(2 * i + 1) % V];
                    (2 * i < V ? ya : yb)[2 * i % V] = turned_a(e, o, cs[i]);
                    (2 * i < V ? ya : yb)[(2 * i + 1) % V] = turned_b(e, o, cs[i]);
                }
            } else {
#pragma unroll
                for (int i = 0; i < V; ++i) ya[i] = turned_a(a[i], b[i], cs[i]), yb[i] = turned_b(a[i], b[i], cs[i]);
            }
            stv<V>(to + ca, ya);
            stv<V>(to + cb, yb);
        };
        int h = h0;
        for (; h + 4 <= h1; h += 4) {
            RawV<V, T> a[4], b[4];
#pragma unroll
            for (int k = 0; k < 4; ++k) {
                a[k].load(src + (h + k) * p.x_head + ca);
                b[k].load(src + (h + k) * p.x_head + (two ? cb : ca));
            }
#pragma unroll
            for (int k = 0; k < 4; ++k) one(dst + (h + k) * p.out_head, a[k], b[k]);
        }
        for (; h < h1; ++h) {
            RawV<V, T> a, b;
            a.load(src + h * p.x_head + ca);
            b.load(src + h * p.x_head + (two ? cb : ca));
            one(dst + h * p.out_head, a, b);
        }
    }
}

// Channels c .. c + 7 (c a multiple of 8) of the head that starts at `head`, turned.  entry: the row's table entries, null:
// as they are.
template <typename T>
__device__ __forceinline__ void turned8(const Rotary& r, const T* head, int c, const float2* entry, float (&x)[8]) {
    const auto load = [&](int at, float (&v)[8]) {
        const float4 a = ld4(head + at), b = ld4(head + at + 4);
        v[0] = a.x, v[1] = a.y, v[2] = a.z, v[3] = a.w, v[4] = b.x, v[5] = b.y, v[6] = b.z, v[7] = b.w;
    };
    load(c, x);
    const int at = c - r.first;
    if (!entry || at + 8 <= 0 || at >= 2 * r.half) return;
    if (r.whole == 8) {
        // eight of the first halves, of the second ones, or four pairs
        const bool low = r.pairs || at < r.half;
        const int j = r.pairs ? at / 2 : low ? at : at - r.half;
        float other[8];
        if (!r.pairs) load(low ? c + r.half : c - r.half, other);
#pragma unroll
        for (int i = 0; i < 8; i += 2) {
            if (r.pairs) {
                const float2 cs = entry[j + i / 2];
                const float e = x[i], o = x[i + 1];
                x[i] = turned_a(e, o, cs), x[i + 1] = turned_b(e, o, cs);
            } else {
                const float4 f = *reinterpret_cast<const float4*>(entry + j + i);
                const float2 c0 = make_float2(f.x, f.y), c1 = make_float2(f.z, f.w);
                x[i] = low ? turned_a(x[i], other[i], c0) : turned_b(other[i], x[i], c0);
                x[i + 1] = low ? turned_a(x[i + 1], other[i + 1], c1) : turned_b(other[i + 1], x[i + 1], c1);
            }
        }
        return;
    }
    // channel by channel
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        const int k = at + i;
        if (k < 0 || k >= 2 * r.half) continue;
        const bool low = r.pairs ? !(k & 1) : k < r.half;
        const int j = r.pairs ? k >> 1 : low ? k : k - r.half, step = r.pairs ? 1 : r.half;
        const float other = ld1(head + c + i + (low ? step : -step));
        x[i] = low ? turned_a(x[i], other, entry[j]) : turned_b(other, x[i], entry[j]);
    }
}

// Two quads of a head of D channels that one thread turns: unit u of D / 8 (of a rotation of whole quads).
struct Turn4 {
    int ca, cb;    // first channels
    bool turn;
    float2 cs[4];
};
__device__ __forceinline__ Turn4 turn4_of(const Rotary& r, int u, const float2* entry) {
    Turn4 t;
    t.turn = 4 * u < r.half;
    if (t.turn) {
        t.ca = r.first + (r.pairs ? 8 * u : 4 * u), t.cb = t.ca + (r.pairs ? 4 : r.half);
    } else {
        const int k = 8 * u - 2 * r.half;  // of the channels that stay
        t.ca = k < r.first ? k : k + 2 * r.half, t.cb = k + 4 < r.first ? k + 4 : k + 4 + 2 * r.half;
    }
    t.turn = t.turn && entry;
#pragma unroll
    for (int i = 0; i < 4; i += 2) {
        const float4 f = t.turn ? *reinterpret_cast<const float4*>(entry + 4 * u + i) : make_float4(1.f, 0.f, 1.f, 0.f);
        t.cs[i] = make_float2(f.x, f.y), t.cs[i + 1] = make_float2(f.z, f.w);
    }
    return t;
}
__device__ __forceinline__ void turn4(const Turn4& t, bool pairs, float4& a, float4& b) {
    if (!t.turn) return;
    const float4 p = a, q = b;
    if (pairs) {
        a = make_float4(turned_a(p.x, p.y, t.cs[0]), turned_b(p.x, p.y, t.cs[0]), turned_a(p.z, p.w, t.cs[1]), turned_b(p.z, p.w, t.cs[1]));
        b = make_float4(turned_a(q.x, q.y, t.cs[2]), turned_b(q.x, q.y, t.cs[2]), turned_a(q.z, q.w, t.cs[3]), turned_b(q.z, q.w, t.cs[3]));
    } else {
        a = make_float4(turned_a(p.x, q.x, t.cs[0]), turned_a(p.y, q.y, t.cs[1]), turned_a(p.z, q.z, t.cs[2]), turned_a(p.w, q.w, t.cs[3]));
        b = make_float4(turned_b(p.x, q.x, t.cs[0]), turned_b(p.y, q.y, t.cs[1]), turned_b(p.z, q.z, t.cs[2]), turned_b(p.w, q.w, t.cs[3]));
    }
}

constexpr int kRotateThreads = 128;

cudaError_t launch_rotate(RotateParams p, int dtype, cudaStream_t s);
// The widest vectors that a rotation of these rows can take: 8, 4 or 1 channels.
int rotate_vector(const RotateParams& p, int dtype);

cudaError_t launch_kv_append(const KvParams& kv, const RotateParams& q, int dtype, cudaStream_t s);

// cos and sin of every angle of positions first .. first + n - 1: turns[j] is pair j's turn a position, as a 64-bit fraction.
struct RotaryTableParams {
    float2* table;
    int64_t first, n;
    int half;
    float magnitude;
    uint64_t turns[kRotaryMaxDim / 2];
};
cudaError_t launch_rotary_table(const RotaryTableParams& p, cudaStream_t s);

}  // namespace ggq
