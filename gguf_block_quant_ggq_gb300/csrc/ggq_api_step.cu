// ggq_api_step.cu -- C ABI of what stands between the packed products of a decoding step
// (include/ggq.h): norms, the rotary table, adapters, log probabilities.
#include <cuda_runtime.h>

#include <algorithm>
#include <cmath>
#include <limits>

#include "../../include/ggq.h"
#include "ggq_adapt.cuh"
#include "ggq_ctx.h"
#include "ggq_logprobs.cuh"
#include "ggq_norm.cuh"
#include "ggq_rope.cuh"

using namespace ggq;

namespace {

constexpr int64_t kMaxRows = 1 << 24;  // tokens of a call

constexpr double kTwoPi = 6.283185307179586476925;

// Channel (as a number of pairs) that turns `turns` times within `len` positions.
double channel_of(double turns, double len, const ggq_rotary_spec& s) {
    return s.turn * std::log(len / (turns * kTwoPi)) / (2.0 * std::log(s.base));
}

}  // namespace

extern "C" {

ggq_status ggq_norm(ggq_ctx* c, const ggq_norm_args* a, void* stream) {
    DeviceScope scope;
    ggq_status s = check_ctx(c, scope);
    if (s != GGQ_OK) return s;
    if (!a) return fail(c, GGQ_ERR_INVALID_ARG, "norm: null arguments");
    const int dt = dtype_of(a->dtype);
    if (dt < 0) return fail(c, GGQ_ERR_UNSUPPORTED, "norm: element type %d; supported: F32, F16, BF16", a->dtype);
    if (a->gate && a->gate_act != GGQ_GATE_LINEAR && a->gate_act != GGQ_GATE_SIGMOID)
        return fail(c, GGQ_ERR_UNSUPPORTED, "norm: gate %d; supported: linear, sigmoid", a->gate_act);
    if (a->T < 0 || a->T > kMaxRows || a->H < 1 || a->H > kNormMaxWidth)
        return fail(c, GGQ_ERR_SHAPE, "norm: %lld tokens of %lld channels (1..%d)", static_cast<long long>(a->T),
                    static_cast<long long>(a->H), kNormMaxWidth);
    if (a->norms < 0 || a->norms > 3 || (a->gate && a->gate_channel != 0 && a->gate_channel != 1))
        return fail(c, GGQ_ERR_INVALID_ARG, "norm: norms=%d (0..3), gate_channel=%lld (0, 1)", a->norms,
                    static_cast<long long>(a->gate_channel));
    if (!std::isfinite(a->scale) || !std::isfinite(a->offset) || !(a->eps >= 0.0f) || !std::isfinite(a->eps))
        return fail(c, GGQ_ERR_INVALID_ARG, "norm: scale and offset must be finite, eps not negative");
    const bool before = (a->norms & 2) != 0;
    if (!before && (a->out || a->packed))
        return fail(c, GGQ_ERR_INVALID_ARG, "norm: out and packed are the norm of the total, which norms=%d leaves out", a->norms);
    int form = NORM_ROWS;
    if (a->packed) {
        form = a->packed_type == GGQ_TYPE_Q8_K ? NORM_Q8_K : a->packed_type == GGQ_TYPE_Q8_1 ? NORM_Q8_1
               : a->packed_type == GGQ_TYPE_Q8_0 ? NORM_Q8_0 : -1;
        if (form < 0) return fail(c, GGQ_ERR_UNSUPPORTED, "norm: packed type %d; supported: Q8_K, Q8_1, Q8_0", a->packed_type);
        if (a->H % (form == NORM_Q8_K ? 256 : 32))
            return fail(c, GGQ_ERR_SHAPE, "norm: H=%lld is no multiple of the block (Q8_K 256, Q8_1 and Q8_0 32)",
                        static_cast<long long>(a->H));
    }
    if (a->T == 0) return GGQ_OK;
    if (!a->x || (before ? !a->out && !a->packed : !a->total)) return fail(c, GGQ_ERR_INVALID_ARG, "norm: null x or no output");
    const int64_t size = dtype_bytes(dt);
    if (!multiple_of(a->x, size) || !multiple_of(a->residual, size) || !multiple_of(a->gate, size) || !multiple_of(a->total, size) ||
        !multiple_of(a->out, size) || !multiple_of(a->after, 4) || !multiple_of(a->before, 4))
        return fail(c, GGQ_ERR_INVALID_ARG, "norm: misaligned pointer");
    const auto apart = [&](const void* to, int64_t to_token, const void* from, int64_t from_token) {
        return to && to == from && a->T > 1 && to_token != from_token;
    };
    if (apart(a->total, a->total_token, a->x, a->x_token) || apart(a->total, a->total_token, a->residual, a->residual_token) ||
        apart(a->out, a->out_token, a->x, a->x_token) || apart(a->out, a->out_token, a->residual, a->residual_token))
        return fail(c, GGQ_ERR_INVALID_ARG, "norm: rows that are updated in place have one stride");
    if (a->total && (a->total == a->out || a->total == a->packed))
        return fail(c, GGQ_ERR_INVALID_ARG, "norm: total and its norm need a place each");
    NormParams p{};
    p.x = a->x;
    p.residual = a->residual;
    p.gate = a->gate;
    p.total = a->total;
    p.out = a->out;
    p.packed = static_cast<uint8_t*>(a->packed);
    p.after_w = a->norms & 1 ? a->after : nullptr;
    p.before_w = before ? a->before : nullptr;
    p.x_token = a->x_token;
    p.residual_token = a->residual_token;
    p.gate_token = a->gate_token;
    p.total_token = a->total_token;
    p.out_token = a->out_token;
    p.T = a->T;
    p.H = static_cast<int>(a->H);
    p.gate_channel = static_cast<int>(a->gate_channel);
    p.sigmoid = a->gate_act == GGQ_GATE_SIGMOID;
    p.after = a->norms & 1;
    p.before = before;
    p.form = form;
    p.scale = a->scale;
    p.eps = a->eps;
    p.offset = a->offset;
    p.inv_width = 1.0f / static_cast<float>(a->H);
    if (p.packed && (!multiple_of(p.packed, form == NORM_Q8_0 ? 2 : 4) || !norm_whole(p, dt)))
        return fail(c, GGQ_ERR_INVALID_ARG, "norm: packed rows need rows, weights and outputs that start at 16 bytes (pointers and strides)");
    const cudaError_t e = launch_norm(p, dt, static_cast<cudaStream_t>(stream));
    return e == cudaSuccess ? GGQ_OK : cuda_fail(c, e, "norm launch");
}

ggq_status ggq_rotary_table(ggq_ctx* c, const ggq_rotary_spec* r, int64_t first, int64_t n, float* table, void* stream) {
    DeviceScope scope;
    ggq_status s = check_ctx(c, scope);
    if (s != GGQ_OK) return s;
    if (!r) return fail(c, GGQ_ERR_INVALID_ARG, "rotary_table: null spec");
    if (r->turn < 2 || r->turn % 2 || r->turn > kRotaryMaxDim || first < 0 || n < 0 || first > (1ll << 31) || n > (1ll << 31) - first)
        return fail(c, GGQ_ERR_SHAPE, "rotary_table: %d channels (even, 2..%d), positions %lld + %lld (at most 2^31)", r->turn,
                    kRotaryMaxDim, static_cast<long long>(first), static_cast<long long>(n));
    if (!std::isfinite(r->base) || r->base <= 1.0 || !std::isfinite(r->factor) || r->factor < 1.0 || r->original_len < 0 ||
        !(std::abs(r->magnitude) <= std::numeric_limits<float>::max()))
        return fail(c, GGQ_ERR_INVALID_ARG, "rotary_table: base above 1, factor of at least 1, original_len not negative, a magnitude that is finite in fp32");
    const bool mixed = r->factor > 1.0 && r->original_len > 0;
    if (mixed && !(std::isfinite(r->beta_fast) && r->beta_slow > 0.0 && r->beta_fast >= r->beta_slow))
        return fail(c, GGQ_ERR_INVALID_ARG, "rotary_table: beta_fast at least beta_slow, both above 0");
    RotaryTableParams p{};
    p.half = r->turn / 2;
    double low = 0.0, high = 0.0;
    if (mixed) {
        low = std::max(std::floor(channel_of(r->beta_fast, static_cast<double>(r->original_len), *r)), 0.0);
        high = std::min(std::ceil(channel_of(r->beta_slow, static_cast<double>(r->original_len), *r)), r->turn - 1.0);
    }
    for (int j = 0; j < p.half; ++j) {
        double f = std::pow(r->base, -2.0 * j / r->turn);
        if (r->factors) {
            if (!(r->factors[j] > 0.0f) || !std::isfinite(r->factors[j]))
                return fail(c, GGQ_ERR_INVALID_ARG, "rotary_table: factor %d of the frequencies is not above 0", j);
            f /= r->factors[j];
        }
        if (mixed) {
            const double slow = std::min(std::max((j - low) / std::max(high - low, 0.001), 0.0), 1.0);
            f = f * (1.0 - slow) + f / r->factor * slow;
        } else {
            f /= r->factor;
        }
        const double turns = f / kTwoPi, part = turns - std::floor(turns);
        p.turns[j] = static_cast<uint64_t>(std::min(part * 0x1p64, 0x1.fffffffffffffp63));
    }
    if (n == 0) return GGQ_OK;
    if (!table) return fail(c, GGQ_ERR_INVALID_ARG, "rotary_table: null table");
    if (!multiple_of(table, 8)) return fail(c, GGQ_ERR_INVALID_ARG, "rotary_table: the table must be 8-byte aligned");
    p.table = reinterpret_cast<float2*>(table);
    p.first = first;
    p.n = n;
    p.magnitude = static_cast<float>(r->magnitude);
    const cudaError_t e = launch_rotary_table(p, static_cast<cudaStream_t>(stream));
    return e == cudaSuccess ? GGQ_OK : cuda_fail(c, e, "rotary_table launch");
}

ggq_status ggq_adapt(ggq_ctx* c, const ggq_adapters* b, const ggq_adapt_args* a, void* stream) {
    DeviceScope scope;
    ggq_status s = check_ctx(c, scope);
    if (s != GGQ_OK) return s;
    if (!b || !a) return fail(c, GGQ_ERR_INVALID_ARG, "adapt: null arguments");
    const int dt = dtype_of(a->dtype), bank = dtype_of(b->dtype);
    if (dt < 0) return fail(c, GGQ_ERR_UNSUPPORTED, "adapt: element type %d; supported: F32, F16, BF16", a->dtype);
    if (bank < 1) return fail(c, GGQ_ERR_UNSUPPORTED, "adapt: adapters of type %d; supported: F16, BF16", b->dtype);
    if (b->max_rank < 8 || b->max_rank > kAdaptMaxRank || b->max_rank % 8 || b->n < 1 || b->n > INT32_MAX || b->K < 8 || b->K % 8 ||
        b->K > (1 << 24) || b->N < 1 || b->N > (1 << 24))
        return fail(c, GGQ_ERR_SHAPE, "adapt: %lld adapters of rank %d (a multiple of 8, at most %d), %lld inputs (a multiple of 8), %lld outputs",
                    static_cast<long long>(b->n), b->max_rank, kAdaptMaxRank, static_cast<long long>(b->K), static_cast<long long>(b->N));
    if (a->T < 0 || a->T > kMaxRows || a->n_seqs < 0 || a->n_seqs > (1 << 20) || (!a->q_start && a->T != a->n_seqs))
        return fail(c, GGQ_ERR_SHAPE, "adapt: %lld rows of %lld sequences", static_cast<long long>(a->T), static_cast<long long>(a->n_seqs));
    if (a->T == 0 || a->n_seqs == 0) return GGQ_OK;
    if (!b->a || !b->b || !a->x || !a->y || !a->out || !a->ids) return fail(c, GGQ_ERR_INVALID_ARG, "adapt: null pointer");
    const int64_t size = dtype_bytes(dt);
    if (!multiple_of(b->a, 16) || !multiple_of(b->b, 16) || !multiple_of(b->ranks, 4) || !multiple_of(b->scales, 4) ||
        !multiple_of(a->ids, 4) || !multiple_of(a->q_start, 4) || !multiple_of(a->y, size) || !multiple_of(a->out, size))
        return fail(c, GGQ_ERR_INVALID_ARG, "adapt: banks must be 16-byte aligned, the others by their elements");
    if (!rows4(a->x, a->T, a->x_token, 1, 0, dt))
        return fail(c, GGQ_ERR_INVALID_ARG, "adapt: rows of x must start at multiples of 4 elements (pointer and stride)");
    if (a->out == a->y && a->T > 1 && a->out_token != a->y_token)
        return fail(c, GGQ_ERR_INVALID_ARG, "adapt: rows that are updated in place have one stride");
    if (a->out == a->x) return fail(c, GGQ_ERR_INVALID_ARG, "adapt: out must not be x, which every part of a row's outputs reads");
    AdaptParams p{};
    p.a = b->a;
    p.b = b->b;
    p.ranks = b->ranks;
    p.scales = b->scales;
    p.n = b->n;
    p.R = b->max_rank;
    p.K = static_cast<int>(b->K);
    p.N = b->N;
    p.x = a->x;
    p.y = a->y;
    p.out = a->out;
    p.x_token = a->x_token;
    p.y_token = a->y_token;
    p.out_token = a->out_token;
    p.ids = a->ids;
    p.q_start = a->q_start;
    p.T = a->T;
    p.seqs = a->n_seqs;
    p.bank = bank;
    p.err = &c->ctrl->err;
    const cudaError_t e = launch_adapt(p, dt, static_cast<cudaStream_t>(stream));
    return e == cudaSuccess ? GGQ_OK : cuda_fail(c, e, "adapt launch");
}

ggq_status ggq_logprobs(ggq_ctx* c, const ggq_logprobs_args* a, void* stream) {
    DeviceScope scope;
    ggq_status s = check_ctx(c, scope);
    if (s != GGQ_OK) return s;
    if (!a) return fail(c, GGQ_ERR_INVALID_ARG, "logprobs: null arguments");
    const int dt = dtype_of(a->dtype);
    if (dt < 0) return fail(c, GGQ_ERR_UNSUPPORTED, "logprobs: element type %d; supported: F32, F16, BF16", a->dtype);
    if (a->T < 0 || a->T > kMaxRows || a->V < 1 || a->V > (1 << 30) || a->top_k < 0 || a->top_k > kLogprobsMaxTop || a->top_k > a->V ||
        a->given < 0 || a->given > 65536)
        return fail(c, GGQ_ERR_SHAPE, "logprobs: %lld tokens of %lld logits, %lld given, top_k=%d (0..%d, at most the vocabulary)",
                    static_cast<long long>(a->T), static_cast<long long>(a->V), static_cast<long long>(a->given), a->top_k, kLogprobsMaxTop);
    if (!std::isfinite(a->scale) || a->scale <= 0.0f) return fail(c, GGQ_ERR_INVALID_ARG, "logprobs: scale must be finite and above 0");
    if (a->T == 0) return GGQ_OK;
    if (!a->logits || (a->given && (!a->tokens || !a->logprobs)) || (a->top_k && (!a->ids || !a->top)) ||
        (!a->given && !a->top_k && !a->entropy))
        return fail(c, GGQ_ERR_INVALID_ARG, "logprobs: null pointer, or nothing asked for");
    if (!multiple_of(a->logits, dtype_bytes(dt)) || !multiple_of(a->tokens, 4) || !multiple_of(a->logprobs, 4) ||
        !multiple_of(a->entropy, 4) || !multiple_of(a->ids, 4) || !multiple_of(a->top, 4))
        return fail(c, GGQ_ERR_INVALID_ARG, "logprobs: misaligned pointer");
    const LogprobsParams p{a->logits, a->row, a->T, static_cast<int>(a->V), a->tokens, static_cast<int>(a->given), a->logprobs, a->entropy,
                           a->top_k, a->ids, a->top, a->scale, &c->ctrl->err};
    const cudaError_t e = launch_logprobs(p, dt, static_cast<cudaStream_t>(stream));
    return e == cudaSuccess ? GGQ_OK : cuda_fail(c, e, "logprobs launch");
}

}  // extern "C"
