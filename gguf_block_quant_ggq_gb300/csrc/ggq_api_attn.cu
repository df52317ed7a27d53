// ggq_api_attn.cu -- C ABI of the key/value cache, the attention over it and
// the expert router (include/ggq.h): argument checks and launches.
#include <cuda_runtime.h>

#include <algorithm>
#include <cmath>

#include "../../include/ggq.h"
#include "ggq_attn.cuh"
#include "ggq_ctx.h"
#include "ggq_kv.cuh"
#include "ggq_rope.cuh"
#include "ggq_route.cuh"

using namespace ggq;

namespace {

bool kv_type_ok(int t) { return t == GGQ_TYPE_Q8_0 || t == GGQ_TYPE_Q4_0; }

ggq_status cache_checks(ggq_ctx* c, const ggq_kv_cache* kv, const char* op) {
    if (!kv) return fail(c, GGQ_ERR_INVALID_ARG, "%s: null cache", op);
    if (!kv_type_ok(kv->k_type) || !kv_type_ok(kv->v_type))
        return fail(c, GGQ_ERR_UNSUPPORTED, "%s: cache types %d and %d; supported: Q8_0, Q4_0", op, kv->k_type, kv->v_type);
    if (kv->n_kv_heads < 1 || kv->n_kv_heads > 16384 || (kv->head_dim != 64 && kv->head_dim != 128 && kv->head_dim != 256) ||
        kv->page_size < 16 || kv->page_size % 16 || kv->n_pages < 1 || kv->n_pages > INT32_MAX / (kv->page_size / 16))
        return fail(c, GGQ_ERR_SHAPE,
                    "%s: %d kv heads of %d channels in %lld pages of %d tokens (head_dim 64, 128 or 256, pages of a "
                    "multiple of 16 tokens)",
                    op, kv->n_kv_heads, kv->head_dim, static_cast<long long>(kv->n_pages), kv->page_size);
    if (!kv->k || !kv->v) return fail(c, GGQ_ERR_INVALID_ARG, "%s: null cache pool", op);
    if (!aligned16(kv->k) || !aligned16(kv->v))
        return fail(c, GGQ_ERR_INVALID_ARG, "%s: cache pools must be 16-byte aligned", op);
    return GGQ_OK;
}

// A page's 16-token groups as a multiplier for division (exact or one too large).
uint32_t page_magic(int page_size) { return static_cast<uint32_t>((1ull << 32) / (page_size / 16) + 1); }

// Partial results of items that two or more CTAs share: two a CTA, for the widest heads
// (whose CTAs an SM and those of narrower ones the streaming kernel asserts to fit).
size_t attn_scratch(const ggq_ctx* c) {
    const size_t ctas = std::min(kAttnMaxCtas, kAttnWideCtas * c->nsm);
    return align_up(2 * ctas * attn_part_floats(256) * sizeof(float));
}

ggq_status kv_params(ggq_ctx* c, const ggq_kv_cache* kv, int dtype, const void* k, int64_t k_token, int64_t k_head,
                     const void* v, int64_t v_token, int64_t v_head, const int64_t* slots, int64_t T, const char* op,
                     KvParams* p, int* dt) {
    ggq_status s = cache_checks(c, kv, op);
    if (s != GGQ_OK) return s;
    *dt = dtype_of(dtype);
    if (*dt < 0) return fail(c, GGQ_ERR_UNSUPPORTED, "%s: element type %d; supported: F32, F16, BF16", op, dtype);
    if (T < 0 || T > INT32_MAX) return fail(c, GGQ_ERR_SHAPE, "%s: T=%lld", op, static_cast<long long>(T));
    if (T == 0) return GGQ_OK;
    if (!k || !v || !slots) return fail(c, GGQ_ERR_INVALID_ARG, "%s: null pointer", op);
    if (reinterpret_cast<uintptr_t>(slots) & 7)
        return fail(c, GGQ_ERR_INVALID_ARG, "%s: slots must be 8-byte aligned", op);
    if (!rows4(k, T, k_token, kv->n_kv_heads, k_head, *dt) || !rows4(v, T, v_token, kv->n_kv_heads, v_head, *dt))
        return fail(c, GGQ_ERR_INVALID_ARG, "%s: rows must start at multiples of 4 elements (pointers and strides)", op);
    *p = KvParams{{static_cast<uint8_t*>(kv->k), kv->k_type == GGQ_TYPE_Q4_0},
                  {static_cast<uint8_t*>(kv->v), kv->v_type == GGQ_TYPE_Q4_0},
                  kv->n_kv_heads, kv->head_dim, kv->page_size, page_magic(kv->page_size), 1, kv->n_pages * kv->page_size,
                  slots, T, k, v, k_token, k_head, v_token, v_head, &c->ctrl->err};
    return GGQ_OK;
}

// The rotation of heads of D channels; positions are the caller's to set.
ggq_status rotary_params(ggq_ctx* c, const ggq_rotary* r, int D, const int32_t* positions, const char* op, Rotary* out) {
    if (!r) return fail(c, GGQ_ERR_INVALID_ARG, "%s: null rotary", op);
    if (r->layout != GGQ_ROTARY_HALF && r->layout != GGQ_ROTARY_PAIRS)
        return fail(c, GGQ_ERR_UNSUPPORTED, "%s: rotary layout %d; supported: halves, pairs", op, r->layout);
    if (D < 1 || D > kRotaryMaxDim || r->turn < 2 || r->turn % 2 || r->first < 0 || r->turn > D || r->first > D - r->turn ||
        r->n_positions < 1)
        return fail(c, GGQ_ERR_SHAPE, "%s: %d channels from %d on turned in heads of %d (at most %d), %lld positions", op, r->turn,
                    r->first, D, kRotaryMaxDim, static_cast<long long>(r->n_positions));
    if (!r->table || !positions) return fail(c, GGQ_ERR_INVALID_ARG, "%s: null table or positions", op);
    if (!multiple_of(r->table, 8) || !multiple_of(positions, 4))
        return fail(c, GGQ_ERR_INVALID_ARG, "%s: the table must be 8-byte and positions 4-byte aligned", op);
    *out = Rotary{reinterpret_cast<const float2*>(r->table), r->n_positions, positions, r->turn / 2, r->first,
                  r->layout == GGQ_ROTARY_PAIRS, 0};
    return GGQ_OK;
}

ggq_status rotate_params(ggq_ctx* c, int dt, int n_heads, int D, const void* x, int64_t x_token, int64_t x_head, void* out,
                         int64_t out_token, int64_t out_head, int64_t T, const char* op, RotateParams* p) {
    if (n_heads < 0 || n_heads > 16384) return fail(c, GGQ_ERR_SHAPE, "%s: %d heads", op, n_heads);
    if (n_heads > 0 && (!x || !out)) return fail(c, GGQ_ERR_INVALID_ARG, "%s: null pointer", op);
    if (!multiple_of(x, dtype_bytes(dt)) || !multiple_of(out, dtype_bytes(dt)))
        return fail(c, GGQ_ERR_INVALID_ARG, "%s: misaligned heads", op);
    p->x = x;
    p->out = out;
    p->x_token = x_token;
    p->x_head = x_head;
    p->out_token = out_token;
    p->out_head = out_head;
    p->T = T;
    p->H = n_heads;
    p->D = D;
    p->in_place = x == out;
    p->err = &c->ctrl->err;
    if (p->in_place && ((T > 1 && x_token != out_token) || (n_heads > 1 && x_head != out_head)))
        return fail(c, GGQ_ERR_INVALID_ARG, "%s: heads turned in place have one stride", op);
    return GGQ_OK;
}

}  // namespace

extern "C" {

size_t ggq_kv_page_bytes(int type, int n_kv_heads, int head_dim, int page_size) {
    if (!kv_type_ok(type) || n_kv_heads < 1 || n_kv_heads > 16384 ||
        (head_dim != 64 && head_dim != 128 && head_dim != 256) || page_size < 16 || page_size % 16)
        return 0;
    return static_cast<size_t>(n_kv_heads) * (page_size / 16) * kv_blob_bytes(type == GGQ_TYPE_Q4_0, head_dim);
}

ggq_status ggq_kv_store(ggq_ctx* c, const ggq_kv_cache* kv, int dtype, const void* k, int64_t k_token, int64_t k_head,
                        const void* v, int64_t v_token, int64_t v_head, const int64_t* slots, int64_t T, void* stream) {
    DeviceScope scope;
    ggq_status s = check_ctx(c, scope);
    if (s != GGQ_OK) return s;
    KvParams p{};
    int dt = -1;
    s = kv_params(c, kv, dtype, k, k_token, k_head, v, v_token, v_head, slots, T, "kv_store", &p, &dt);
    if (s != GGQ_OK) return s;
    const cudaError_t e = launch_kv_store(p, dt, static_cast<cudaStream_t>(stream));
    return e == cudaSuccess ? GGQ_OK : cuda_fail(c, e, "kv_store launch");
}

ggq_status ggq_rotate(ggq_ctx* c, const ggq_rotary* r, const ggq_rotate_args* a, void* stream) {
    DeviceScope scope;
    ggq_status s = check_ctx(c, scope);
    if (s != GGQ_OK) return s;
    if (!a) return fail(c, GGQ_ERR_INVALID_ARG, "rotate: null arguments");
    const int dt = dtype_of(a->dtype);
    if (dt < 0) return fail(c, GGQ_ERR_UNSUPPORTED, "rotate: element type %d; supported: F32, F16, BF16", a->dtype);
    if (a->T < 0 || a->T > INT32_MAX) return fail(c, GGQ_ERR_SHAPE, "rotate: T=%lld", static_cast<long long>(a->T));
    if (a->T == 0 || a->n_heads == 0) return GGQ_OK;
    RotateParams p{};
    s = rotary_params(c, r, a->D, a->positions, "rotate", &p.r);
    if (s == GGQ_OK)
        s = rotate_params(c, dt, a->n_heads, a->D, a->x, a->x_token, a->x_head, a->out, a->out_token, a->out_head, a->T, "rotate", &p);
    if (s != GGQ_OK) return s;
    const cudaError_t e = launch_rotate(p, dt, static_cast<cudaStream_t>(stream));
    return e == cudaSuccess ? GGQ_OK : cuda_fail(c, e, "rotate launch");
}

ggq_status ggq_kv_append(ggq_ctx* c, const ggq_kv_cache* kv, const ggq_rotary* r, const ggq_append_args* a, void* stream) {
    DeviceScope scope;
    ggq_status s = check_ctx(c, scope);
    if (s != GGQ_OK) return s;
    if (!a) return fail(c, GGQ_ERR_INVALID_ARG, "kv_append: null arguments");
    KvParams p{};
    int dt = -1;
    s = kv_params(c, kv, a->dtype, a->k, a->k_token, a->k_head, a->v, a->v_token, a->v_head, a->slots, a->T, "kv_append", &p, &dt);
    if (s != GGQ_OK || a->T == 0) return s;
    RotateParams rot{};
    s = rotary_params(c, r, kv->head_dim, a->positions, "kv_append", &rot.r);
    if (s == GGQ_OK)
        s = rotate_params(c, dt, a->n_heads, kv->head_dim, a->q, a->q_token, a->q_head, a->q_out, a->q_out_token, a->q_out_head, a->T,
                          "kv_append", &rot);
    if (s != GGQ_OK) return s;
    rot.slots = a->slots;
    const cudaError_t e = launch_kv_append(p, rot, dt, static_cast<cudaStream_t>(stream));
    return e == cudaSuccess ? GGQ_OK : cuda_fail(c, e, "kv_append launch");
}

ggq_status ggq_kv_load(ggq_ctx* c, const ggq_kv_cache* kv, int dtype, const int64_t* slots, int64_t T, void* k,
                       int64_t k_token, int64_t k_head, void* v, int64_t v_token, int64_t v_head, void* stream) {
    DeviceScope scope;
    ggq_status s = check_ctx(c, scope);
    if (s != GGQ_OK) return s;
    KvParams p{};
    int dt = -1;
    s = kv_params(c, kv, dtype, k, k_token, k_head, v, v_token, v_head, slots, T, "kv_load", &p, &dt);
    if (s != GGQ_OK) return s;
    const cudaError_t e = launch_kv_load(p, dt, static_cast<cudaStream_t>(stream));
    return e == cudaSuccess ? GGQ_OK : cuda_fail(c, e, "kv_load launch");
}

ggq_status ggq_attention(ggq_ctx* c, const ggq_kv_cache* kv, const ggq_attn* a, void* stream) {
    DeviceScope scope;
    ggq_status s = check_ctx(c, scope);
    if (s != GGQ_OK) return s;
    s = cache_checks(c, kv, "attention");
    if (s != GGQ_OK) return s;
    if (!a) return fail(c, GGQ_ERR_INVALID_ARG, "attention: null arguments");
    const int dt = dtype_of(a->dtype);
    if (dt < 0) return fail(c, GGQ_ERR_UNSUPPORTED, "attention: element type %d; supported: F32, F16, BF16", a->dtype);
    if (a->n_heads < 1 || a->n_heads % kv->n_kv_heads || a->n_heads > 16384)
        return fail(c, GGQ_ERR_SHAPE, "attention: %d query heads on %d kv heads", a->n_heads, kv->n_kv_heads);
    if (a->n_tokens < 0 || a->n_tokens > kAttnMaxRows || a->n_seqs < 0 || a->n_seqs > (1 << 20) ||
        (!a->q_start && a->n_tokens != a->n_seqs) || a->table_stride < 0 || a->max_len < 0 || a->max_q < 0)
        return fail(c, GGQ_ERR_SHAPE, "attention: %lld rows of %lld sequences, max_q=%lld, max_len=%lld",
                    static_cast<long long>(a->n_tokens), static_cast<long long>(a->n_seqs),
                    static_cast<long long>(a->max_q), static_cast<long long>(a->max_len));
    if (!std::isfinite(a->scale) || !std::isfinite(a->cap))
        return fail(c, GGQ_ERR_INVALID_ARG, "attention: scale and cap must be finite");
    if (a->n_tokens == 0 || a->n_seqs == 0) return GGQ_OK;
    if (!a->q || !a->out || !a->lens || (!a->table && a->table_stride > 0))
        return fail(c, GGQ_ERR_INVALID_ARG, "attention: null pointer");
    if (!rows4(a->q, a->n_tokens, a->q_token, a->n_heads, a->q_head, dt) ||
        !rows4(a->out, a->n_tokens, a->out_token, a->n_heads, a->out_head, dt))
        return fail(c, GGQ_ERR_INVALID_ARG, "attention: rows must start at multiples of 4 elements (pointers and strides)");
    if ((reinterpret_cast<uintptr_t>(a->lens) | reinterpret_cast<uintptr_t>(a->q_start) |
         reinterpret_cast<uintptr_t>(a->table) | reinterpret_cast<uintptr_t>(a->slopes)) & 3)
        return fail(c, GGQ_ERR_INVALID_ARG, "attention: lens, q_start, table and slopes must be 4-byte aligned");
    int64_t room = a->table_stride * kv->page_size;  // what a table row can name
    if (a->max_len > 0 && a->max_len < room) room = a->max_len;
    if (room > kAttnMaxLen) room = kAttnMaxLen;
    AttnParams p{};
    p.q = a->q;
    p.out = a->out;
    p.q_token = a->q_token;
    p.q_head = a->q_head;
    p.out_token = a->out_token;
    p.out_head = a->out_head;
    p.k = static_cast<const uint8_t*>(kv->k);
    p.v = static_cast<const uint8_t*>(kv->v);
    p.table = a->table;
    p.lens = a->lens;
    p.q_start = a->q_start;
    p.slopes = a->slopes;
    p.table_stride = a->table_stride;
    p.n_pages = kv->n_pages;
    p.n_tokens = a->n_tokens;
    p.n_seqs = a->n_seqs;
    p.dtype = dt;
    p.H = a->n_heads;
    p.Hkv = kv->n_kv_heads;
    p.G = a->n_heads / kv->n_kv_heads;
    p.D = kv->head_dim;
    p.page = kv->page_size;
    p.page_magic = page_magic(kv->page_size);
    p.k_q4 = kv->k_type == GGQ_TYPE_Q4_0;
    p.v_q4 = kv->v_type == GGQ_TYPE_Q4_0;
    p.max_q = static_cast<int>(!a->q_start ? 1 : a->max_q < a->n_tokens ? a->max_q : a->n_tokens);
    p.max_len = static_cast<int>(room);
    // a window of all that a sequence can hold is none: positions minus windows stay in range, the rows
    // before the first key (position -1 and below) included
    p.window = static_cast<int>(a->window <= 0 || a->window >= room ? 0 : a->window);
    p.scale = a->scale;
    // beyond 2^+-100 the quotients by the cap leave fp32, and a larger (smaller) cap changes no result
    p.cap = a->cap > 0.0f ? std::min(std::max(a->cap, 0x1p-100f), 0x1p100f) : 0.0f;
    p.err = &c->ctrl->err;
    s = need_scratch(c, attn_scratch(c));
    if (s != GGQ_OK) return s;
    p.min_share = 4;  // one sequence of 777 tokens, 8 kv heads: 11.8 us; 13.6 at 2, 12.6 at 8, 15.1 at 16
    p.parts = reinterpret_cast<float*>(c->pool);
    p.pieces = c->ctrl->attn_pieces;
    const cudaError_t e = launch_attention(p, c->nsm, static_cast<cudaStream_t>(stream));
    return e == cudaSuccess ? GGQ_OK : cuda_fail(c, e, "attention launch");
}

ggq_status ggq_reserve_attention(ggq_ctx* c, void* stream) {
    DeviceScope scope;
    ggq_status s = check_ctx(c, scope);
    return s == GGQ_OK ? grow_pool(c, attn_scratch(c), stream) : s;
}

ggq_status ggq_moe_route(ggq_ctx* c, const ggq_router* r, int dtype, const void* logits, int64_t T, int64_t E,
                         int32_t* ids, float* weights, void* stream) {
    DeviceScope scope;
    ggq_status s = check_ctx(c, scope);
    if (s != GGQ_OK) return s;
    if (!r) return fail(c, GGQ_ERR_INVALID_ARG, "moe_route: null router");
    const int dt = dtype_of(dtype);
    if (dt < 0) return fail(c, GGQ_ERR_UNSUPPORTED, "moe_route: element type %d; supported: F32, F16, BF16", dtype);
    if (r->scoring != GGQ_SCORE_SOFTMAX && r->scoring != GGQ_SCORE_SIGMOID)
        return fail(c, GGQ_ERR_UNSUPPORTED, "moe_route: scoring %d; supported: softmax, sigmoid", r->scoring);
    if (T < 0 || T > INT32_MAX || E < 1 || E > kRouteMaxExperts || r->top_k < 1 || r->top_k > kRouteMaxTopK || r->top_k > E)
        return fail(c, GGQ_ERR_SHAPE, "moe_route: T=%lld, E=%lld (1..%d), top_k=%d (1..%d, at most E)",
                    static_cast<long long>(T), static_cast<long long>(E), kRouteMaxExperts, r->top_k, kRouteMaxTopK);
    if (r->n_groups < 1 || r->n_groups > kRouteMaxGroups || E % r->n_groups || r->top_groups < 1 ||
        r->top_groups > r->n_groups || r->top_k > r->top_groups * (E / r->n_groups) || r->group_best < 1 || r->group_best > 2)
        return fail(c, GGQ_ERR_SHAPE,
                    "moe_route: %d groups (1..%d, dividing E=%lld), %d of them open for top_k=%d, group_best=%d (1 or 2)",
                    r->n_groups, kRouteMaxGroups, static_cast<long long>(E), r->top_groups, r->top_k, r->group_best);
    if (!std::isfinite(r->scale)) return fail(c, GGQ_ERR_INVALID_ARG, "moe_route: scale must be finite");
    if (T == 0) return GGQ_OK;
    if (!logits || !ids || !weights) return fail(c, GGQ_ERR_INVALID_ARG, "moe_route: null pointer");
    if ((reinterpret_cast<uintptr_t>(logits) % static_cast<uintptr_t>(dtype_bytes(dt))) ||
        ((reinterpret_cast<uintptr_t>(ids) | reinterpret_cast<uintptr_t>(weights) | reinterpret_cast<uintptr_t>(r->bias)) & 3))
        return fail(c, GGQ_ERR_INVALID_ARG, "moe_route: misaligned pointer");
    const RouteParams p{logits, r->bias, T, static_cast<int>(E), r->top_k, r->n_groups, r->top_groups, r->group_best,
                        r->scoring == GGQ_SCORE_SIGMOID, r->normalize != 0, 0, r->scale, ids, weights};
    const cudaError_t e = launch_route(p, dt, static_cast<cudaStream_t>(stream));
    return e == cudaSuccess ? GGQ_OK : cuda_fail(c, e, "moe_route launch");
}

}  // extern "C"
