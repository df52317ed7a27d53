// ggq_ctx.h -- the context behind the C ABI and the helpers every entry point
// uses: errors, scratch, the device of a call (host only, not part of the ABI).
#pragma once
#include <cuda_runtime.h>

#include <cstdarg>
#include <cstdio>
#include <string>
#include <vector>

#include "../../include/ggq.h"
#include "ggq_attn_plan.h"

namespace ggq {

constexpr size_t kAlign = 256;

inline size_t align_up(size_t v, size_t a = kAlign) { return (v + a - 1) / a * a; }

// Layout of the control block (allocated once at create).
struct Ctrl {
    int err;
    int pad[63];
    int attn_pieces[kAttnCounters];  // attention: arrived pieces and groups of pieces of shared items, zero between calls
};

}  // namespace ggq

struct ggq_ctx {
    int device = 0;
    int nsm = 0;
    uint8_t* pool = nullptr;
    size_t pool_bytes = 0;
    std::vector<void*> retired;
    ggq::Ctrl* ctrl = nullptr;
    int static_weights = 0;  // weights never written while calls are in flight
    int direct_max = 32;     // largest token count of the direct MoE route (calls of <= 4 tokens above 4)
    unsigned long long* tel_pairs = nullptr;  // expert-load telemetry (caller's device buffers)
    unsigned long long* tel_calls = nullptr;
    int64_t tel_experts = 0;
    std::string err;
};

namespace ggq {

inline bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15) == 0; }

inline ggq_status fail(ggq_ctx* c, ggq_status s, const char* fmt, ...) {
    char buf[512];
    va_list ap;
    va_start(ap, fmt);
    vsnprintf(buf, sizeof buf, fmt, ap);
    va_end(ap);
    if (c) c->err = buf;
    return s;
}

inline ggq_status cuda_fail(ggq_ctx* c, cudaError_t e, const char* what) {
    return fail(c, GGQ_ERR_CUDA, "%s: %s", what, cudaGetErrorString(e));
}

inline ggq_status need_scratch(ggq_ctx* c, size_t bytes) {
    if (bytes <= c->pool_bytes) return GGQ_OK;
    return fail(c, GGQ_ERR_CAPACITY, "call needs %zu scratch bytes but the pool holds %zu: call ggq_reserve first",
                bytes, c->pool_bytes);
}

// The grow-only pool: a larger one replaces it, the old one lives until ggq_destroy.
inline ggq_status grow_pool(ggq_ctx* c, size_t need, void* stream) {
    if (need <= c->pool_bytes) return GGQ_OK;
    cudaStreamCaptureStatus cs = cudaStreamCaptureStatusNone;
    cudaError_t e = cudaStreamIsCapturing(static_cast<cudaStream_t>(stream), &cs);
    if (e != cudaSuccess) return cuda_fail(c, e, "reserve: cudaStreamIsCapturing");
    if (cs != cudaStreamCaptureStatusNone)
        return fail(c, GGQ_ERR_CAPTURE_ALLOC, "reserve: pool must grow to %zu bytes while the stream is capturing",
                    need);
    void* p = nullptr;
    e = cudaMalloc(&p, need);
    if (e != cudaSuccess) return cuda_fail(c, e, "reserve: cudaMalloc");
    if (c->pool) c->retired.push_back(c->pool);  // work in flight may still use it
    c->pool = static_cast<uint8_t*>(p);
    c->pool_bytes = need;
    return GGQ_OK;
}

// Makes the context's device current for one call and puts the caller's
// device back when the call returns.
struct DeviceScope {
    int prev = -1;
    ~DeviceScope() {
        if (prev >= 0) cudaSetDevice(prev);
    }
};

inline ggq_status check_ctx(ggq_ctx* c, DeviceScope& scope) {
    if (!c) return GGQ_ERR_INVALID_ARG;
    int cur = -1;
    cudaError_t e = cudaGetDevice(&cur);
    if (e != cudaSuccess) return cuda_fail(c, e, "cudaGetDevice");
    if (cur != c->device) {
        e = cudaSetDevice(c->device);
        if (e != cudaSuccess) return cuda_fail(c, e, "cudaSetDevice");
        scope.prev = cur;
    }
    return GGQ_OK;
}

}  // namespace ggq
