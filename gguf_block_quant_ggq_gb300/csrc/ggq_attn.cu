// ggq_attn.cu -- which kernel an attention call over the packed cache takes.
#include "ggq_attn.cuh"
#include "ggq_internal.h"

namespace ggq {

// The streaming kernel cuts all (8 or 16 query rows, kv head, key) work into equal
// shares over the SMs; the tile kernels give 64, 128 or 256 rows of a kv head to one
// CTA, which passes over its keys alone, at a time that hardly depends on how many of
// its rows are there.  So the tile kernels take a call when their waves, each `ratio`
// times a streaming item's time a key, cost less than the streaming items spread over
// the SMs.  `ratio` is measured (ns for 16 keys, of a tile and of an item on one SM):
//   fp32, 8-row items:      425 / 65 (64 channels), 750 / 115 (128), 1850 / 235 (256, 64-row tiles)
//   16 bits, 16-row items:  260 / 76,               340 / 129,       500 / 466
// and what an item and a tile cost beside their keys as keys: 320 and 128.  Both sides
// of the rule at 32 heads on 8 of 128 channels, 64 rows a kv head (us, tiles / stream):
//   fp32: 16 sequences of 4096 keys 205 / 221, 4 of 32768 1537 / 399
//   bf16: 16 of 4096 96 / 133, 16 of 512 24 / 45, 4 of 4096 92 / 50, 4 of 32768 623 / 220
// Over 560 calls of 16 to 512 rows the choice takes 1.01 times the better side's time.
static bool tiles_pay(const AttnParams& p, int nsm) {
    const double rows = static_cast<double>(p.max_q) * p.G, all = static_cast<double>(p.n_tokens) * p.G;
    const int item = p.dtype != 0 && rows > 8 ? 16 : 8;
    const int tile = p.dtype != 0 ? (p.D <= 128 ? 256 : 128) : p.D <= 128 ? 128 : 64;
    const double ratio = p.dtype != 0 ? (p.D <= 128 ? 3.0 : 1.2) : p.D <= 128 ? 6.5 : 8.0;
    const auto parts = [&](int of) {  // of all sequences and kv heads: few rows a sequence, or many of few
        const double each = static_cast<double>(p.n_seqs) * static_cast<double>((static_cast<int64_t>(rows) + of - 1) / of);
        const double most = all / of + static_cast<double>(p.n_seqs);
        return (each < most ? each : most) * p.Hkv;
    };
    double keys = p.max_len;
    if (p.window > 0 && static_cast<double>(p.window) + p.max_q < keys) keys = static_cast<double>(p.window) + p.max_q;
    const double waves = static_cast<double>((static_cast<int64_t>(parts(tile)) + nsm - 1) / nsm);
    const double seen = p.window > 0 ? keys : keys - 0.5 * (p.max_q < keys ? p.max_q : keys);  // by a tile, on average
    const double tiles = (waves * seen > keys ? waves * seen : keys) + 128.0 * waves;
    return ratio * tiles * nsm < parts(item) * (keys + 320.0);
}

cudaError_t launch_attention(const AttnParams& p, int nsm, cudaStream_t s) {
    const int64_t rows = static_cast<int64_t>(p.max_q) * p.G;
    const bool fits = rows <= 64ll * 65535 && p.n_seqs * p.Hkv <= INT32_MAX &&  // the tile kernels' grids
                      (p.dtype == 0 || p.cap <= kWideCap);
    if (fits && tiles_pay(p, nsm)) {
        if (p.dtype == 0) {
            if (p.D == 64) return launch_attn_promptf_64(p, s);
            if (p.D == 128) return launch_attn_promptf_128(p, s);
            return launch_attn_rows_256(p, s);
        }
        if (p.D == 64) return launch_attn_prompt_64(p, s);
        if (p.D == 128) return launch_attn_prompt_128(p, s);
        return launch_attn_prompt_256(p, s);
    }
    if (p.D == 64) return launch_attn_stream_64(p, nsm, s);
    if (p.D == 128) return launch_attn_stream_128(p, nsm, s);
    return launch_attn_stream_256(p, nsm, s);
}

}  // namespace ggq
