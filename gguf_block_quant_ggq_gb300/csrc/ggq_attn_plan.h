// ggq_attn_plan.h -- how the streaming attention kernel's CTAs divide and join their
// items (host and device; the tests walk it on the CPU).
//
// All items lie one behind the other in a list of N positions: an item of n units has
// kItemCost positions that stand for no unit (its queries, merge and output), then n.
// CTA c of C takes the positions [N c / C, N (c + 1) / C).  The units of an item that
// fall to one CTA are a piece; the pieces of an item belong to neighbouring CTAs.
#pragma once
#include <stdint.h>

namespace ggq {

constexpr int kAttnMaxCtas = 1024;

// What an item counts in the shares beside its units, measured on 64 ragged sequences
// of up to 4096 tokens (units of 32 tokens, 128 channels): 82 us at 0, 68 at 6, 63.6 at
// 12, 65 at 20.  Other units (16 tokens of 256 channels, 64 of 4-bit 64 channels) use the
// same count, not measured by itself.
constexpr int kItemCost = 12;

// Sixteen neighbouring pieces are joined by the last of them, then these results by
// the last of the groups, always in the order of the pieces.
constexpr int kJoin = 16;

// Arrival counters of the context: pieces of items' first groups and groups of items (by
// the item's first CTA, which begins no other shared item), pieces of the other groups
// (by the group's first CTA, whose share begins inside the item).  The first two and the
// last are apart: the CTA that an item's last group begins with may begin the next item.
constexpr int kAttnCounters = 3 * kAttnMaxCtas;

// The pieces of the item at position p0: CTAs c0 (where its units begin) .. c1.  Each is
// a partial result in its CTA's slot 0 if the CTA's share begins inside the item, else in
// slot 1 (c0's only).
struct AttnPieces {
    int c0, c1, slot0;
    __host__ __device__ __forceinline__ AttnPieces(int64_t p0, int span, int64_t N, int C) {
        c0 = static_cast<int>(((p0 + kItemCost + 1) * C - 1) / N);
        c1 = static_cast<int>(((p0 + span) * C - 1) / N);
        slot0 = N * c0 / C >= p0 ? 0 : 1;
    }
    __host__ __device__ __forceinline__ int slot(int c) const { return c == c0 ? slot0 : 0; }
    // first piece of the group that CTA c's piece belongs to, and the group's pieces
    __host__ __device__ __forceinline__ int group(int c) const { return c0 + (c - c0) / kJoin * kJoin; }
    __host__ __device__ __forceinline__ int group_pieces(int g) const { return g + kJoin - 1 < c1 ? kJoin : c1 - g + 1; }
    __host__ __device__ __forceinline__ int groups() const { return (c1 - c0) / kJoin + 1; }
    // counters: pieces of the group that begins with g, groups of the item
    __host__ __device__ __forceinline__ int piece_counter(int g) const { return g == c0 ? g : 2 * kAttnMaxCtas + g; }
    __host__ __device__ __forceinline__ int group_counter() const { return kAttnMaxCtas + c0; }
};

// The copies of a warp's ring that are on their way when it leaves its units early, for
// which it waits before its CTA's shared memory goes to another one.  A warp fills its
// places in turn and takes them in turn; the next one it would take is `slot`, whose copy
// completes the barrier phase of parity `phase` (the places before it: of the other
// parity).  All places hold or await a copy until the share's last one, which is noted.
constexpr int kMoreCopies = -1, kNoCopies = -2;
__host__ __device__ constexpr int attn_last_copy(int slot, uint32_t parity) { return 2 * slot + static_cast<int>(parity); }
template <typename WAIT>
__host__ __device__ __forceinline__ void attn_drain(int last, int places, int slot, uint32_t phase, WAIT wait) {
    const auto parity = [&](int at) { return at >= slot ? phase : phase ^ 1u; };
    int n = places;
    if (last != kMoreCopies) {
        const int at = last >> 1;
        if (last == kNoCopies || static_cast<uint32_t>(last & 1) != parity(at)) return;  // all taken
        n = (at >= slot ? at - slot : at - slot + places) + 1;
    }
    for (int k = 0, at = slot; k < n; ++k, at = at + 1 == places ? 0 : at + 1) wait(at, parity(at));
}

}  // namespace ggq
