"""Shares, pieces and joins of the streaming attention kernel (csrc/ggq_attn_plan.h), on CPU.

A host program compiled with nvcc against the library's own header lays the items of
random batches (few sequences of very different lengths among them) into the list of
positions, gives every CTA its share, and checks from the definition alone: the CTAs that
hold units of an item are the ones that the plan names, no two pieces of shared items lie
in one place of a CTA, every group of pieces and every item that is joined in groups has
an arrival counter of its own, and the places whose results a join reads are the ones
that were written.  The counters' rule of one array for all groups, by the group's first
CTA alone, is counted beside it: the batches have to reach the case where it fails.

A second program gives up a warp's ring of copies at every point of its work, with the copies
landing late or not at all until then, and checks that the drain waits for each that is on its
way, and for nothing else.
"""
import os
import shutil
import subprocess

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
CSRC = os.path.join(ROOT, "gguf_block_quant_ggq_gb300", "csrc")

PROGRAM = r"""
#include <algorithm>
#include <cmath>
#include <cstdio>
#include <map>
#include <random>
#include <set>
#include <vector>
#include "ggq_attn_plan.h"
using namespace ggq;

static long violations = 0, shared = 0, grouped = 0, meeting = 0;
#define CHECK(c, ...) do { if (!(c)) { if (violations++ < 20) { std::printf(__VA_ARGS__); std::printf("\n"); } } } while (0)

// The items' units, in order; C CTAs.
static void walk(const std::vector<int>& units, int C) {
    int64_t N = 0;
    for (int n : units) N += n + kItemCost;
    std::set<int> counters;                      // of groups of pieces and of items' groups
    std::map<int, int> alone;                    // uses of a group's first CTA
    std::set<std::pair<int, int>> places;        // (CTA, slot)
    int64_t p0 = 0;
    for (size_t i = 0; i < units.size(); p0 += units[i] + kItemCost, ++i) {
        std::vector<int> holders;  // CTAs with units of the item
        std::vector<int> slots;
        const int64_t u0 = p0 + kItemCost, u1 = u0 + units[i];
        for (int c = static_cast<int>(std::max<int64_t>(0, u0 * C / N - 2)); c < C && N * c / C < u1; ++c) {
            const int64_t lo = N * c / C, hi = N * (c + 1) / C;
            if (std::max(lo, u0) < std::min(hi, u1)) {
                holders.push_back(c);
                slots.push_back(lo >= p0 ? 0 : 1);
            }
        }
        const AttnPieces q(p0, units[i] + kItemCost, N, C);
        CHECK(!holders.empty() && q.c0 == holders.front() && q.c1 == holders.back() &&
              q.c1 - q.c0 + 1 == static_cast<int>(holders.size()), "item %zu: CTAs %d..%d", i, q.c0, q.c1);
        if (holders.size() < 2) continue;
        ++shared;
        std::map<int, int> arrivals;  // pieces of each group
        for (size_t k = 0; k < holders.size(); ++k) {
            const int c = holders[k];
            CHECK(q.slot(c) == slots[k], "item %zu CTA %d: slot %d", i, c, q.slot(c));
            CHECK(places.insert({c, q.slot(c)}).second, "item %zu CTA %d: place taken", i, c);
            ++arrivals[q.group(c)];
        }
        CHECK(q.groups() == static_cast<int>(arrivals.size()), "item %zu: %d groups", i, q.groups());
        for (const auto& [g, n] : arrivals) {
            CHECK(g >= q.c0 && g <= q.c1 && q.group_pieces(g) == n && n <= kJoin, "item %zu group %d", i, g);
            const int at = q.piece_counter(g);
            CHECK(at >= 0 && at < kAttnCounters && counters.insert(at).second, "item %zu: counter %d of two groups", i, at);
            if (alone[g]++) ++meeting;
        }
        if (q.groups() > 1) {
            ++grouped;
            const int at = q.group_counter();
            CHECK(at >= 0 && at < kAttnCounters && counters.insert(at).second, "item %zu: counter %d of two", i, at);
        }
    }
}

static void batch(const std::vector<int>& lens, int heads, int tiles, int unit, int ctas) {
    std::vector<int> units;
    int64_t N = 0;
    for (int len : lens)
        for (int k = 0; k < heads * tiles; ++k) {
            units.push_back((len + unit - 1) / unit);
            N += units.back() + kItemCost;
        }
    walk(units, static_cast<int>(std::min<int64_t>((N + 3) / 4, ctas)));
}

int main() {
    // batches of 8 kv heads and units of 32 tokens whose heads one counter array loses
    batch({38421, 6670}, 8, 1, 32, 304);
    batch({96394, 1557, 13709}, 8, 1, 32, 304);
    batch({1094, 5198, 50458, 1056}, 8, 1, 32, 304);
    std::printf("known %ld\n", meeting);
    std::mt19937 rng(7);
    const auto log_uniform = [&](double lo, double hi) {
        return static_cast<int>(std::exp(std::uniform_real_distribution<>(std::log(lo), std::log(hi))(rng)));
    };
    for (int i = 0; i < 6000; ++i) {
        const int units[] = {16, 32, 64}, all_ctas[] = {152, 304, 456, 1024};
        std::vector<int> lens(1 + rng() % 12);
        for (int& x : lens) x = log_uniform(1, 131072);
        batch(lens, 1 + rng() % 16, rng() % 4 ? 1 : 1 + rng() % 5, units[rng() % 3], all_ctas[rng() % 4]);
    }
    std::printf("shared %ld grouped %ld meeting %ld violations %ld\n", shared, grouped, meeting, violations);
    return violations == 0 ? 0 : 1;
}
"""

RING = r"""
#include <cstdio>
#include <random>
#include "ggq_attn_plan.h"
using namespace ggq;

// A barrier of one arrival and its copy's bytes: `done` phases are over.
struct Barrier {
    int issued = 0, done = 0;
    bool test(uint32_t parity) const { return (static_cast<uint32_t>(done) & 1u) != parity; }  // the phase of that parity is over
};

int main() {
    std::mt19937 rng(3);
    long waits = 0, violations = 0;
    for (int round = 0; round < 20000; ++round) {
        const int S = 2 + rng() % 5, units = rng() % 20, leave = rng() % (units + 1);
        Barrier bars[6];
        int fetched = 0, last = units ? kMoreCopies : kNoCopies;
        const auto fetch = [&](int at, uint32_t parity) {  // as the kernel's: one unit into a place whose last copy is over
            if (fetched >= units) return;
            ++fetched;
            if (bars[at].issued != bars[at].done) ++violations;
            ++bars[at].issued;
            if (fetched == units) last = attn_last_copy(at, parity);
        };
        for (int i = 0; i < S; ++i) fetch(i, 0u);
        int slot = 0;
        uint32_t phase = 0;
        for (int u = 0; u < leave; ++u) {
            const int at = slot;
            bars[at].done = bars[at].issued;  // the copy lands
            if (!bars[at].test(phase)) ++violations;
            fetch(at, phase ^ 1u);
            if (++slot == S) slot = 0, phase ^= 1u;
        }
        for (Barrier& b : bars)  // some of the others have landed, some are on their way
            if (rng() % 2) b.done = b.issued;
        attn_drain(last, S, slot, phase, [&](int at, uint32_t parity) {
            if (at < 0 || at >= S || bars[at].issued == 0) ++violations;
            const bool pending = bars[at].issued != bars[at].done;
            if (bars[at].test(parity) == pending) ++violations;  // a copy on its way is waited for, no other one
            bars[at].done = bars[at].issued;
            if (!bars[at].test(parity)) ++violations;            // and the wait ends with it
            ++waits;
        });
        for (const Barrier& b : bars)
            if (b.issued != b.done) ++violations;
    }
    std::printf("waits %ld violations %ld\n", waits, violations);
    return violations == 0 ? 0 : 1;
}
"""


def _nvcc():
    for cand in (shutil.which("nvcc"), "/usr/local/cuda/bin/nvcc"):
        if cand and os.path.exists(cand):
            return cand
    return None


def run(program, tmp_path):
    nvcc = _nvcc()
    if nvcc is None:
        pytest.skip("nvcc not available")
    src = tmp_path / "attn_plan_check.cu"
    src.write_text(program)
    exe = tmp_path / "attn_plan_check"
    r = subprocess.run([nvcc, "-std=c++17", "-O1", "-gencode", "arch=compute_103a,code=sm_103a", "-I", CSRC,
                        str(src), "-o", str(exe)], capture_output=True, text=True, timeout=600)
    assert r.returncode == 0, r.stderr[-3000:]
    r = subprocess.run([str(exe)], capture_output=True, text=True, timeout=600)
    assert r.returncode == 0, r.stdout[-3000:]
    return r.stdout


def test_every_group_of_pieces_has_a_counter_and_a_place(tmp_path):
    known, rest = run(PROGRAM, tmp_path).splitlines()
    assert int(known.split()[1]) >= 3  # the named batches bring two groups to one CTA
    assert int(rest.split()[5]) >= 100 and rest.endswith("violations 0")


def test_a_ring_that_gives_up_waits_for_its_copies(tmp_path):
    out = run(RING, tmp_path).split()
    assert int(out[1]) > 1000 and out[2:] == ["violations", "0"]
