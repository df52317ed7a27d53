"""ggq_moe_route against the definition in 64 bits: the chosen experts exactly
(choices that differ by less than an fp32 rounding aside), the weights within a
few fp32 roundings, ties, NaN, infinities, groups, and the refusals; and a routed
expert layer fed by it against the layer that routes by itself."""
import math

import pytest

import ggq_synth as syn
from tests.gpu_util import to_dev

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

import gguf_block_quant_ggq_gb300 as ggq  # noqa: E402

DTYPES = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}


@pytest.fixture(scope="module")
def ctx():
    assert torch.cuda.is_available(), "GPU tests need a CUDA device"
    from gguf_block_quant_ggq_gb300 import _build
    _build.build()
    c = ggq.Context(0)
    yield c
    c.close()


def reference(logits, k, scoring, bias, groups, top, best, normalize, scale):
    """(ids, weights, choice margin of each rank) of one row, in Python floats."""
    x = [float(v) for v in logits]
    real = [v for v in x if v == v]
    if scoring == "softmax":
        m = max(real, default=-math.inf)
        e = [0.0 if v != v or m == -math.inf else 1.0 if v == m else math.exp(v - m) for v in x]
        total = sum(e)
        score = [v / total if total else 0.0 for v in e]
    else:
        score = [0.0 if v != v else 0.0 if v == -math.inf else 1.0 / (1.0 + math.exp(-max(v, -700.0))) for v in x]
    if bias is not None:
        choice = [s + float(b) for s, b in zip(score, bias)]
    else:
        choice = list(score) if scoring == "sigmoid" else list(x)
    choice = [(-math.inf, 1) if v != v else (c, 0) for v, c in zip(x, choice)]  # NaN after -inf
    key = lambda i: (-choice[i][0], choice[i][1], i)  # noqa: E731
    E = len(x)
    open_ = set(range(E))
    if groups > 1:
        per = E // groups
        gs = []
        for g in range(groups):
            c = sorted((choice[i][0] for i in range(g * per, (g + 1) * per)), reverse=True)
            gs.append(sum(c[:best]))
        kept = sorted(range(groups), key=lambda g: (-gs[g], g))[:top]
        open_ = {i for g in kept for i in range(g * per, (g + 1) * per)}
    order = sorted(open_, key=key)
    ids = order[:k]
    w = [score[i] for i in ids]
    if normalize:
        s = sum(w)
        w = [v / s if s > 0 else 0.0 for v in w]
    return ids, [v * scale for v in w]


def grid(T, E, seed, dtype):
    """Logits on a grid of 1/64 with many ties: sums, scores and their order are the same in 32 and 64 bits or tied."""
    g = torch.Generator()
    g.manual_seed(seed)
    return (torch.randint(-256, 256, (T, E), generator=g).float() / 64).to(DTYPES[dtype])


CASES = [  # T, E, k, scoring, bias, groups, top, best
    (1, 128, 8, "softmax", False, 1, 1, 1), (5, 8, 2, "softmax", False, 1, 1, 1), (3, 60, 4, "softmax", False, 1, 1, 1),
    (7, 1, 1, "softmax", False, 1, 1, 1), (4, 33, 32, "softmax", False, 1, 1, 1), (130, 256, 8, "softmax", False, 1, 1, 1),
    (9, 512, 8, "softmax", False, 1, 1, 1), (3, 513, 6, "softmax", False, 1, 1, 1), (2, 4096, 8, "softmax", False, 1, 1, 1),
    (11, 64, 6, "sigmoid", False, 1, 1, 1), (6, 256, 8, "sigmoid", False, 8, 4, 1), (5, 160, 6, "softmax", False, 8, 3, 1),
    (5, 96, 3, "softmax", False, 32, 1, 1), (4, 4000, 8, "sigmoid", False, 20, 7, 1),
]


@pytest.mark.parametrize("T,E,k,scoring,bias,groups,top,best", CASES)
@pytest.mark.parametrize("dtype", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("normalize,scale", [(True, 1.0), (False, 2.5)])
def test_ids_and_weights(ctx, T, E, k, scoring, bias, groups, top, best, dtype, normalize, scale):
    x = grid(T, E, E + T, dtype)
    ids, w = ctx.moe_route(x.cuda(), k, scoring=scoring, n_groups=groups, top_groups=top, group_best=best,
                           normalize=normalize, scale=scale)
    ctx.sync_status()
    for t in range(T):
        want, ww = reference(x[t], k, scoring, None, groups, top, best, normalize, scale)
        assert ids[t].tolist() == want
        # exp and a division within 2 fp32 roundings each; the sums of E or k terms add (E or k) more at most
        tol = (8 + k + (0 if normalize and scoring == "softmax" or scoring == "sigmoid" else math.sqrt(E))) * 2.0 ** -23
        assert all(abs(a - b) <= tol * b + 1e-38 for a, b in zip(w[t].tolist(), ww))


@pytest.mark.parametrize("scoring", ["softmax", "sigmoid"])
@pytest.mark.parametrize("E,groups,top,best,k", [(64, 1, 1, 1, 6), (256, 8, 4, 2, 8), (160, 8, 3, 2, 6), (1024, 16, 5, 2, 8)])
def test_bias_moves_the_choice_and_not_the_weights(ctx, scoring, E, groups, top, best, k):
    """Biases a multiple of 2^-10 apart rank the experts; the scores are too small to change that order."""
    T = 5
    g = torch.Generator()
    g.manual_seed(E)
    x = torch.randn((T, E), generator=g) * 0.01 - (8.0 if scoring == "sigmoid" else 0.0)
    x = x - 3.0 * (torch.arange(E) % 7 == 0)
    bias = torch.randperm(E, generator=g).float() * 0.125
    ids, w = ctx.moe_route(x.cuda(), k, scoring=scoring, bias=bias.cuda(), n_groups=groups, top_groups=top, group_best=best)
    ctx.sync_status()
    for t in range(T):
        want, ww = reference(x[t], k, scoring, bias, groups, top, best, True, 1.0)
        assert ids[t].tolist() == want
        assert all(abs(a - b) <= (10 + k) * 2.0 ** -23 * b for a, b in zip(w[t].tolist(), ww))


@pytest.mark.parametrize("scoring", ["softmax", "sigmoid"])
def test_infinities_nan_and_equal_rows(ctx, scoring):
    E, k = 40, 4
    inf, nan = math.inf, math.nan
    x = torch.zeros((7, E))
    x[1] = -inf
    x[2] = nan
    x[3] = -inf
    x[3, 30], x[3, 2] = 1.0, 0.5            # fewer numbers than choices: -inf by index
    x[4, 5], x[4, 9] = inf, inf
    x[5, :38] = nan                          # two numbers, then NaN by index
    x[6, ::2] = -0.0                         # -0 ties with +0
    ids, w = ctx.moe_route(x.cuda(), k, scoring=scoring)
    ctx.sync_status()
    for t in range(7):
        want, ww = reference(x[t], k, scoring, None, 1, 1, 1, True, 1.0)
        assert ids[t].tolist() == want, t
        assert all(abs(a - b) <= 1e-6 for a, b in zip(w[t].tolist(), ww)), t
    assert torch.isfinite(w).all()


def test_feeds_the_expert_layer(ctx):
    """moe_route and the routed layer give what the layer gives when it routes by itself."""
    E, H, I, k = 16, 512, 256, 4
    g = syn.rng(91, 0)
    w8 = [to_dev(syn.expert_bank(f, E, r, c, g)) for f, r, c in (("Q4_K", I, H), ("Q4_K", I, H), ("Q6_K", H, I))]
    weights = ctx.moe_weights("Q4_K", w8[0], "Q4_K", w8[1], "Q6_K", w8[2])
    for T in (1, 3, 40):
        x, lg = to_dev(syn.activations(T, H, g)), to_dev(syn.router_logits(T, E, g))
        a = ctx.moe_experts(weights, E, H, I, k, x, logits=lg)
        ids, rw = ctx.moe_route(lg, k)
        b = ctx.moe_experts(weights, E, H, I, k, x, ids=ids, route_w=rw)
        ctx.sync_status()
        # the same experts and integer dots; the weights may differ by a rounding
        assert float((a - b).norm() / a.norm()) <= 1e-6


def test_refusals(ctx):
    x = torch.zeros((2, 64), device="cuda")
    for kw in (dict(top_k=0), dict(top_k=65), dict(top_k=33), dict(top_k=2, n_groups=7), dict(top_k=2, n_groups=0),
               dict(top_k=2, n_groups=8, top_groups=9), dict(top_k=9, n_groups=8, top_groups=1),
               dict(top_k=2, group_best=3), dict(top_k=2, n_groups=64, top_groups=3)):
        with pytest.raises(ggq.GGQError, match="moe_route"):
            ctx.moe_route(x, **kw)
    with pytest.raises(ggq.GGQError, match="moe_route"):
        ctx.moe_route(torch.zeros((1, 4097), device="cuda"), 2)
    with pytest.raises(ggq.GGQError, match="finite"):
        ctx.moe_route(x, 2, scale=math.inf)
    with pytest.raises(ValueError, match="logits"):
        ctx.moe_route(x.double(), 2)
    with pytest.raises(ValueError, match="bias"):
        ctx.moe_route(x, 2, bias=torch.zeros(3, device="cuda"))
    with pytest.raises(ValueError, match="contiguous"):
        ctx.moe_route(x[:, ::2], 2)
    with pytest.raises(KeyError):
        ctx.moe_route(x, 2, scoring="relu")
    ids, w = ctx.moe_route(x[:0], 2)
    assert ids.shape == (0, 2) and w.shape == (0, 2)
    ctx.sync_status()
