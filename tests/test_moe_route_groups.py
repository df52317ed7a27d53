"""The groups of ggq_moe_route: their scores are sums of the experts' choices (score + bias), for softmax too.

The reference is in 64 bits; the logits lie on a grid of 1/64, so that equal sums are equal in 32 bits as
well, and `gap` makes sure that no other sums come closer than 32-bit roundings (2^-20 of their size)."""
import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

from test_moe_route import DTYPES, ctx, grid  # noqa: E402,F401


def reference(x, k, groups, top, best, scoring, bias):
    """(ids, weights, gap between the last open group's score and the next different one) of rows x, in 64 bits."""
    x = x.double()
    score = torch.softmax(x, -1) if scoring == "softmax" else torch.sigmoid(x)
    choice = score if bias is None else score + bias.double()
    best = min(best, x.shape[1] // groups)
    sums = choice.unflatten(1, (groups, -1)).sort(dim=-1, descending=True).values[..., :best].sum(-1)
    order = sums.sort(dim=-1, descending=True, stable=True)
    open_ = torch.zeros_like(sums, dtype=torch.bool).scatter_(1, order.indices[:, :top], True)
    edge = order.values[:, top - 1:top]
    other = (order.values - edge).abs()
    gap = torch.where(other < 1e-14, 1.0, other / edge.abs()).amin() if top < groups else torch.tensor(1.0)
    masked = choice.masked_fill(~open_.repeat_interleave(x.shape[1] // groups, 1), -1e300)
    ids = masked.sort(dim=-1, descending=True, stable=True).indices[:, :k]
    w = score.gather(1, ids)
    return ids, w / w.sum(-1, keepdim=True), float(gap)


@pytest.mark.parametrize("row,want", [([10.0, -10.0, 4.0, 4.0], [0, 1]), ([5.0, -5.0, 2.0, 2.0], [0, 1]),
                                      ([4.0, 4.0, 5.0, 3.0], [2, 3]), ([-90.0, -99.0, -91.0, -91.0], [0, 1])])
def test_two_scores_are_added_and_not_two_logits(ctx, row, want):  # noqa: F811
    ids, _ = ctx.moe_route(torch.tensor([row], device="cuda"), 2, n_groups=2, top_groups=1, group_best=2)
    assert ids[0].tolist() == want


# groups of whole lanes, of parts of lanes, of a lane and a part, and more than 512 experts
@pytest.mark.parametrize("T,E,groups,top,k", [(40, 64, 8, 3, 6), (33, 256, 8, 4, 8), (21, 160, 8, 3, 6), (9, 512, 16, 2, 4),
                                              (7, 60, 5, 2, 8), (5, 1024, 16, 5, 8), (3, 4000, 20, 7, 8), (25, 24, 12, 4, 6)])
@pytest.mark.parametrize("dtype", ["f32", "f16", "bf16"])
def test_softmax_groups(ctx, T, E, groups, top, k, dtype):  # noqa: F811
    x = grid(T, E, 3 * E + T, dtype)
    want, weights, gap = reference(x, k, groups, top, 2, "softmax", None)
    assert gap > 2.0 ** -20
    ids, w = ctx.moe_route(x.cuda(), k, n_groups=groups, top_groups=top, group_best=2)
    assert torch.equal(ids.cpu().long(), want)
    assert ((w.cpu().double() - weights).abs() <= (10 + k + E ** 0.5) * 2.0 ** -23 * weights).all()
    # a bias of zeros changes no expert
    with_bias, _ = ctx.moe_route(x.cuda(), k, n_groups=groups, top_groups=top, group_best=2, bias=torch.zeros(E, device="cuda"))
    assert torch.equal(ids, with_bias)
    ctx.sync_status()


@pytest.mark.parametrize("T,E,top,k", [(6, 32, 5, 5), (9, 8, 3, 2), (4, 17, 16, 16)])
@pytest.mark.parametrize("scoring,bias", [("softmax", False), ("softmax", True), ("sigmoid", False), ("sigmoid", True)])
def test_groups_of_one_expert(ctx, T, E, top, k, scoring, bias):  # noqa: F811
    """No second choice to add: the group's score is its expert's."""
    x = grid(T, E, E, "f32")
    b = torch.randperm(E, generator=torch.Generator().manual_seed(E)).float() / 4 if bias else None
    want, weights, gap = reference(x, k, E, top, 2, scoring, b)
    assert gap > 2.0 ** -20
    args = dict(scoring=scoring, n_groups=E, top_groups=top, bias=None if b is None else b.cuda())
    ids, w = ctx.moe_route(x.cuda(), k, group_best=2, **args)
    assert torch.equal(ids.cpu().long(), want)
    assert ((w.cpu().double() - weights).abs() <= (10 + k + E ** 0.5) * 2.0 ** -23 * weights).all()
    assert torch.equal(ids, ctx.moe_route(x.cuda(), k, group_best=1, **args)[0])
    ctx.sync_status()
