"""ggq_attention at the edges of its plan, its masks and its ranges: batches whose items meet in one CTA's
counters, and the rows that must not notice what they do not see.

The reference and the tolerance are those of test_attention_tiles."""
import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

from test_attention import Case, ctx  # noqa: E402,F401
from test_attention_tiles import check  # noqa: E402


@pytest.mark.parametrize("dtype,news", [("f32", 1), ("bf16", 1), ("bf16", 2), ("f32", 3)])
@pytest.mark.parametrize("lens", [[38421, 6670], [96394, 1557, 13709], [1094, 5198, 50458, 1056]])
def test_long_sequences_beside_short_ones(ctx, lens, dtype, news):  # noqa: F811
    """The last group of one item's pieces begins with the CTA that begins the next item: every
    row is written, the same way in every call on the context."""
    c = Case(ctx, lens, [news] * len(lens), 32, 8, 128, dtype=dtype, page=64, seed=len(lens))
    out = torch.full_like(c.q, 7.0)
    c.call(out=out)
    ctx.sync_status()
    check(c, out)
    for _ in range(3):
        again = torch.full_like(c.q, 9.0)
        c.call(out=again)
        assert torch.equal(out, again)
    ctx.sync_status()
