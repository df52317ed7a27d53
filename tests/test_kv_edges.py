"""The key/value cache's calls at the edges of their arguments: devices, strides of axes of one element, and
buffers that are given for a part of the results."""
import types

import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

import gguf_block_quant_ggq_gb300 as ggq  # noqa: E402
from test_attention import Case, ctx  # noqa: E402,F401


def test_pools_and_caches_of_another_device_are_refused(ctx):  # noqa: F811
    """A context of device 1 (none is needed: the refusal comes before any call) and a cache of device 0, and the reverse."""
    mine = ctx.kv_cache("Q8_0", "Q4_0", 2, 16, 1, 64)
    other = types.SimpleNamespace(_torch=torch, device=1)
    with pytest.raises(ValueError, match="cuda:1"):
        ggq.KVCache(other, "Q8_0", "Q4_0", 2, 16, 1, 64, k=mine.k, v=mine.v)
    mine.device = 1
    rows, slots = torch.zeros((1, 1, 64), device="cuda"), torch.zeros(1, dtype=torch.int64, device="cuda")
    lens, table = torch.ones(1, dtype=torch.int32, device="cuda"), torch.zeros((1, 1), dtype=torch.int32, device="cuda")
    with pytest.raises(ValueError, match="cuda:1"):
        ctx.kv_store(mine, rows, rows, slots)
    with pytest.raises(ValueError, match="cuda:1"):
        ctx.kv_load(mine, slots)
    with pytest.raises(ValueError, match="cuda:1"):
        ctx.attention(mine, rows, lens, table)
