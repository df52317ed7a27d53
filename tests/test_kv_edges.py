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


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_strides_of_axes_of_one_element(ctx, dtype):  # noqa: F811
    """One token, or one head, whose stride no address depends on: any is taken."""
    g = torch.Generator(device="cuda")
    g.manual_seed(1)
    for tokens, heads in ((1, 4), (6, 1), (1, 1)):
        cache, want = (ctx.kv_cache("Q8_0", "Q8_0", 2, 16, heads, 64) for _ in range(2))
        x = torch.randn((3, tokens, heads, 64), device="cuda", generator=g).to(dtype)
        slots = torch.arange(tokens, device="cuda")
        # odd strides of the axes of one element
        odd = [t.as_strided(t.shape, (t.stride(0) if tokens > 1 else 4097, t.stride(1) if heads > 1 else 33, 1)) for t in x]
        ctx.kv_store(cache, odd[0], odd[1], slots)
        ctx.kv_store(want, x[0], x[1], slots)
        assert torch.equal(cache.k, want.k) and torch.equal(cache.v, want.v)
        lens = torch.full((tokens,), tokens, dtype=torch.int32, device="cuda")
        table = torch.zeros((tokens, 1), dtype=torch.int32, device="cuda")
        assert torch.equal(ctx.attention(cache, odd[2], lens, table), ctx.attention(cache, x[2], lens, table))
    ctx.sync_status()


def test_one_given_buffer_sets_the_type_of_both(ctx):  # noqa: F811
    c = Case(ctx, [21], [1], 2, 2, 64)
    want = ctx.kv_load(c.cache, c.slots, dtype=torch.bfloat16)
    for name in ("k", "v"):
        given = torch.empty_like(want[0])
        got = ctx.kv_load(c.cache, c.slots, **{name: given})
        assert got["kv".index(name)] is given
        assert all(torch.equal(a, b) for a, b in zip(got, want))
    ctx.sync_status()


def test_outputs_are_of_the_given_streams_memory(ctx):  # noqa: F811
    """What a call makes for itself comes from the memory of the stream that writes it: the block goes back to
    that stream when the output is dropped, and to no other one."""
    c = Case(ctx, [21, 40], [1, 1], 2, 2, 64)
    x = torch.zeros((3, 70000), device="cuda")
    calls = {
        "attention": lambda s: ctx.attention(c.cache, c.q, c.dlens, c.table, stream=s),
        "kv_load": lambda s: ctx.kv_load(c.cache, c.slots, stream=s)[1],
        "moe_route": lambda s: ctx.moe_route(x[:, :64].contiguous(), 2, stream=s)[0],
        "quantize_act": lambda s: ctx.quantize_act("Q8_0", x[:, :256].contiguous(), stream=s),
    }
    s = torch.cuda.Stream()
    for name, call in calls.items():
        torch.cuda.synchronize()
        torch.cuda.empty_cache()
        out = call(s)
        torch.cuda.synchronize()
        at, size = out.untyped_storage().data_ptr(), out.untyped_storage().nbytes()
        del out
        with torch.cuda.stream(s):
            blocks = [torch.empty(size, dtype=torch.uint8, device="cuda") for _ in range(4)]
        assert at in [b.data_ptr() for b in blocks], name
    ctx.sync_status()
