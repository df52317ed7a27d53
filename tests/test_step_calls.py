"""How the calls of a decoding step behave as calls: captured into graphs and replayed on new inputs, on given streams
and on two streams at once, with offsets beyond 32 bits, and with requests for nothing."""
import os
import subprocess
import sys

import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

import gguf_block_quant_ggq_gb300 as ggq  # noqa: E402


@pytest.fixture(scope="module")
def ctx():
    assert torch.cuda.is_available(), "GPU tests need a CUDA device"
    from gguf_block_quant_ggq_gb300 import _build
    _build.build()
    c = ggq.Context(0)
    yield c
    c.close()


def ints(a, dtype=torch.int32):
    return torch.tensor(a, dtype=dtype, device="cuda")


class Calls:
    """A small call of each kind on inputs that refill() changes in place."""

    def __init__(self, ctx, seed=0):
        self.ctx, self.gen = ctx, torch.Generator(device="cuda")
        self.gen.manual_seed(seed)
        self.x, self.res = torch.empty((2, 37, 520), device="cuda", dtype=torch.bfloat16).unbind(0)
        self.heads = torch.empty((37, 6, 64), device="cuda")
        self.logits = torch.empty((37, 5003), device="cuda", dtype=torch.float16)
        self.y = torch.empty((37, 300), device="cuda", dtype=torch.bfloat16)
        self.pos, self.tokens, self.ids = (torch.empty(37, dtype=torch.int32, device="cuda") for _ in range(3))
        self.slots = torch.empty(37, dtype=torch.int64, device="cuda")
        self.w = torch.rand(520, device="cuda", generator=self.gen)
        self.table = ctx.rotary_table(100, 64)
        self.cache = ctx.kv_cache("Q8_0", "Q4_0", 3, 32, 2, 64)
        self.adapters = ctx.adapters(torch.randn((3, 16, 520), device="cuda", generator=self.gen).bfloat16(),
                                     torch.randn((3, 300, 16), device="cuda", generator=self.gen).bfloat16())
        self.start = ints([0, 20, 20, 37])
        self.refill()

    def refill(self):
        for t in (self.x, self.res, self.heads, self.logits, self.y):
            t.copy_(torch.randn(t.shape, device="cuda", generator=self.gen))
        for t, n in ((self.pos, 100), (self.tokens, 5003), (self.ids, 3)):
            t.copy_(torch.randint(0, n, (37,), device="cuda", generator=self.gen))
        self.slots.copy_(torch.randperm(96, device="cuda", generator=self.gen)[:37])

    def run(self, stream=None, ctx=None):
        c, s = ctx or self.ctx, dict(stream=stream)
        q, k, v = self.heads.split([2, 2, 2], 1)
        return [*c.norm(self.x, before=self.w, after=self.w, residual=self.res, **s), c.norm(self.x[:, :512], before=True, act="Q8_K", **s)[0],
                c.rotate(self.heads, self.table, self.pos, **s), c.kv_append(self.cache, k, v, self.slots, self.table, self.pos, q=q, **s),
                *c.kv_load(self.cache, self.slots, **s), c.adapt(self.adapters, self.x, self.y, self.ids, **s),
                c.adapt(self.adapters, self.x, self.y, self.ids[:3], q_start=self.start, **s), *c.logprobs(self.logits, self.tokens, top_k=4, **s),
                c.rotary_table(50, 32, **s)]


def test_captured_calls_follow_their_inputs(ctx):
    calls = Calls(ctx)
    calls.run()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = calls.run()
    for _ in range(3):
        calls.refill()
        graph.replay()
        got_now = [g.clone() for g in got]
        for a, b in zip(got_now, calls.run()):
            assert torch.equal(a, b)
    ctx.sync_status()


def test_streams_given_and_two_contexts_at_once(ctx):
    """Each stream has a context of its own; the calls of both are under way at once."""
    other = ggq.Context(0)
    a, b = Calls(ctx, 1), Calls(other, 2)
    want = [a.run(), b.run()]
    s = [torch.cuda.Stream(), torch.cuda.Stream()]
    torch.cuda.synchronize()
    for _ in range(20):
        got = [a.run(stream=s[0]), b.run(stream=s[1])]
    torch.cuda.synchronize()
    for g, w in zip(got, want):
        for x, y in zip(g, w):
            assert torch.equal(x, y)
    other.sync_status()
    other.close()
    ctx.sync_status()


def test_outputs_are_of_the_given_streams_memory(ctx):
    calls = Calls(ctx)
    big = torch.zeros((64, 32768), device="cuda")
    made = {
        "norm": lambda s: ctx.norm(big, before=True, stream=s)[0],
        "packed": lambda s: ctx.norm(big, before=True, act="Q8_K", stream=s)[0],
        "rotate": lambda s: ctx.rotate(big.view(64, 512, 64), calls.table, ints([1] * 64), stream=s),
        "table": lambda s: ctx.rotary_table(70000, 32, stream=s),
        "logprobs": lambda s: ctx.logprobs(big, ints([[1] * 20000] * 64), stream=s)[0],
        "adapt": lambda s: ctx.adapt(ctx.adapters(torch.zeros((1, 8, 520), device="cuda").half(), torch.zeros((1, 32768, 8), device="cuda").half()),
                                     torch.zeros((64, 520), device="cuda"), big, ints([0] * 64), stream=s),
    }
    s = torch.cuda.Stream()
    for name, call in made.items():
        torch.cuda.synchronize()
        torch.cuda.empty_cache()
        out = call(s)
        torch.cuda.synchronize()
        at, size = out.untyped_storage().data_ptr(), out.untyped_storage().nbytes()
        del out
        # the block is the given stream's again, and no other's
        with torch.cuda.stream(s):
            assert torch.empty(size, dtype=torch.uint8, device="cuda").data_ptr() == at, name


def test_offsets_beyond_32_bits(ctx):
    """Two rows 2^31 elements apart (and banks that long): the same as side by side."""
    far = 1 << 31
    buf = torch.empty(far + (1 << 16), dtype=torch.bfloat16, device="cuda")
    g = torch.Generator(device="cuda")
    g.manual_seed(1)

    def apart(t):
        """t's two rows with 2^31 elements between them."""
        flat = t.reshape(2, -1)
        view = buf.as_strided(flat.shape, (far, 1))
        view.copy_(flat)
        inner = t.stride()[1:]
        return buf.as_strided(t.shape, (far, *inner))
    x = torch.randn((2, 1032), device="cuda", generator=g).bfloat16()
    want = ctx.norm(x, before=True)[0]
    assert torch.equal(ctx.norm(apart(x), before=True)[0], want)
    out = buf.as_strided((2, 1032), (far, 1), 8192)
    ctx.norm(x, before=True, out=out)
    assert torch.equal(out, want)
    table, pos = ctx.rotary_table(50, 64), ints([3, 40])
    heads = torch.randn((2, 4, 64), device="cuda", generator=g).bfloat16()
    want = ctx.rotate(heads, table, pos)
    assert torch.equal(ctx.rotate(apart(heads), table, pos), want)
    slots = ints([5, 17], torch.int64)
    a, b = (ctx.kv_cache("Q8_0", "Q8_0", 2, 16, 4, 64) for _ in range(2))
    ctx.kv_append(a, heads, heads, slots, table, pos)
    there = apart(heads)
    q = ctx.kv_append(b, there, there, slots, table, pos, q=there)
    assert torch.equal(a.k, b.k) and torch.equal(a.v, b.v) and torch.equal(q, want)
    logits, tokens = torch.randn((2, 9001), device="cuda", generator=g).bfloat16(), ints([[5], [9000]])
    for u, v in zip(ctx.logprobs(logits, tokens, top_k=3), ctx.logprobs(apart(logits), tokens, top_k=3)):
        # the rows' alignment differs: the sums' order does
        assert torch.equal(u, v) if u.dtype is torch.int32 else float((u - v).abs().max()) <= 1e-5
    ad = ctx.adapters(torch.randn((2, 16, 1032), device="cuda", generator=g).bfloat16(), torch.randn((2, 200, 16), device="cuda", generator=g).bfloat16())
    y = torch.randn((2, 200), device="cuda", generator=g).bfloat16()
    for start, ids in ((None, ints([1, 0])), (ints([0, 2]), ints([1]))):
        assert torch.equal(ctx.adapt(ad, apart(x), y, ids, q_start=start), ctx.adapt(ad, x, y, ids, q_start=start))
        assert torch.equal(ctx.adapt(ad, x, apart(y), ids, q_start=start), ctx.adapt(ad, x, y, ids, q_start=start))
    del buf, there, out
    torch.cuda.empty_cache()
    # the last of so many adapters that its banks start beyond 2^31 elements
    n, R, K = 130, 256, 65536
    a, b = torch.zeros((n, R, K), dtype=torch.float16, device="cuda"), torch.zeros((n, 40, R), dtype=torch.float16, device="cuda")
    a[-1] = torch.randn((R, K), device="cuda", generator=g) / 256
    b[-1] = torch.randn((40, R), device="cuda", generator=g)
    x, y = torch.randn((3, K), device="cuda", generator=g), torch.randn((3, 40), device="cuda", generator=g)
    many, one = ctx.adapters(a, b), ctx.adapters(a[-1:].clone(), b[-1:].clone())
    assert torch.equal(ctx.adapt(many, x, y, ints([n - 1] * 3)), ctx.adapt(one, x, y, ints([0] * 3)))
    ctx.sync_status()


def test_many_tokens(ctx):
    """More rows than a grid's second axis holds: every row is reached."""
    n = 70000
    x = torch.randn((n, 64), device="cuda")
    assert torch.equal(ctx.norm(x, before=True)[0][[0, 65535, 65536, n - 1]], ctx.norm(x[[0, 65535, 65536, n - 1]], before=True)[0])
    table, pos = ctx.rotary_table(n, 64), torch.arange(n, device="cuda", dtype=torch.int32)
    got = ctx.rotate(x.view(n, 1, 64), table, pos)
    assert torch.equal(got[65530:], ctx.rotate(x[65530:].view(-1, 1, 64), table, pos[65530:]))
    cache, want = (ctx.kv_cache("Q8_0", "Q4_0", (n + 15) // 16, 16, 1, 64) for _ in range(2))
    slots = torch.arange(n, device="cuda")
    ctx.kv_append(cache, x.view(n, 1, 64), x.view(n, 1, 64), slots, table, pos)
    ctx.kv_store(want, got, x.view(n, 1, 64), slots)
    assert torch.equal(cache.k, want.k) and torch.equal(cache.v, want.v)
    lp, ent, ids, top = ctx.logprobs(x, pos % 64, top_k=2)
    z = torch.log_softmax(x.double(), 1)
    assert float((lp - z.gather(1, (pos % 64).long()[:, None])[:, 0]).abs().max()) <= 1e-5
    assert torch.equal(ids[:, 0].long(), x.argmax(1))
    ad = ctx.adapters(torch.randn((2, 8, 64), device="cuda").half(), torch.randn((2, 24, 8), device="cuda").half())
    y, which = torch.randn((n, 24), device="cuda"), torch.arange(n, device="cuda", dtype=torch.int32)[:4000] % 2
    got = ctx.adapt(ad, x, y, ints([1]), q_start=ints([0, n]))
    exact = y.double() + (x.double() @ ad.a[1].double().T) @ ad.b[1].double().T
    size = y.double().abs() + (x.double().abs() @ ad.a[1].double().abs().T) @ ad.b[1].double().abs().T
    assert bool(((got - exact).abs() <= 64 * 2.0 ** -24 * size).all())
    one = ctx.adapt(ad, x[:4000], y[:4000], which)  # many single tokens
    exact = y[:4000].double() + torch.stack([(x[:4000].double() @ ad.a[i].double().T) @ ad.b[i].double().T for i in range(2)])[which.long(), torch.arange(4000, device="cuda")]
    size = y[:4000].double().abs() + torch.stack([(x[:4000].double().abs() @ ad.a[i].double().abs().T) @ ad.b[i].double().abs().T for i in range(2)])[which.long(), torch.arange(4000, device="cuda")]
    assert bool(((one - exact).abs() <= 64 * 2.0 ** -24 * size).all())
    ctx.sync_status()


FIRST = """
import torch
import gguf_block_quant_ggq_gb300 as ggq
ctx = ggq.Context(0)
x, ids = torch.randn(300, 1024, device="cuda"), torch.zeros(300, dtype=torch.int32, device="cuda")
wide, logits = torch.randn(4, 8192, device="cuda"), torch.randn(3, 131072, device="cuda")
ad = ctx.adapters(torch.randn(2, 16, 1024, device="cuda").half(), torch.randn(2, 1024, 16, device="cuda").half())
cache = ctx.kv_cache("Q8_0", "Q4_0", 10, 32, 2, 64)
k = x.view(300, 16, 64)
def run():
    table = ctx.rotary_table(100, 64)
    return [table, ctx.norm(x, before=True)[0], ctx.norm(wide, before=True)[0], ctx.adapt(ad, x, x, ids), ctx.rotate(k, table, ids),
            ctx.kv_append(cache, k[:, :2], k[:, 2:4], torch.arange(300, device="cuda"), table, ids, q=k), ctx.logprobs(logits, ids[:3], top_k=3)[0]]
torch.cuda.synchronize()
graph = torch.cuda.CUDAGraph()
with torch.cuda.graph(graph):
    got = run()
graph.replay()
torch.cuda.synchronize()
assert all(torch.equal(a, b) for a, b in zip(got, run()))
ctx.sync_status()
"""


def test_first_calls_of_a_process_are_captured(ctx):
    done = subprocess.run([sys.executable, "-c", FIRST], capture_output=True, text=True, timeout=300,
                          cwd=os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
    assert done.returncode == 0, done.stderr[-2000:]
