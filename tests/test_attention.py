"""ggq_attention against softmax attention in 64 bits over the values that the
cache's blocks stand for.

Tolerance.  With S the largest scale * sum_d |q_d k_d| of a row and A = sum_j p_j
|v_j| per channel, an error of e S in the scores moves each p_j by at most 2 e S
relative, and rounding p and summing adds a few e: |error| <= e (8 + 2 S) A.  fp32
activations: e = 2^-21 (operands split into fp16 pairs of 22 bits, fp32 sums).
fp16 and bf16: e = 2^-11 (cache values and probabilities rounded to fp16), plus
one rounding of the output, 2^-11 or 2^-8 of it."""
import math

import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

import gguf_block_quant_ggq_gb300 as ggq  # noqa: E402

DTYPES = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}
SPLIT = {"f32": 2.0 ** -21, "f16": 2.0 ** -11, "bf16": 2.0 ** -11}
ROUND = {"f32": 2.0 ** -23, "f16": 2.0 ** -11, "bf16": 2.0 ** -8}


@pytest.fixture(scope="module")
def ctx():
    assert torch.cuda.is_available(), "GPU tests need a CUDA device"
    from gguf_block_quant_ggq_gb300 import _build
    _build.build()
    c = ggq.Context(0)
    yield c
    c.close()


class Case:
    """A cache whose unused places hold NaN scales, with tables whose unused entries are -1."""

    def __init__(self, ctx, lens, news, H=4, Hkv=2, D=64, k_type="Q8_0", v_type="Q8_0", dtype="f32", page=16, seed=0,
                 spare_pages=2, q_mul=1.0):
        self.ctx, self.lens, self.news, self.H, self.Hkv, self.D, self.dtype = ctx, lens, news, H, Hkv, D, dtype
        g = torch.Generator(device="cuda")
        g.manual_seed(seed)
        pages = [(x + page - 1) // page for x in lens]
        n_pages = sum(pages) + spare_pages
        self.cache = ctx.kv_cache(k_type, v_type, n_pages, page, Hkv, D)
        self.cache.k.fill_(0xFF)
        self.cache.v.fill_(0xFF)
        order = torch.randperm(n_pages, generator=g, device="cuda").tolist()
        table = torch.full((len(lens), max(pages + [1])), -1, dtype=torch.int32)
        slots, k0 = [], 0
        for i, x in enumerate(lens):
            own = order[k0:k0 + pages[i]]
            k0 += pages[i]
            table[i, :pages[i]] = torch.tensor(own, dtype=torch.int32)
            slots += [own[j // page] * page + j % page for j in range(x)]
        self.table = table.cuda()
        n = len(slots)
        self.slots = torch.tensor(slots, dtype=torch.int64, device="cuda")
        if n:
            k = torch.randn((n, Hkv, D), device="cuda", generator=g)
            v = torch.randn((n, Hkv, D), device="cuda", generator=g)
            ctx.kv_store(self.cache, k, v, self.slots)
        self.k, self.v = (x.double() for x in ctx.kv_load(self.cache, self.slots))
        self.q = (torch.randn((sum(news), H, D), device="cuda", generator=g) * q_mul).to(DTYPES[dtype])
        self.dlens = torch.tensor(lens, dtype=torch.int32, device="cuda")
        self.q_start = torch.tensor([sum(news[:i]) for i in range(len(news) + 1)], dtype=torch.int32, device="cuda")

    def call(self, **kw):
        args = dict(q_start=self.q_start, max_q=max(self.news))
        args.update(kw)
        return self.ctx.attention(self.cache, args.pop("q", self.q), self.dlens, self.table, **args)

    def check(self, out, scale=None, cap=0.0, window=0, slopes=None, q=None):
        q = (self.q if q is None else q).double()
        G, scale = self.H // self.Hkv, self.D ** -0.5 if scale is None else scale
        r0 = k0 = 0
        for length, new in zip(self.lens, self.news):
            k, v = self.k[k0:k0 + length], self.v[k0:k0 + length]
            pos = torch.arange(length - new, length, device="cuda")
            key = torch.arange(length, device="cuda")
            seen = key[None] <= pos[:, None]
            if window:
                seen &= key[None] > pos[:, None] - window
            for h in range(self.H):
                qq, kk, vv = q[r0:r0 + new, h], k[:, h // G], v[:, h // G]
                got = out[r0:r0 + new, h].double()
                x = scale * qq @ kk.T
                size = abs(scale) * qq.abs() @ kk.abs().T
                if cap > 0:
                    x = cap * torch.tanh(x / cap)
                if slopes is not None:
                    far = float(slopes[h]) * (key[None] - pos[:, None])
                    x, size = x + far, size + far.abs()
                x = x.masked_fill(~seen, -math.inf)
                some = seen.any(1)
                p = torch.where(some[:, None], torch.softmax(x, -1), 0.0).nan_to_num(0.0)
                # keys far below the row's largest score weigh nothing: their scores' errors do not count
                S = (size * (p > 1e-9)).amax(1, keepdim=True) if length else torch.zeros((new, 1), device="cuda")
                want, A = p @ vv, p @ vv.abs()
                bound = SPLIT[self.dtype] * (8 + 2 * S) * A + ROUND[self.dtype] * want.abs() + 1e-30
                err = (got - want).abs()
                assert torch.isfinite(got).all()
                assert (err <= bound).all(), f"head {h}: worst {float((err / bound).max()):.3g} of the bound"
                assert (got[~some] == 0).all()
            r0 += new
            k0 += length


ONE = [1, 2, 15, 16, 17, 0, 31, 33, 100, 1000, 5]


@pytest.mark.parametrize("k_type,v_type", [("Q8_0", "Q8_0"), ("Q4_0", "Q4_0"), ("Q8_0", "Q4_0"), ("Q4_0", "Q8_0")])
@pytest.mark.parametrize("dtype", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("H,Hkv,D,page", [(4, 2, 64, 16), (32, 8, 128, 64), (7, 1, 128, 48), (6, 3, 256, 32), (16, 1, 64, 16),
                                          (20, 1, 128, 16)])
def test_single_tokens(ctx, H, Hkv, D, page, dtype, k_type, v_type):
    c = Case(ctx, ONE, [1] * len(ONE), H, Hkv, D, k_type, v_type, dtype, page, seed=H + D)
    out = c.call(q_start=None)
    ctx.sync_status()
    c.check(out)
    assert torch.equal(out, c.call(max_len=1000))  # the same rows with their starts and a bound given
    ctx.sync_status()


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("seqs,length", [(1, 20000), (3, 7001), (300, 90)])
def test_single_tokens_long_and_many(ctx, seqs, length, dtype):
    lens = [max(1, length - 37 * i) for i in range(seqs)]
    c = Case(ctx, lens, [1] * seqs, 8, 2, 128, "Q8_0", "Q8_0", dtype, 64, seed=seqs)
    out = c.call(q_start=None)
    ctx.sync_status()
    c.check(out)


@pytest.mark.parametrize("k_type,v_type", [("Q8_0", "Q8_0"), ("Q4_0", "Q4_0"), ("Q8_0", "Q4_0")])
@pytest.mark.parametrize("dtype", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("H,Hkv,D", [(8, 2, 64), (7, 1, 128), (4, 2, 256)])
def test_several_tokens(ctx, H, Hkv, D, dtype, k_type, v_type):
    """Drafted tokens, a prompt from nothing, a chunk, rows before the first key, an empty sequence, none new."""
    lens, news = [300, 40, 129, 3, 0, 77, 512], [5, 40, 17, 6, 2, 0, 1]
    c = Case(ctx, lens, news, H, Hkv, D, k_type, v_type, dtype, 32, seed=D)
    out = c.call()
    ctx.sync_status()
    c.check(out)


@pytest.mark.parametrize("dtype", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("H,Hkv,D,lens,news", [
    (8, 2, 128, [700], [700]), (4, 4, 64, [513, 1000], [513, 200]), (7, 1, 128, [391, 130, 64], [391, 129, 64]),
    (4, 2, 256, [300, 257], [300, 256]), (32, 8, 128, [2100], [333]), (16, 1, 64, [127, 128, 129], [127, 128, 129]),
])
def test_prompts(ctx, H, Hkv, D, lens, news, dtype):
    c = Case(ctx, lens, news, H, Hkv, D, "Q8_0", "Q8_0", dtype, 16, seed=len(lens))
    out = c.call()
    ctx.sync_status()
    c.check(out)


@pytest.mark.parametrize("news", [[1, 1, 1, 1], [6, 3, 1, 4], [260, 90, 17, 130]])
@pytest.mark.parametrize("opts", [dict(window=1), dict(window=50), dict(cap=5.0), dict(slopes=True), dict(scale=-0.3),
                                  dict(window=64, cap=30.0, slopes=True, scale=0.2)])
@pytest.mark.parametrize("dtype,D,v_type", [("f32", 64, "Q8_0"), ("bf16", 128, "Q4_0"), ("f16", 256, "Q8_0")])
def test_masks_caps_and_biases(ctx, dtype, D, v_type, opts, news):
    c = Case(ctx, [260, 333, 17, 500], news, 6, 2, D, "Q8_0", v_type, dtype, 16, seed=7)
    opts = dict(opts)
    if opts.get("slopes"):
        opts["slopes"] = torch.exp2(-1.0 - torch.arange(6, device="cuda"))
    out = c.call(**opts)
    ctx.sync_status()
    c.check(out, **opts)


@pytest.mark.parametrize("news", [[1, 1, 1], [200, 90, 333]])
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_peaked_scores(ctx, dtype, news):
    """Scores of a few hundred: one key takes all."""
    c = Case(ctx, [500, 90, 1200], news, 4, 2, 128, dtype=dtype, seed=3, q_mul=30.0)
    out = c.call()
    ctx.sync_status()
    c.check(out)


@pytest.mark.parametrize("news", [[1, 1], [40, 150]])
def test_strided_rows_and_another_stream(ctx, news):
    c = Case(ctx, [200, 170], news, 8, 2, 64, dtype="bf16", seed=5)
    n = sum(news)
    wide = torch.zeros((n, 3, 8, 96), dtype=torch.bfloat16, device="cuda")
    wide[:, 1, :, 32:] = c.q
    out = torch.full((8, n + 1, 64), 9.0, dtype=torch.bfloat16, device="cuda")
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    with torch.cuda.stream(s):
        c.call(q=wide[:, 1, :, 32:], out=out[:, :n].transpose(0, 1))
    s.synchronize()
    c.check(out[:, :n].transpose(0, 1))
    assert (out[:, n] == 9.0).all()


@pytest.mark.parametrize("news", [[1, 1, 1, 1], [3, 150, 1, 20]])
def test_graph_replay_follows_lengths_and_pages(ctx, news):
    c = Case(ctx, [300, 150, 64, 200], news, 8, 2, 64, dtype="bf16", seed=8)
    want = c.call(max_len=320)
    out = torch.zeros_like(want)
    g = torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(g):
        c.call(max_len=320, out=out)
    g.replay()
    torch.cuda.synchronize()
    assert torch.equal(out, want)
    # the same pages, two sequences exchanged: the captured launch reads the new tables and lengths
    swap = torch.tensor([0, 3, 2, 1], device="cuda")
    if max(news) == 1:
        c.table.copy_(c.table[swap].clone())
        c.dlens.copy_(c.dlens[swap].clone())
        c.q.copy_(c.q[swap].clone())
        g.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, want[swap])
    ctx.sync_status()


def test_places_beyond_32_bits(ctx):
    """A pool of more than 4 GiB whose last pages are the sequence's."""
    Hkv, D, page = 8, 128, 128
    n_pages = (1 << 32) // (Hkv * (page // 16) * 17 * D) + 20
    cache = ctx.kv_cache("Q8_0", "Q8_0", n_pages, page, Hkv, D)
    small = ctx.kv_cache("Q8_0", "Q8_0", 4, page, Hkv, D)
    n = 4 * page - 3
    k, v = (torch.randn((n, Hkv, D), device="cuda") for _ in range(2))
    q = torch.randn((200, 16, D), device="cuda")
    lens = torch.tensor([n], dtype=torch.int32, device="cuda")
    for first, pool in ((n_pages - 4, cache), (0, small)):
        ctx.kv_store(pool, k, v, first * page + torch.arange(n, device="cuda"))
    far = torch.arange(n_pages - 4, n_pages, dtype=torch.int32, device="cuda")[None]
    near = torch.arange(4, dtype=torch.int32, device="cuda")[None]
    for rows in (1, 200):
        start = torch.tensor([0, rows], dtype=torch.int32, device="cuda")
        a = ctx.attention(cache, q[:rows], lens, far, q_start=start)
        b = ctx.attention(small, q[:rows], lens, near, q_start=start)
        ctx.sync_status()
        assert torch.equal(a, b) and bool(torch.isfinite(a).all())


@pytest.mark.parametrize("news", [[1, 1], [40, 150]])
def test_bad_pages_and_lengths_are_reported(ctx, news):
    c = Case(ctx, [200, 170], news, 4, 2, 64, seed=6)
    c.call()
    ctx.sync_status()
    c.table[1, 2] = 10 ** 6
    c.call()
    with pytest.raises(ggq.GGQError, match="outside the key/value cache"):
        ctx.sync_status()
    c.table[1, 2] = 0
    c.call(max_len=199)
    with pytest.raises(ggq.GGQError, match="outside the key/value cache"):
        ctx.sync_status()
    ctx.sync_status()


def test_refusals(ctx):
    c = Case(ctx, [20, 30], [1, 1], 4, 2, 64, seed=9)
    att = ctx.attention
    with pytest.raises(ggq.GGQError, match="query heads"):
        att(c.cache, torch.zeros((2, 5, 64), device="cuda"), c.dlens, c.table)
    with pytest.raises(ValueError, match="tensor"):
        att(c.cache, torch.zeros((2, 4, 32), device="cuda"), c.dlens, c.table)
    with pytest.raises(ValueError, match="float32"):
        att(c.cache, c.q.double(), c.dlens, c.table)
    with pytest.raises(ValueError, match="q_start"):
        att(c.cache, torch.zeros((3, 4, 64), device="cuda"), c.dlens, c.table)
    with pytest.raises(ValueError, match="int32"):
        att(c.cache, c.q, c.dlens.long(), c.table)
    with pytest.raises(ValueError, match="table row"):
        att(c.cache, c.q, c.dlens, c.table[:1])
    with pytest.raises(ValueError, match="slopes"):
        att(c.cache, c.q, c.dlens, c.table, slopes=torch.zeros(3, device="cuda"))
    with pytest.raises(ValueError, match="q's type"):
        att(c.cache, c.q, c.dlens, c.table, out=c.q.half())
    with pytest.raises(ggq.GGQError, match="finite"):
        att(c.cache, c.q, c.dlens, c.table, scale=float("nan"))
    with pytest.raises(ggq.GGQError, match="multiples of 4"):
        att(c.cache, torch.zeros((2, 4, 66), device="cuda")[..., :64], c.dlens, c.table)
    assert att(c.cache, c.q[:0], c.dlens[:0], c.table[:0]).shape == (0, 4, 64)
    ctx.sync_status()
