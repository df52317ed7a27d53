"""ggq_logprobs against 64 bits: values, ids in order with ties, masks that leave little or nothing, odd rows, refusals.

Tolerance: the sum of exponentials passes at most V / (512 parts) + 60 additions (units of 2^-24); an exponential is off
by 2^-22 and by three units of its argument z = scale (x - max), whose mean is the row's mean |z|; that is an absolute
error of the sum's logarithm.  log p adds two units of |z| and of the logarithm, the entropy twice all of that, once for
each of its two sums, weighted with 1 + mean |z|."""
import ctypes
import math

import pytest

torch = pytest.importorskip("torch")

import gguf_block_quant_ggq_gb300 as ggq  # noqa: E402

gpu = pytest.mark.gpu
DTYPES = [torch.float32, torch.float16, torch.bfloat16]
U = 2.0 ** -24


@pytest.fixture(scope="module")
def ctx():
    assert torch.cuda.is_available(), "GPU tests need a CUDA device"
    from gguf_block_quant_ggq_gb300 import _build
    _build.build()
    c = ggq.Context(0)
    yield c
    c.close()


def check(ctx, x, tokens, top, scale=1.0):
    lp, ent, ids, best = ctx.logprobs(x, tokens, top_k=top, scale=scale)
    V = x.shape[1]
    z = x.double() * scale
    z = z - z.amax(1, keepdim=True)
    e = z.exp()
    S = e.sum(1, keepdim=True)
    mean = torch.where(e > 0, -z * e, 0.0).sum(1, keepdim=True) / S
    log = S.log()
    room = (V / 512 + 60 + 4 + 3 * mean) * U  # of log S
    want = z.gather(1, tokens.long().view(len(x), -1)) - log

    def near(got, want, z, what):
        err = torch.where(got.double() == want, 0.0, (got.double() - want).abs())
        far = room + 2 * U * (z.abs().nan_to_num(posinf=0.0) + log.abs()) + U * want.abs().nan_to_num(posinf=0.0)
        assert bool((err <= far).all()), (what, float((err / far).max()))
    near(lp.view(len(x), -1), want, want + log, "given")
    near(ent[:, None], log + mean, 2 * mean + (V / 512 + 64 + 3 * mean) * (1 + mean), "entropy")
    if top:
        order = x.float().sort(dim=1, descending=True, stable=True).indices[:, :top]
        assert torch.equal(ids, order.int())
        near(best, z.gather(1, order) - log, z.gather(1, order), "alternatives")
    else:
        assert ids is None and best is None
    return lp, ent, ids, best


def logits(n, V, dtype, seed, pad=0):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return (torch.randn((n, V + pad), device="cuda", generator=g) * 2.5).to(dtype)[:, pad:], g


@gpu
@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("n,V", [(1, 1), (3, 5), (2, 31), (7, 257), (5, 1000), (1, 8192), (2, 32003), (160, 4099), (1, 131072), (3, 262143),
                                 (400, 20001), (20, 50257)])
def test_against_64_bits(ctx, dtype, n, V):
    x, g = logits(n, V, dtype, V + n, pad=3 if V % 2 else 0)
    for top, scale in ((0, 1.0), (1, 0.5), (min(5, V), 1.0), (min(32, V), 2.0)):
        tokens = torch.randint(0, V, (n, 3), device="cuda", generator=g, dtype=torch.int32)
        check(ctx, x, tokens, top, scale)
    ctx.sync_status()


@gpu
@pytest.mark.parametrize("dtype", DTYPES)
def test_every_alignment_of_a_row(ctx, dtype):
    for shift in range(9):
        x, _ = logits(3, 700, dtype, shift, pad=shift)
        check(ctx, x, torch.tensor([[0], [699], [350]], dtype=torch.int32, device="cuda"), 20)


@gpu
@pytest.mark.parametrize("top", [1, 7, 20, 32])
def test_ties_and_orders(ctx, top):
    tokens = torch.zeros((4, 1), dtype=torch.int32, device="cuda")
    for V in (40, 5000, 70001):
        i = torch.arange(V, device="cuda")
        x = torch.stack([torch.zeros(V, device="cuda"), (i % 13).float(), -i.float() / 64, i.float() / 64])
        x[0, V // 2] = -0.0  # as large as 0
        check(ctx, x, tokens, top)
        check(ctx, x.flip(1).contiguous(), tokens, top)


@gpu
@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("low", ["-inf", "lowest"])
def test_masks(ctx, dtype, low):
    V = 9001
    x, _ = logits(6, V, dtype, 4)
    value = -math.inf if low == "-inf" else torch.finfo(dtype).min
    keep = [[8000], [5, 6, 7000], list(range(4000, 4010)), [V - 1], [0], list(range(V))]
    for r, ids in enumerate(keep):
        m = torch.full((V,), value, device="cuda", dtype=dtype)
        m[ids] = x[r, ids]
        x[r] = m
    tokens = torch.tensor([[k[0], 17] for k in keep], dtype=torch.int32, device="cuda")
    lp, ent, ids, best = check(ctx, x, tokens, 8)
    assert float(lp[0, 0]) == 0.0 and float(ent[0]) == 0.0 and int(ids[0, 0]) == 8000
    assert [int(i) for i in ids[0, 1:]] == list(range(7))  # the lowest ids among what is left out
    ctx.sync_status()


@gpu
def test_rows_without_a_finite_value(ctx):
    V = 3001
    x = torch.full((5, V), -math.inf, device="cuda")
    x[1] = torch.finfo(torch.float32).min  # all alike
    x[2, 7] = math.inf
    x[3] = math.nan
    x[4] = torch.linspace(-1, 1, V)
    x[4, 5:9] = math.nan
    tokens = torch.tensor([3, 4, 7, 1, 6], dtype=torch.int32, device="cuda")
    lp, ent, ids, best = ctx.logprobs(x, tokens, top_k=4)
    assert float(lp[0]) == -math.inf and float(ent[0]) == 0.0 and ids[0].tolist() == [0, 1, 2, 3] and bool((best[0] == -math.inf).all())
    assert abs(float(lp[1]) + math.log(V)) < 1e-5 and abs(float(ent[1]) - math.log(V)) < 1e-5 and ids[1].tolist() == [0, 1, 2, 3]
    assert math.isnan(float(lp[2])) and math.isnan(float(ent[2])) and int(ids[2, 0]) == 7
    assert float(lp[3]) == -math.inf and float(ent[3]) == 0.0 and ids[3].tolist() == [0, 1, 2, 3]
    # a NaN counts as left out
    y = x[4].clone()
    y[5:9] = -math.inf
    want = ctx.logprobs(y[None], tokens[4:], top_k=4)
    assert float(lp[4]) == -math.inf
    assert torch.equal(ent[4], want[1][0]) and torch.equal(ids[4], want[2][0]) and torch.equal(best[4], want[3][0])
    ctx.sync_status()


@gpu
def test_tokens_outside(ctx):
    x, _ = logits(3, 100, torch.float32, 1)
    tokens = torch.tensor([[-1, 5], [100, 6], [7, -100]], dtype=torch.int32, device="cuda")
    lp = ctx.logprobs(x, tokens)[0]
    with pytest.raises(ggq.GGQError, match="vocabulary"):
        ctx.sync_status()
    assert float(lp[0, 0]) == 0 and float(lp[1, 0]) == 0 and float(lp[2, 1]) == 0
    assert torch.equal(lp[0, 1], ctx.logprobs(x, tokens[:, 1].contiguous().clamp(min=0))[0][0])
    ctx.sync_status()


@gpu
def test_many_given_tokens_and_nothing_given(ctx):
    x, g = logits(2, 5000, torch.bfloat16, 8)
    tokens = torch.randint(0, 5000, (2, 1000), device="cuda", generator=g, dtype=torch.int32)
    check(ctx, x, tokens, 3)
    lp, ent, ids, best = ctx.logprobs(x, top_k=2)
    assert lp is None and ids.shape == (2, 2)
    assert ctx.logprobs(x[:0], tokens[:0], top_k=2)[0].shape == (0, 1000)


@gpu
def test_refusals(ctx):
    x = torch.zeros((2, 64), device="cuda")
    t = torch.zeros((2, 1), dtype=torch.int32, device="cuda")
    f = torch.zeros((2, 1), device="cuda")
    for bad in (dict(logits=x[0]), dict(logits=x.double()), dict(logits=x.t().contiguous().t()), dict(tokens=t.long()), dict(tokens=t[:1]),
                dict(logprobs=f[:1]), dict(logprobs=f.half()), dict(entropy=f.view(-1)[:1]), dict(ids=t), dict(top=f), dict(top_k=2, ids=t),
                dict(tokens=None, logprobs=f), dict(logits=x.cpu())):
        with pytest.raises(ValueError):
            ctx.logprobs(**{**dict(logits=x, tokens=t), **bad})
    for bad in (dict(scale=0.0), dict(scale=-1.0), dict(scale=float("nan")), dict(top_k=33, ids=torch.zeros((2, 33), dtype=torch.int32, device="cuda")),
                dict(logits=x[:, :3].contiguous(), top_k=4)):
        with pytest.raises(ggq.GGQError):
            ctx.logprobs(**{**dict(logits=x, tokens=t), **bad})
    ctx.sync_status()


def test_null_context():
    assert ggq.load().ggq_logprobs(None, ctypes.byref(ggq.ggq_logprobs_args()), None) == 1
