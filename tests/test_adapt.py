"""ggq_adapt against the same in 64 bits: types, ranks, layouts of rows and sequences, shared adapters, and refusals.

Tolerance (fp32 sums of exact products; units of 2^-24 of the sum of magnitudes): a lane adds at most 16 products of
every 512 inputs, 5 joins of lanes, K / 512 steps and 32 parts of the inputs, the scale, then 8 products and 5 joins of
the outputs and the addition of y.  fp32 rows are three terms of 8 bits, whose products below the last bit are left out,
and so is A x: twelve units cover both."""
import ctypes

import pytest

torch = pytest.importorskip("torch")

import gguf_block_quant_ggq_gb300 as ggq  # noqa: E402

gpu = pytest.mark.gpu
DTYPES = [torch.float32, torch.float16, torch.bfloat16]
BANKS = [torch.bfloat16, torch.float16]


@pytest.fixture(scope="module")
def ctx():
    assert torch.cuda.is_available(), "GPU tests need a CUDA device"
    from gguf_block_quant_ggq_gb300 import _build
    _build.build()
    c = ggq.Context(0)
    yield c
    c.close()


class Case:
    def __init__(self, n, R, K, N, dtype, bank, seed=0, ranks=None):
        g = torch.Generator(device="cuda")
        g.manual_seed(seed + 31 * R + K)
        self.g, self.dtype, self.K, self.N, self.R = g, dtype, K, N, R
        self.a = (torch.randn((n, R, K), device="cuda", generator=g) * K ** -0.5).to(bank)
        self.b = torch.randn((n, N, R), device="cuda", generator=g).to(bank)
        self.ranks = None if ranks is None else torch.tensor(ranks, dtype=torch.int32, device="cuda")
        self.scales = torch.rand(n, device="cuda", generator=g) + 0.5

    def rows(self, T, pad=0):
        x = torch.randn((T, self.K + 4 * pad), device="cuda", generator=self.g).to(self.dtype)
        y = torch.randn((T, self.N + pad), device="cuda", generator=self.g).to(self.dtype)
        return x[:, 4 * pad:], y[:, pad:]

    def exact(self, x, y, ids, start=None):
        """(out, sum of magnitudes) in 64 bits; rows of no sequence: NaN."""
        start = start or list(range(len(ids) + 1))
        out, mag = torch.full(y.shape, float("nan"), dtype=torch.float64, device="cuda"), y.double().abs()
        for i, a in enumerate(ids):
            s = slice(start[i], start[i + 1])
            out[s] = y[s].double()
            if a < 0 or a >= self.a.shape[0] or start[i] == start[i + 1]:
                continue
            r = self.R if self.ranks is None else int(self.ranks[a])
            A, B, sc = self.a[a, :r].double(), self.b[a, :, :r].double(), float(self.scales[a])
            out[s] += sc * ((x[s].double() @ A.T) @ B.T)
            mag[s] += sc * ((x[s].double().abs() @ A.abs().T) @ B.abs().T)
        return out, mag

    def check(self, got, x, y, ids, start=None):
        want, mag = self.exact(x, y, ids, start)
        there = ~want.isnan()
        units = 16 + 5 + self.K / 512 + 32 + 1 + 8 + 5 + 1 + (12 if self.dtype is torch.float32 else 0)
        off = units * 2.0 ** -24 * mag
        if self.dtype is not torch.float32:
            off = off + (want.abs() + off) * torch.finfo(self.dtype).eps / 2 + 2.0 ** -25
        err = (got.double() - want).abs()
        assert bool((err <= off)[there].all()), float((err / off)[there].max())


def ints(a):
    return torch.tensor(a, dtype=torch.int32, device="cuda")


@gpu
@pytest.mark.parametrize("bank", BANKS)
@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("R,K,N", [(8, 8, 1), (8, 256, 33), (16, 4096, 1000), (24, 1032, 100), (32, 2048, 64), (64, 4096, 515),
                                   (128, 520, 96), (256, 264, 37), (4, 512, 40), (13, 14336, 64)])
def test_single_tokens(ctx, dtype, bank, R, K, N):
    c = Case(5, R, K, N, dtype, bank, ranks=[R, 1, (R + 1) // 2, R, 0])
    ad = ctx.adapters(c.a, c.b, ranks=c.ranks, scales=c.scales)
    for ids in ([0], [2, 2, -1, 1], [3] * 9 + [4, 0], [i * i % 5 for i in range(40)] + [-7], [1] * 300 + [2], [i * i % 6 - 1 for i in range(261)]):
        x, y = c.rows(len(ids), pad=1)
        got = ctx.adapt(ad, x, y, ints(ids))
        c.check(got, x, y, ids)
        same = y.clone()
        ctx.adapt(ad, x, same, ints(ids), out=same)
        assert torch.equal(same, got)
    ctx.sync_status()


@gpu
@pytest.mark.parametrize("bank", BANKS)
@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("R,K,N", [(8, 64, 8), (16, 1024, 260), (32, 4096, 77), (64, 520, 128), (128, 1032, 200), (256, 512, 64), (20, 256, 129)])
def test_ragged_sequences(ctx, dtype, bank, R, K, N):
    c = Case(4, R, K, N, dtype, bank, ranks=[R, R // 2, 3, R])
    ad = ctx.adapters(c.a, c.b, ranks=c.ranks, scales=c.scales)
    for lens, ids in (([1], [0]), ([8, 9, 0, 1], [1, 2, 3, 0]), ([300], [3]), ([63, 64, 65, 128, 2], [0, -1, 3, 1, 3]), ([17] * 30, [i % 5 - 1 for i in range(30)]),
                      ([0, 0, 129], [0, 1, 2])):
        start = [sum(lens[:i]) for i in range(len(lens) + 1)]
        x, y = c.rows(start[-1] + 3, pad=3)  # three rows behind the last sequence
        out = torch.full((start[-1] + 3, c.N), 9.0, device="cuda", dtype=dtype)
        got = ctx.adapt(ad, x, y, ints(ids), q_start=ints(start), out=out)
        assert got is out and bool((out[start[-1]:] == 9).all())
        c.check(out[:start[-1]], x[:start[-1]], y[:start[-1]], ids, start)
        same = y.clone()
        ctx.adapt(ad, x, same, ints(ids), q_start=ints(start), out=same)
        assert torch.equal(same[:start[-1]], out[:start[-1]]) and torch.equal(same[start[-1]:], y[start[-1]:])
    ctx.sync_status()


@gpu
@pytest.mark.parametrize("bank", BANKS)
@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("R,K,N", [(8, 72, 40), (16, 1024, 260), (32, 520, 77), (64, 4096, 128), (128, 1032, 200), (77, 264, 65), (256, 512, 64)])
def test_long_prompts(ctx, dtype, bank, R, K, N):
    """From some hundred rows on: groups of 16 rows on four CTAs, then tiles of 32."""
    c = Case(3, R, K, N, dtype, bank, ranks=[R, (R + 1) // 2, max(1, R - 3)])
    ad = ctx.adapters(c.a, c.b, ranks=c.ranks, scales=c.scales)
    for lens, ids in (([480], [0]), ([150, 0, 33, 417], [2, 0, 1, 0]), ([1300], [2]), ([31, 700, 64, 1, 900], [0, 1, -1, 2, 0]), ([2400], [1])):
        start = [sum(lens[:i]) for i in range(len(lens) + 1)]
        x, y = c.rows(start[-1] + 2, pad=1)
        out = torch.full((start[-1] + 2, c.N), 9.0, device="cuda", dtype=dtype)
        ctx.adapt(ad, x, y, ints(ids), q_start=ints(start), out=out)
        assert bool((out[start[-1]:] == 9).all())
        c.check(out[:start[-1]], x[:start[-1]], y[:start[-1]], ids, start)
        same = y.clone()
        ctx.adapt(ad, x, same, ints(ids), q_start=ints(start), out=same)
        assert torch.equal(same[:start[-1]], out[:start[-1]]) and torch.equal(same[start[-1]:], y[start[-1]:])
    ctx.sync_status()


@gpu
@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("R", [16, 64, 96, 160])
@pytest.mark.parametrize("n", [20, 45, 90])
def test_many_adapters(ctx, dtype, R, n):
    """Single tokens and short sequences of more adapters than SMs take at once."""
    c = Case(n, R, 520, 100, dtype, torch.bfloat16, ranks=[R if i % 3 else R // 2 for i in range(n)])
    ad = ctx.adapters(c.a, c.b, ranks=c.ranks, scales=c.scales)
    ids = [(7 * i) % (n + 1) - 1 for i in range(200)]
    x, y = c.rows(200)
    c.check(ctx.adapt(ad, x, y, ints(ids)), x, y, ids)
    start = [4 * i for i in range(51)]
    c.check(ctx.adapt(ad, x, y, ints(ids[:50]), q_start=ints(start)), x, y, ids[:50], start)
    ctx.sync_status()


@gpu
@pytest.mark.parametrize("T", [3, 200])
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_what_stands_behind_a_rank_is_not_used(ctx, dtype, T):
    c = Case(2, 24, 512, 70, dtype, torch.bfloat16, ranks=[5, 16])
    c.a[0, 5:], c.b[0, :, 5:] = float("nan"), float("inf")
    c.a[1, 16:], c.b[1, :, 16:] = float("inf"), float("nan")
    ad = ctx.adapters(c.a, c.b, ranks=c.ranks, scales=c.scales)
    x, y = c.rows(2 * T)
    c.check(ctx.adapt(ad, x, y, ints([0, 1]), q_start=ints([0, T, 2 * T])), x, y, [0, 1], [0, T, 2 * T])
    c.check(ctx.adapt(ad, x, y, ints([0, 1] * T)), x, y, [0, 1] * T)


@gpu
@pytest.mark.parametrize("T", [2, 200])
def test_values_that_are_not_finite_stay_in_their_row(ctx, T):
    c = Case(1, 16, 512, 64, torch.float32, torch.bfloat16)
    ad = ctx.adapters(c.a, c.b)
    x, y = c.rows(2 * T)
    want = ctx.adapt(ad, x, y, ints([0]), q_start=ints([0, 2 * T]))
    x[1, 3], y[0, 5] = float("nan"), float("inf")
    got = ctx.adapt(ad, x, y, ints([0]), q_start=ints([0, 2 * T]))
    assert bool(got[1].isnan().all()) and float(got[0, 5]) == float("inf")
    want[1], want[0, 5] = got[1], got[0, 5]
    assert torch.equal(got.nan_to_num(), want.nan_to_num())


@gpu
@pytest.mark.parametrize("T", [1, 100])
def test_large_and_small_fp32_values(ctx, T):
    """Rows of very different size: products keep their bits whatever the exponents are."""
    c = Case(1, 16, 1024, 64, torch.float32, torch.float16)
    ad = ctx.adapters(c.a, c.b, scales=c.scales)
    x, y = c.rows(T)
    x = x * torch.exp2(torch.randint(-60, 61, (T, 1), device="cuda", generator=c.g).float())
    y = torch.zeros_like(y)
    c.check(ctx.adapt(ad, x, y, ints([0]), q_start=ints([0, T])), x, y, [0], [0, T])


@gpu
def test_outside_ids_and_ranges(ctx):
    c = Case(2, 8, 64, 40, torch.float32, torch.float16)
    ad = ctx.adapters(c.a, c.b, scales=c.scales)
    x, y = c.rows(3)
    got = ctx.adapt(ad, x, y, ints([0, 2, 1]))
    with pytest.raises(ggq.GGQError, match="adapter"):
        ctx.sync_status()
    c.check(got, x, y, [0, -1, 1])
    for start, cut in (([0, 2, 9], [0, 2, 3]), ([-4, 1, 3], [0, 1, 3])):
        out = torch.zeros_like(y)
        ctx.adapt(ad, x, y, ints([0, 1]), q_start=ints(start), out=out)
        with pytest.raises(ggq.GGQError, match="row range"):
            ctx.sync_status()
    ctx.sync_status()


@gpu
def test_results_do_not_depend_on_the_company(ctx):
    """A row's value is the same in any order of the batch (single tokens)."""
    c = Case(3, 32, 1024, 300, torch.bfloat16, torch.bfloat16)
    ad = ctx.adapters(c.a, c.b)
    ids = [0, 1, 0, 2, 0, 0, 1, 0, 0, 0, 0, 0]
    x, y = c.rows(len(ids))
    first = ctx.adapt(ad, x, y, ints(ids))
    again = ctx.adapt(ad, x, y, ints(ids))
    assert torch.equal(first, again)
    order = [5, 11, 0, 3, 1, 2, 4, 6, 7, 8, 9, 10]
    assert torch.equal(ctx.adapt(ad, x[order].contiguous(), y[order].contiguous(), ints([ids[i] for i in order])), first[order])


@gpu
def test_refusals(ctx):
    c = Case(2, 8, 64, 40, torch.float32, torch.bfloat16)
    ad = ctx.adapters(c.a, c.b)
    x, y = c.rows(4)
    ids = ints([0, 1, 0, 1])
    for bad in (dict(x=x[:3]), dict(x=x.half()), dict(y=y[:, :39]), dict(y=y[:3]), dict(ids=ids[:3]), dict(ids=ids.long()), dict(q_start=ids),
                dict(out=y.half()), dict(x=x.double()), dict(x=x[:, :32]), dict(y=y.t().contiguous().t())):
        with pytest.raises(ValueError):
            ctx.adapt(**{**dict(adapters=ad, x=x, y=y, ids=ids), **bad})
    for bad in (dict(a=c.a.float(), b=c.b.float()), dict(a=c.a.half()), dict(a=c.a[:1]), dict(b=c.b[:, :, :4]), dict(a=c.a[0]), dict(ranks=ints([1])),
                dict(scales=c.scales.half()), dict(a=c.a.cpu())):
        with pytest.raises((ValueError, RuntimeError)):
            ctx.adapters(**{**dict(a=c.a, b=c.b), **bad})
    wide = torch.zeros((4, 68), device="cuda")
    with pytest.raises(ggq.GGQError, match="multiples of 4"):
        ctx.adapt(ad, wide[:, 1:65], y, ids)
    with pytest.raises(ggq.GGQError, match="must not be x"):
        square = ctx.adapters(c.a, torch.zeros((2, 64, 8), device="cuda").bfloat16())
        ctx.adapt(square, x, x, ids, out=x)
    with pytest.raises(ggq.GGQError, match="one stride"):
        big = torch.zeros((8, 40), device="cuda")
        ctx.adapt(ad, x, big[:4], ids, out=big[::2][:4])
    with pytest.raises(ggq.GGQError, match="multiple of 8"):
        ctx.adapt(ctx.adapters(torch.zeros((1, 8, 60), device="cuda").half(), torch.zeros((1, 40, 8), device="cuda").half()), wide[:, :60], y, ids)
    with pytest.raises(ggq.GGQError, match="at most 256"):
        ctx.adapt(ctx.adapters(torch.zeros((1, 264, 64), device="cuda").half(), torch.zeros((1, 40, 264), device="cuda").half()), x, y, ids)
    mine = ctx.adapters(c.a, c.b)
    mine.device = 1
    with pytest.raises(ValueError, match="cuda:1"):
        ctx.adapt(mine, x, y, ids)
    assert ctx.adapt(ad, x[:0], y[:0], ids[:0]).shape == (0, 40)
    ctx.sync_status()


def test_null_context():
    assert ggq.load().ggq_adapt(None, ctypes.byref(ggq.ggq_adapters()), ctypes.byref(ggq.ggq_adapt_args()), None) == 1
