"""ggq_norm against the same in 64 bits, its packed rows against ggq_quantize_act, and its refusals.

Tolerances (units of 2^-24, relative): a sum of squares passes at most 8 * 4 multiply-adds a thread and 10 joins,
each off by one, so the inverse root by half of 42, and rsqrtf by 4; then come at most 6 products and, with a
sigmoid, 8.  The total is off by 40 such units of its second term and one of itself; the second norm adds 40 of
itself and what the errors of the total do to the row's length."""
import ctypes

import pytest

torch = pytest.importorskip("torch")

import gguf_block_quant_ggq_gb300 as ggq  # noqa: E402

gpu = pytest.mark.gpu
U = 2.0 ** -24
DTYPES = [torch.float32, torch.float16, torch.bfloat16]


@pytest.fixture(scope="module")
def ctx():
    assert torch.cuda.is_available(), "GPU tests need a CUDA device"
    from gguf_block_quant_ggq_gb300 import _build
    _build.build()
    c = ggq.Context(0)
    yield c
    c.close()


def half_step(t, dtype):
    """Rounding of the values t (64 bits) to dtype."""
    if dtype is torch.float32:
        return t.abs() * 0.0
    return t.abs() * torch.finfo(dtype).eps / 2 + (2.0 ** -25 if dtype is torch.float16 else 0.0)


def formula(x, after, gate, sigmoid, scale, residual, before, eps, offset):
    """(out, total) in 64 bits and what the kernel's may be off by, before rounding."""
    u = x.double()
    if after is not None:
        w = 1.0 if after is True else after.double() + offset
        u = u * torch.rsqrt(u.square().mean(1, keepdim=True) + eps) * w
    if gate is not None:
        u = u * (torch.sigmoid(gate.double()) if sigmoid else gate.double())
    u = u * scale
    t = u + residual.double() if residual is not None else u
    off = 40 * U * u.abs() + U * t.abs()
    if before is None:
        return None, t, None, off
    inv = torch.rsqrt(t.square().mean(1, keepdim=True) + eps)
    w = 1.0 if before is True else before.double() + offset
    out = t * inv * w
    far = off.norm(dim=1, keepdim=True) / t.norm(dim=1, keepdim=True).clamp(min=1e-300)
    return out, t, off * (inv * w).abs() + out.abs() * (40 * U + far), off


def check(got, want, off, dtype):
    assert got.dtype is dtype
    err = (got.double() - want).abs()
    room = off * 1.01 + half_step(want.abs() + off, dtype) + 1e-40
    assert bool((err <= room).all()), float((err / room).max())


@gpu
@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("rows,width", [(1, 1), (3, 7), (5, 64), (9, 256), (1, 4096), (130, 264), (33, 1000), (7, 2051), (2, 4104),
                                        (2, 8192), (3, 8200), (2, 12289), (2, 16384), (1, 20000), (2, 32768)])
def test_against_64_bits(ctx, dtype, rows, width):
    g = torch.Generator(device="cuda")
    g.manual_seed(rows * 131 + width)
    rn = lambda *s: torch.randn(s, device="cuda", generator=g)  # noqa: E731
    size = torch.exp(rn(width))
    x, res = (rn(rows, width) * size).to(dtype), (rn(rows, width) * 4 * size).to(dtype)
    wa, wb = 0.3 * rn(width), 0.3 * rn(width)
    gates = [None, rn(rows, width).to(dtype), rn(width).to(dtype), rn(rows, 1).to(dtype)]
    for i, (after, before, residual) in enumerate([(None, wb, None), (None, True, res), (wa, None, res), (wa, wb, res), (True, None, None),
                                                   (None, None, res)]):
        gate, act = gates[(i + width) % 4], "sigmoid" if i % 2 else "none"
        out, total = ctx.norm(x, before=before, after=after, gate=gate, gate_act=act, scale=0.3, residual=residual, eps=1e-5, offset=1.0)
        want, t, off_out, off_t = formula(x, after, gate, act == "sigmoid", 0.3, residual, before, 1e-5, 1.0)
        assert (out is None) == (before is None) and (total is None) == (residual is None and before is not None)
        if total is not None:
            check(total, t, off_t, dtype)
        if out is not None:
            check(out, want, off_out, dtype)
    ctx.sync_status()


@gpu
@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("pad,shift", [(8, 0), (3, 1)])  # aligned rows inside wider ones, and rows at any element
def test_strided_rows_and_outputs_in_place(ctx, dtype, pad, shift):
    g = torch.Generator(device="cuda")
    g.manual_seed(5)
    n, H = 6, 520

    def rows():
        wide = torch.full((n, H + pad + 8), 7.0, device="cuda", dtype=dtype)
        part = wide[:, shift:shift + H]
        part.copy_(torch.randn((n, H), device="cuda", generator=g))
        return wide, part
    (wx, x), (wr, res), (wo, out) = rows(), rows(), rows()
    w = torch.rand(H, device="cuda", generator=g)
    want, total = torch.empty_like(wo)[:, shift:shift + H], torch.empty_like(wo)[:, shift:shift + H]
    ctx.norm(x, before=w, after=w, residual=res, out=want, total=total)
    exact, t, off_out, off_t = formula(x, w, None, False, 1.0, res, w, 1e-6, 0.0)
    check(want, exact, off_out, dtype)
    check(total, t, off_t, dtype)
    assert ctx.norm(x, before=w, after=w, residual=res, out=out, total=res)[1] is res  # the residual is updated
    assert torch.equal(out, want) and torch.equal(res, total)
    assert ctx.norm(res, before=w, out=x)[0] is x  # the second norm of the same rows elsewhere, and in place
    ctx.norm(res, before=w, out=res)
    assert torch.equal(res, x)
    for wide in (wx, wr, wo):  # nothing beside the rows
        assert bool((wide[:, :shift] == 7).all()) and bool((wide[:, shift + H:] == 7).all())


@gpu
@pytest.mark.parametrize("act", ["Q8_K", "Q8_1", "Q8_0"])
@pytest.mark.parametrize("rows,width", [(1, 256), (5, 2048), (3, 4096), (2, 8448), (3, 17408), (1, 32768), (4, 32), (2, 288), (3, 1056)])
def test_packed_rows_are_the_quantizers(ctx, act, rows, width):
    if act == "Q8_K" and width % 256:
        pytest.skip("whole blocks only")
    g = torch.Generator(device="cuda")
    g.manual_seed(width)
    x, res = torch.randn((2, rows, width), device="cuda", generator=g).unbind(0)
    res[0, :32] = 0.0
    x[0, :32] = 0.0  # a block of zeros
    w = torch.randn(width, device="cuda", generator=g)
    rows32, total = ctx.norm(x, before=w, residual=res)
    both = torch.empty_like(rows32)
    packed, total2 = ctx.norm(x, before=w, residual=res, act=act, out=both)
    alone, _ = ctx.norm(x, before=w, residual=res, act=act)
    want = ctx.quantize_act(act, rows32)
    assert torch.equal(both, rows32) and torch.equal(total, total2)
    assert torch.equal(packed, want) and torch.equal(alone, want)
    # 16-bit rows: the blocks are of the unrounded fp32 rows
    half = ctx.norm(x.half(), before=w, residual=res.half(), act=act)[0]
    assert torch.equal(half, ctx.norm(x.half().float(), before=w, residual=res.half().float(), act=act)[0])


@gpu
def test_packed_rows_feed_the_products(ctx):
    import ggq_synth as syn
    W = torch.from_numpy(syn.weights("Q4_K", 96, 512, syn.rng(3, 0))).cuda()
    x = torch.randn((3, 512), device="cuda")
    rows, _ = ctx.norm(x, before=True)
    packed, _ = ctx.norm(x, before=True, act="Q8_K")
    assert torch.equal(ctx.mul_mat_vec_q("Q4_K", W, 96, 512, packed, 3), ctx.mul_mat_vec("Q4_K", W, 96, 512, rows))


@gpu
def test_zeros_nan_and_no_tokens(ctx):
    x = torch.zeros((3, 128), device="cuda")
    assert bool((ctx.norm(x, before=True)[0] == 0).all())
    assert bool((ctx.norm(x, before=True, eps=0.0)[0]).isnan().all())  # 0 * inf
    x[1, 5] = float("nan")
    x[2, 7] = float("inf")
    y = ctx.norm(x, before=True)[0]
    assert bool((y[0] == 0).all()) and bool(y[1].isnan().all()) and bool(y[2, 7].isnan())
    out, total = ctx.norm(x[:0], before=True, residual=x[:0])
    assert out.shape == (0, 128) and total.shape == (0, 128)


@gpu
def test_refusals(ctx):
    x = torch.zeros((2, 256), device="cuda")
    w = torch.ones(256, device="cuda")
    for bad in (dict(before=w[:255]), dict(before=w.half()), dict(residual=x[:1]), dict(residual=x.half()), dict(before=w, out=x.half()),
                dict(gate=x[:, :3]), dict(out=x), dict(act="Q8_K"), dict(residual=x.t().contiguous().t()), dict(residual=x.cpu())):
        with pytest.raises(ValueError):
            ctx.norm(x, **bad)
    with pytest.raises(ValueError):
        ctx.norm(x.double(), before=w)
    for bad, status in ((dict(before=w, scale=float("nan")), 1), (dict(before=w, eps=-1.0), 1), (dict(before=w, act="Q8_K"), 0),
                        (dict(before=w, act="Q4_K"), 3)):
        if status:
            with pytest.raises(ggq.GGQError) as e:
                ctx.norm(x, **bad)
            assert e.value.status == status
    with pytest.raises(ggq.GGQError, match="a place each"):
        ctx.norm(x, before=w, out=x, total=x)
    wide = torch.zeros((4, 256), device="cuda")
    for bad in (dict(total=wide[:2]), dict(before=w, out=wide[:2]), dict(residual=wide[:2], total=wide[::2])):
        with pytest.raises(ggq.GGQError, match="one stride"):
            ctx.norm(wide[::2], **bad)
    odd = torch.zeros((2, 264), device="cuda")[:, 1:257]
    with pytest.raises(ggq.GGQError, match="16 bytes"):
        ctx.norm(odd, before=True, act="Q8_K")
    with pytest.raises(ggq.GGQError, match="block"):
        ctx.norm(torch.zeros((1, 48), device="cuda"), before=True, act="Q8_1", packed=torch.zeros((1, 36), dtype=torch.uint8, device="cuda"))
    with pytest.raises(ggq.GGQError, match="32768"):
        ctx.norm(torch.zeros((1, 32776), device="cuda"), before=True)
    ctx.sync_status()


def test_null_context():
    assert ggq.load().ggq_norm(None, ctypes.byref(ggq.ggq_norm_args()), None) == 1
