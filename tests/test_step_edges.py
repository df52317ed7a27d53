"""Calls of a decoding step at the edges of what they take: alignments, streams, places, scales, sizes, precision."""
import math

import pytest

torch = pytest.importorskip("torch")

import test_adapt  # noqa: E402
import test_norm  # noqa: E402
import test_rotary  # noqa: E402
import gguf_block_quant_ggq_gb300 as ggq  # noqa: E402

pytestmark = pytest.mark.gpu
DTYPES = [torch.float32, torch.float16, torch.bfloat16]


@pytest.fixture(scope="module")
def ctx():
    assert torch.cuda.is_available(), "GPU tests need a CUDA device"
    from gguf_block_quant_ggq_gb300 import _build
    _build.build()
    c = ggq.Context(0)
    yield c
    c.close()


def ints(a):
    return torch.tensor(a, dtype=torch.int32, device="cuda")


def at(t, shift, pad=16):
    """The rows of t, `shift` elements behind 16 bytes, inside wider ones whose stride is a multiple of 16 elements."""
    rows, width = t.shape
    wide = torch.full((rows, (width + shift + pad) // 16 * 16 + 16), 5.0, device="cuda", dtype=t.dtype)
    part = wide[:, shift:shift + width]
    part.copy_(t)
    return part


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("R,K,N", [(16, 520, 1000), (64, 1032, 40), (72, 264, 520), (160, 264, 328)])
@pytest.mark.parametrize("shifts", [(4, 0, 0), (4, 4, 0), (0, 4, 0), (4, 0, 4), (4, 0, 1), (0, 1, 0), (12, 8, 8)])  # of x, y, out
def test_adapt_rows_of_each_alignment(ctx, dtype, R, K, N, shifts):
    """Rows of x at 8 bytes beside rows of y and out at 16, and the other way round: outputs of no whole block, and parts of
    the outputs shorter than a block."""
    c = test_adapt.Case(5, R, K, N, dtype, torch.bfloat16, ranks=[R, R // 2, R - 3, R, 8])
    ad = ctx.adapters(c.a, c.b, ranks=c.ranks, scales=c.scales)
    for lens, ids in (([1] * 3, [2, 0, -1]), ([1] * 70, [i * i % 6 - 1 for i in range(70)]), ([1] * 270, [i % 5 for i in range(270)]), ([37], [1]),
                      ([700, 0, 801], [3, 0, 2])):
        start = [sum(lens[:i]) for i in range(len(lens) + 1)]
        x, y = (at(t, s) for t, s in zip(c.rows(start[-1]), shifts))
        out = at(torch.zeros_like(y), shifts[2])
        q_start = None if max(lens) == 1 else ints(start)
        assert ctx.adapt(ad, x, y, ints(ids), q_start=q_start, out=out) is out
        c.check(out, x, y, ids, start)
        for t in (x, y, out):  # nothing beside the rows
            assert bool((t._base[:, t.shape[1] + t.storage_offset():] == 5).all())
    ctx.sync_status()


@pytest.mark.parametrize("rank", [4, 13, 16])
def test_adapters_are_ready_for_every_stream(ctx, rank):
    """Banks that are laid out anew while the current stream is busy, and a call on another stream right behind them."""
    c = test_adapt.Case(3, rank, 520, 96, torch.bfloat16, torch.float16)
    x, y = c.rows(9)
    ids = [0, 2, 1, 0, -1, 2, 2, 1, 0]
    which, s = ints(ids), torch.cuda.Stream()
    for given in (None, s):
        torch.cuda.synchronize()
        torch.cuda._sleep(50_000_000)  # some 25 ms
        ad = ctx.adapters(c.a, c.b, scales=c.scales, stream=given)
        got = ctx.adapt(ad, x, y, which, stream=s)
        torch.cuda.synchronize()
        c.check(got, x, y, ids)
    ctx.sync_status()


def test_adapters_new_layout_is_of_the_given_streams_memory(ctx):
    a, b = torch.ones((1, 9, 4096), device="cuda").half(), torch.ones((1, 65536, 9), device="cuda").half()
    s = torch.cuda.Stream()
    torch.cuda.synchronize()
    torch.cuda.empty_cache()
    ad = ctx.adapters(a, b, stream=s)
    where, size = ad.b.data_ptr(), ad.b.untyped_storage().nbytes()
    torch.cuda.synchronize()
    del ad
    with torch.cuda.stream(s):  # the block is the given stream's again
        assert torch.empty(size, dtype=torch.uint8, device="cuda").data_ptr() == where


def test_adapters_made_inside_a_capture(ctx):
    c = test_adapt.Case(2, 5, 264, 40, torch.float32, torch.bfloat16)
    x, y = c.rows(3)
    which = ints([1, 0, 1])
    ctx.adapt(ctx.adapters(c.a, c.b, scales=c.scales), x, y, which)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = ctx.adapt(ctx.adapters(c.a, c.b, scales=c.scales), x, y, which)
    for _ in range(2):
        c.a.copy_(c.a.flip(1))
        c.b.copy_(c.b * 0.5)
        graph.replay()
        c.check(got, x, y, [1, 0, 1])
    ctx.sync_status()


def same_bits(a, b):
    """Equal bit for bit, but for the bits inside a NaN."""
    whole = {4: torch.int32, 2: torch.int16}[a.element_size()]
    return torch.equal(a.isnan(), b.isnan()) and bool(((a.contiguous().view(whole) == b.contiguous().view(whole)) | a.isnan()).all())


@pytest.mark.parametrize("layout", ["half", "pairs"])
@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("D,turn,first", [(64, 64, 0), (128, 64, 64), (64, 24, 20), (64, 10, 3)])  # eight, four and one at once
def test_positions_outside_turn_nothing(ctx, dtype, layout, D, turn, first):
    """Rows of such positions come as they are: infinities, NaN and signs of zeros too."""
    table = ctx.rotary_table(10, turn)
    g = torch.Generator(device="cuda")
    g.manual_seed(turn)
    x = torch.randn((6, 5, D), device="cuda", generator=g).to(dtype)
    odd = torch.tensor([math.inf, -math.inf, math.nan, -0.0, 0.0, -1.0], device="cuda").to(dtype)
    x[1:5] = torch.where(torch.rand((4, 5, D), device="cuda", generator=g) < 0.4, odd[torch.randint(0, 6, (4, 5, D), device="cuda", generator=g)], x[1:5])
    pos = ints([3, 10, -1, 2 ** 31 - 1, -2 ** 31, 9])
    want = test_rotary.turned(x, table, pos, layout, first).to(dtype)
    want[1:5] = x[1:5]
    assert same_bits(ctx.rotate(x, table, pos, layout=layout, first=first), want)
    y = x.clone()
    ctx.rotate(y, table, pos, layout=layout, first=first, out=y)
    assert same_bits(y, want)
    # queries on the way into the cache; padded rows are not reported
    cache = ctx.kv_cache("Q8_0", "Q8_0", 1, 16, 5, D)
    slots = torch.tensor([0, -1, -1, -1, -1, 5], device="cuda")
    keys = torch.zeros_like(x)
    with pytest.raises(ggq.GGQError, match="position"):
        ctx.sync_status()
    assert same_bits(ctx.kv_append(cache, keys, keys, slots, table, pos, layout=layout, first=first, q=x), want)
    ctx.sync_status()


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("V", [5, 5000, 131072])
def test_logprobs_at_the_ends_of_the_scale(ctx, dtype, V):
    """Scales whose product with log2(e) leaves fp32: the largest logits alone remain; and scales that leave them all alike."""
    x = ((torch.arange(V, device="cuda") * 7919) % V).to(torch.float32).div(V).to(dtype)[None].repeat(2, 1)
    x[0, V // 2], x[1, 1], x[1, V - 2] = 3.0, 3.0, 3.0
    tokens = ints([[V // 2, 0], [V - 2, 2]])
    for scale in (1e30, 2.35e38, 2.5e38, 3.4e38):
        lp, ent, ids, top = ctx.logprobs(x, tokens, top_k=2, scale=scale)
        # log p of the others is below -2 scale (rounded), the sums are 1 and 2 exactly
        assert lp[0, 0] == 0.0 and abs(float(lp[1, 0]) + math.log(2.0)) <= 2.0 ** -23 and bool((lp[:, 1].double() < -1.9 * scale).all())
        assert ent[0] == 0.0 and abs(float(ent[1]) - math.log(2.0)) <= 2.0 ** -23
        assert ids[0, 0] == V // 2 and ids[1].tolist() == [1, V - 2]
        assert top[0, 0] == 0.0 and float(top[0, 1]) < -1.9 * scale and float((top[1] + math.log(2.0)).abs().max()) <= 2.0 ** -23
    room = (V / 512 + 64) * 2.0 ** -24 + 2.0 ** -22 + 2.0 ** -23 * math.log(V)  # of a sum of ones, and its logarithm
    for scale in (1e-30, 1.2e-38, 1e-44):
        lp, ent, ids, top = ctx.logprobs(x, tokens, top_k=2, scale=scale)
        for t in (lp, top, -ent):
            assert float((t.double() + math.log(V)).abs().max()) <= room
        assert ids[0, 0] == V // 2 and ids[1].tolist() == [1, V - 2]
    ctx.sync_status()


def test_a_buffer_for_packed_rows_needs_their_format(ctx):
    """Given buffers are written or the call is refused: nothing is left as it was without a word."""
    x, w = torch.randn((3, 256), device="cuda"), torch.ones(256, device="cuda")
    packed = torch.zeros((3, ggq.row_bytes("Q8_K", 256)), dtype=torch.uint8, device="cuda")
    for more in (dict(before=w), dict(before=w, out=torch.empty_like(x)), dict(after=w), dict(residual=x)):
        with pytest.raises(ValueError, match="act"):
            ctx.norm(x, packed=packed, **more)
    assert not bool(packed.any())
    assert ctx.norm(x, before=w, act="Q8_K", packed=packed)[0] is packed and bool(packed.any())


def test_magnitudes_beyond_fp32_are_refused(ctx):
    """A table of infinities and of 0 times infinity is no table."""
    for magnitude in (1e39, -1e39, 3.4028236e38):
        with pytest.raises(ggq.GGQError, match="magnitude"):
            ctx.rotary_table(4, 8, magnitude=magnitude)
    assert bool(ctx.rotary_table(4, 8, magnitude=3e38).isfinite().all())
    ctx.sync_status()


def plans(n):
    """(lengths, adapters) whose rows go as one group, many groups, more groups than SMs take at once, prompts in tiles."""
    return [([1], [0]), ([1] * 40, [i % n for i in range(40)]), ([1] * 200, [i % n for i in range(200)]), ([1] * 300, [i % n for i in range(300)]),
            ([33, 100], [0, n - 1]), ([700, 800], [0, n - 1]), ([2500], [n - 1])]


@pytest.mark.parametrize("bank", [torch.bfloat16, torch.float16])
@pytest.mark.parametrize("R", [8, 64, 72, 128, 256])
@pytest.mark.parametrize("n", [2, 90])
def test_adapt_keeps_the_bits_of_fp32_rows(ctx, bank, R, n):
    """A one a rank and a one an output: the outputs are inputs.  Each of the two products may cut what its additions do not
    hold, 2^-23 of a value; a term of 8 bits less in either would show as up to 2^-18."""
    K, N = 264, 300
    g = torch.Generator(device="cuda")
    g.manual_seed(R)
    pick = torch.stack([torch.randperm(K, device="cuda", generator=g)[:R] for _ in range(n)])  # input of each rank
    a = torch.zeros((n, R, K), device="cuda", dtype=bank)
    a.scatter_(2, pick[:, :, None], 1.0)
    b = torch.zeros((n, N, R), device="cuda", dtype=bank)
    to = torch.randint(0, R, (n, N), device="cuda", generator=g)  # rank of each output
    b.scatter_(2, to[:, :, None], 1.0)
    ad = ctx.adapters(a, b)
    for lens, ids in plans(n):
        T = sum(lens)
        x, y = torch.randn((T, K), device="cuda", generator=g), torch.zeros((T, N), device="cuda")
        start = [sum(lens[:i]) for i in range(len(lens) + 1)]
        got = ctx.adapt(ad, x, y, ints(ids), q_start=None if max(lens) == 1 else ints(start))
        of = torch.repeat_interleave(torch.tensor(ids, device="cuda"), torch.tensor(lens, device="cuda"))
        want = x.gather(1, pick.gather(1, to)[of])
        off = ((got.double() - want.double()).abs() / want.double().abs()).max()
        assert float(off) <= 2.0 ** -22, (lens[:3], float(off) * 2 ** 24)
    ctx.sync_status()


@pytest.mark.parametrize("bank", [torch.bfloat16, torch.float16])
@pytest.mark.parametrize("R", [16, 64, 96, 256])
def test_adapt_sums_fp32_rows_in_fp32(ctx, bank, R):
    """A value passes at most 88 additions of 4096 inputs and their rank (the bound in test_adapt.py), each off by one unit of
    2^-24 of what is summed so far, whose mean square is at most the whole's: sqrt(88) units together, 5.6e-7."""
    c = test_adapt.Case(2, R, 4096, 256, torch.float32, bank)
    ad = ctx.adapters(c.a, c.b, scales=c.scales)
    for lens, ids in plans(2):
        start = [sum(lens[:i]) for i in range(len(lens) + 1)]
        x, y = c.rows(start[-1])
        y = torch.zeros_like(y)
        got = ctx.adapt(ad, x, y, ints(ids), q_start=None if max(lens) == 1 else ints(start))
        want, _ = c.exact(x, y, ids, start)
        off = float((got.double() - want).norm() / want.norm())
        assert off <= 5.6e-7, (lens[:3], off)
    ctx.sync_status()


@pytest.mark.parametrize("form", ["both", "after", "before", "in place"])
@pytest.mark.parametrize("rows,width,dtype", [
    (1000, 4096, torch.bfloat16), (1000, 4096, torch.float32), (500, 8192, torch.float32), (7400, 264, torch.float16),  # 304, 304, 152, 2432 CTAs
    (15000, 64, torch.bfloat16), (15000, 37, torch.float32),  # 1216 CTAs of four rows
    (1400, 2051, torch.bfloat16), (470, 8200, torch.float16), (470, 16384, torch.bfloat16), (470, 20001, torch.float32)])  # 456, 152, 152, 152
def test_norm_of_several_rows_a_cta(ctx, rows, width, dtype, form):
    """As many rows as three turns of every CTA take, all of them against 64 bits."""
    g = torch.Generator(device="cuda")
    g.manual_seed(rows + width)
    rn = lambda *s: torch.randn(s, device="cuda", generator=g)  # noqa: E731
    size = torch.exp(2 * rn(rows, 1))  # rows differ, so that a neighbour's sum shows
    x, res, gate = (rn(rows, width) * size).to(dtype), (rn(rows, width) * size.flip(0)).to(dtype), rn(rows, width).to(dtype)
    wa, wb = 0.3 * rn(width), 0.3 * rn(width)
    if form == "after":
        gate = rn(rows, 1).to(dtype)
    after, before = None if form == "before" else wa, None if form == "after" else wb
    residual = None if form == "before" else res
    want, t, off_out, off_t = test_norm.formula(x, after, gate, True, 0.3, residual, before, 1e-5, 1.0)
    x_in, r_in = x.clone(), res.clone()
    out, total = ctx.norm(x_in, before=before, after=after, gate=gate, gate_act="sigmoid", scale=0.3,
                          residual=None if residual is None else r_in, eps=1e-5, offset=1.0,
                          **(dict(out=x_in, total=r_in) if form == "in place" else {}))
    if total is not None:
        test_norm.check(total, t, off_t, dtype)
    if out is not None:
        test_norm.check(out, want, off_out, dtype)
    if form != "in place":
        assert torch.equal(x_in, x) and torch.equal(r_in, res)
    ctx.sync_status()


@pytest.mark.parametrize("act,rows,width", [("Q8_K", 1000, 4096), ("Q8_0", 500, 8192), ("Q8_1", 15000, 96), ("Q8_K", 15000, 256), ("Q8_K", 470, 16384)])
def test_packed_norm_of_several_rows_a_cta(ctx, act, rows, width):
    g = torch.Generator(device="cuda")
    g.manual_seed(width)
    x, res = torch.randn((2, rows, width), device="cuda", generator=g).unbind(0)
    w = torch.randn(width, device="cuda", generator=g)
    rows32, total = ctx.norm(x, before=w, after=True, residual=res)
    packed, same = ctx.norm(x, before=w, after=True, residual=res, act=act)
    assert torch.equal(packed, ctx.quantize_act(act, rows32)) and torch.equal(total, same)
    ctx.sync_status()
