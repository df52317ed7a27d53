"""The rotary table against 60-digit arithmetic, the rotation against the same products in torch (bit for bit) and
in 64 bits, and the rotated write into the cache against ggq_rotate followed by ggq_kv_store."""
import ctypes
import math
from decimal import Decimal, getcontext

import pytest

torch = pytest.importorskip("torch")

import gguf_block_quant_ggq_gb300 as ggq  # noqa: E402

gpu = pytest.mark.gpu
DTYPES = [torch.float32, torch.float16, torch.bfloat16]
LAYOUTS = ["half", "pairs"]


@pytest.fixture(scope="module")
def ctx():
    assert torch.cuda.is_available(), "GPU tests need a CUDA device"
    from gguf_block_quant_ggq_gb300 import _build
    _build.build()
    c = ggq.Context(0)
    yield c
    c.close()


def turned(x, table, positions, layout, first):
    """fp32 rows turned with every product and sum rounded by itself; positions outside the table turn nothing."""
    x = x.float()
    half = table.shape[1]
    ok = (positions >= 0) & (positions < table.shape[0])
    cs = table[torch.where(ok, positions, 0).long()]
    cs = torch.where(ok[:, None, None], cs, torch.tensor([1.0, 0.0], device=x.device))[:, None]
    c, s = cs[..., 0], cs[..., 1]
    i = torch.arange(half, device=x.device)
    a = first + (2 * i if layout == "pairs" else i)
    b = a + (1 if layout == "pairs" else half)
    out = x.clone()
    out[..., a] = x[..., a] * c - x[..., b] * s
    out[..., b] = x[..., a] * s + x[..., b] * c
    return out


PI2 = 2 * Decimal("3.14159265358979323846264338327950288419716939937510582097494459")


def exact_angles(n, turn, base, divide):
    """Angles of positions n as fractions of a turn, from 60 digits; divide(j): what frequency j is divided by."""
    getcontext().prec = 60
    ln = Decimal(base).ln()
    f = [(-ln * 2 * j / turn).exp() / Decimal(divide(j)) / PI2 for j in range(turn // 2)]
    return [[float(p * x % 1) for x in f] for p in n]


@gpu
@pytest.mark.parametrize("turn,base", [(2, 10000.0), (64, 10000.0), (128, 500000.0), (130, 1e6), (1024, 10000.0)])
def test_table_at_all_distances(ctx, turn, base):
    """Off by the product's 2^-27 of a turn (times 2 pi), sincospif's last two bits and the rounding: below 2.5e-7 up to
    position 2^26; beyond it the frequency's rounding to 64 bits counts, 2^-53 of the angle."""
    for first in (0, 1000, 131071, 1 << 22, (1 << 26) - 5, (1 << 31) - 4):
        n = 4
        got = ctx.rotary_table(n, turn, base=base, first=first).double().cpu()
        t = torch.tensor(exact_angles(range(first, first + n), turn, base, lambda j: 1)).double() * (2 * math.pi)
        room = 2.5e-7 + 2.0 ** -51 * first
        assert float((got[..., 0] - t.cos()).abs().max()) <= room
        assert float((got[..., 1] - t.sin()).abs().max()) <= room


@gpu
def test_table_scaled(ctx):
    n, turn, base = 300, 128, 10000.0
    two = ctx.rotary_table(2 * n, turn)
    assert float((ctx.rotary_table(n, turn, factor=2.0)[::2] - two[:n][:n // 2]).abs().max()) <= 5e-7  # every position half as far
    factors = [1.0 + 0.1 * j for j in range(turn // 2)]
    t = torch.tensor(exact_angles(range(7), turn, base, lambda j: 1.0 + 0.1 * j)).double() * (2 * math.pi)
    for f in (factors, torch.tensor(factors)):
        got = ctx.rotary_table(7, turn, factors=f, magnitude=1.25).double().cpu()
        # the factors are fp32: a relative 2^-24 of angles up to 6
        assert float((got - 1.25 * torch.stack([t.cos(), t.sin()], -1)).abs().max()) <= 1.25 * (2.5e-7 + 6 * 2.0 ** -24)
    # by channel: the fast ones as they are, the slow ones divided, a ramp between
    L, factor = 4096, 8.0
    place = lambda turns: turn * math.log(L / (turns * 2 * math.pi)) / (2 * math.log(base))  # noqa: E731
    low, high = max(math.floor(place(32.0)), 0), min(math.ceil(place(1.0)), turn - 1)
    mix = [min(max((j - low) / (high - low), 0.0), 1.0) for j in range(turn // 2)]
    assert mix[0] == 0.0 and mix[-1] == 1.0 and 0 < mix[(low + high) // 2] < 1
    f = torch.tensor([base ** (-2.0 * j / turn) * (1 - m + m / factor) for j, m in enumerate(mix)], dtype=torch.float64)
    got = ctx.rotary_table(n, turn, factor=factor, original_len=L).double().cpu()
    a = torch.arange(n, dtype=torch.float64)[:, None] * f
    assert float((got - torch.stack([a.cos(), a.sin()], -1)).abs().max()) <= 3e-7


@gpu
@pytest.mark.parametrize("layout", LAYOUTS)
@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("heads,D,turn,first", [(1, 64, 64, 0), (8, 128, 128, 0), (5, 128, 64, 64), (3, 128, 64, 16), (3, 80, 80, 0),
                                                (2, 96, 40, 8), (7, 192, 64, 128), (4, 256, 256, 0), (2, 30, 10, 3), (1, 2, 2, 0),
                                                (6, 1024, 1024, 0), (3, 13, 6, 4)])
def test_rotate_bit_for_bit(ctx, dtype, layout, heads, D, turn, first):
    g = torch.Generator(device="cuda")
    g.manual_seed(D * 7 + turn)
    table = ctx.rotary_table(500, turn)
    for n in (1, 3, 70):
        pos = torch.randint(0, 500, (n,), device="cuda", generator=g, dtype=torch.int32)
        wide = torch.randn((n, heads + 2, D + 8), device="cuda", generator=g).to(dtype)
        views = [lambda w: w[:, :heads, :D].contiguous(), lambda w: w[:, 1:heads + 1, :D], lambda w: w[:, 1:heads + 1, 5:D + 5]]
        for view in views:
            x = view(wide)
            want = turned(x, table, pos, layout, first).to(dtype)
            assert torch.equal(ctx.rotate(x, table, pos, layout=layout, first=first), want)
            buf = wide.clone()
            y = view(buf)
            assert ctx.rotate(y, table, pos, layout=layout, first=first, out=y) is y  # in place
            assert torch.equal(y, want)
            view(buf).copy_(x)
            y.copy_(x)
            assert torch.equal(buf, wide)  # nothing beside the heads
    ctx.sync_status()


@gpu
def test_rotation_keeps_dot_products_by_distance(ctx):
    """q . k after the rotation is a function of the distance of their positions (64-bit check of the whole)."""
    table = ctx.rotary_table(4000, 64)
    q, k = torch.randn((2, 1, 64), device="cuda").unbind(0)
    x = torch.stack([q, k], 1).expand(3, 2, 64).contiguous()
    pos = lambda a: torch.tensor(a, dtype=torch.int32, device="cuda")  # noqa: E731
    a, b = ctx.rotate(x, table, pos([5, 1005, 3990])), ctx.rotate(x, table, pos([2, 1002, 3987]))
    dots = (a[:, 0].double() * b[:, 1].double()).sum(1)
    assert float((dots - dots[0]).abs().max()) <= 64 * float(q.norm() * k.norm()) * 2.0 ** -22


@gpu
def test_positions_outside_the_table(ctx):
    table = ctx.rotary_table(10, 64)
    x = torch.randn((4, 2, 64), device="cuda")
    pos = torch.tensor([3, 10, -1, 9], dtype=torch.int32, device="cuda")
    got = ctx.rotate(x, table, pos)
    with pytest.raises(ggq.GGQError, match="position"):
        ctx.sync_status()
    ctx.sync_status()  # reported once
    assert torch.equal(got, turned(x, table, pos, "half", 0))
    assert torch.equal(got[1:3], x[1:3])


CACHES = [("Q8_0", "Q8_0", 3, 128, torch.float32), ("Q4_0", "Q4_0", 2, 64, torch.bfloat16), ("Q8_0", "Q4_0", 1, 256, torch.float16),
          ("Q4_0", "Q8_0", 5, 64, torch.float32), ("Q8_0", "Q8_0", 8, 128, torch.bfloat16)]
SLOTS = {"one": [51], "run": list(range(5, 58)), "scattered": [(i * 37 + 11) % 144 for i in range(21)],
         "padded": [-1, 7] + list(range(32, 48)) + [-5] + list(range(64, 81))}


@gpu
@pytest.mark.parametrize("where", sorted(SLOTS))
@pytest.mark.parametrize("layout", LAYOUTS)
@pytest.mark.parametrize("k_type,v_type,H,D,dtype", CACHES)
def test_append_is_rotate_then_store(ctx, k_type, v_type, H, D, dtype, layout, where):
    g = torch.Generator(device="cuda")
    g.manual_seed(D + H)
    slots = torch.tensor(SLOTS[where], device="cuda")
    n, heads = len(slots), 2 * H
    for turn, first in ((D, 0), (D // 2, D // 2), (12, 20), (16, 8)):
        table = ctx.rotary_table(3000, turn)
        pos = torch.randint(0, 3000, (n,), device="cuda", generator=g, dtype=torch.int32)
        row = torch.randn((n, heads + 2 * H, D), device="cuda", generator=g).to(dtype)
        q, k, v = row.split([heads, H, H], 1)
        got, want = (ctx.kv_cache(k_type, v_type, 3, 48, H, D) for _ in range(2))
        for c in (got, want):
            c.k.fill_(0xA5)
            c.v.fill_(0x5A)
        q_out = ctx.kv_append(got, k, v, slots, table, pos, layout=layout, first=first, q=q)
        assert ctx.kv_append(got, k, v, slots, table, pos, layout=layout, first=first) is None  # without queries
        ctx.kv_store(want, turned(k, table, pos, layout, first), v.float(), slots)
        assert torch.equal(got.k, want.k) and torch.equal(got.v, want.v)
        assert torch.equal(q_out, turned(q, table, pos, layout, first).to(dtype))
        keep = row.clone()
        ctx.kv_append(got, k, v, slots, table, pos, layout=layout, first=first, q=q, q_out=q)  # in place, inside the fused row
        assert torch.equal(q, q_out) and torch.equal(row[:, heads:], keep[:, heads:]) and torch.equal(got.k, want.k)
    ctx.sync_status()


@gpu
def test_append_of_many_heads_and_a_long_prompt(ctx):
    """Several heads a CTA (many windows), and query heads of a number that no part divides."""
    g = torch.Generator(device="cuda")
    g.manual_seed(9)
    n, H, heads, D, page = 8200, 8, 24, 64, 64
    table = ctx.rotary_table(9000, D)
    pos = torch.arange(n, device="cuda", dtype=torch.int32) + 77
    q, k, v = torch.randn((n, heads + 2 * H, D), device="cuda", generator=g).bfloat16().split([heads, H, H], 1)
    slots = torch.arange(n, device="cuda") + 21
    got, want = (ctx.kv_cache("Q8_0", "Q4_0", 130, page, H, D) for _ in range(2))
    out = ctx.kv_append(got, k, v, slots, table, pos, q=q)
    ctx.kv_store(want, turned(k, table, pos, "half", 0), v.float(), slots)
    assert torch.equal(got.k, want.k) and torch.equal(got.v, want.v)
    assert torch.equal(out, turned(q, table, pos, "half", 0).bfloat16())


@gpu
def test_append_reports_and_pads(ctx):
    table = ctx.rotary_table(16, 64)
    cache, want = (ctx.kv_cache("Q8_0", "Q8_0", 2, 16, 1, 64) for _ in range(2))
    x = torch.randn((3, 1, 64), device="cuda")
    tensor = lambda a, t: torch.tensor(a, dtype=t, device="cuda")  # noqa: E731
    # a padded row's position is not looked at
    q = ctx.kv_append(cache, x, x, tensor([3, -1, 20], torch.int64), table, tensor([1, 99, 2], torch.int32), q=x)
    ctx.sync_status()
    assert torch.equal(q[1], x[1])
    # a position outside the table: stored unturned, and reported
    ctx.kv_append(cache, x[:1], x[:1], tensor([3], torch.int64), table, tensor([16], torch.int32))
    with pytest.raises(ggq.GGQError, match="position"):
        ctx.sync_status()
    ctx.kv_store(want, x[:1], x[:1], tensor([3], torch.int64))
    assert torch.equal(ctx.kv_load(cache, tensor([3], torch.int64))[0], ctx.kv_load(want, tensor([3], torch.int64))[0])
    # a slot outside the cache: not stored, and reported
    keep = cache.k.clone()
    ctx.kv_append(cache, x[:1], x[:1], tensor([32], torch.int64), table, tensor([1], torch.int32))
    with pytest.raises(ggq.GGQError, match="slot"):
        ctx.sync_status()
    assert torch.equal(cache.k, keep)


@gpu
def test_refusals(ctx):
    table = ctx.rotary_table(16, 64)
    x = torch.zeros((2, 3, 64), device="cuda")
    pos = torch.zeros(2, dtype=torch.int32, device="cuda")
    slots = torch.zeros(2, dtype=torch.int64, device="cuda")
    cache = ctx.kv_cache("Q8_0", "Q8_0", 1, 16, 3, 64)
    for bad in (dict(table=table[0]), dict(table=table.double()), dict(positions=pos[:1]), dict(positions=pos.long()),
                dict(out=x.half()), dict(out=x[:1]), dict(x=x.double()), dict(x=x[0]), dict(x=x.transpose(1, 2))):
        with pytest.raises(ValueError):
            ctx.rotate(**{**dict(x=x, table=table, positions=pos), **bad})
    with pytest.raises(KeyError):
        ctx.rotate(x, table, pos, layout="thirds")
    for bad, match in ((dict(first=2), "turned"), (dict(first=-1), "turned"), (dict(x=x[:, :, :32].contiguous()), "turned")):
        with pytest.raises(ggq.GGQError, match=match):
            ctx.rotate(**{**dict(x=x, table=table, positions=pos), **bad})
    wide = torch.zeros((2, 6, 64), device="cuda")
    with pytest.raises(ggq.GGQError, match="one stride"):
        ctx.rotate(wide[:, :3], table, pos, out=wide[:, ::2])
    for bad in (dict(k=x.half()), dict(slots=slots[:1]), dict(q=x[:1]), dict(q_out=x), dict(q=x, q_out=x.half())):
        with pytest.raises(ValueError):
            ctx.kv_append(**{**dict(cache=cache, k=x, v=x, slots=slots, table=table, positions=pos), **bad})
    for bad in (dict(turn=0), dict(turn=7), dict(turn=1026), dict(n=-1), dict(first=-1), dict(first=1 << 31), dict(base=1.0),
                dict(factor=0.5), dict(factors=[0.0] * 4), dict(factor=2.0, original_len=4, beta_fast=1.0, beta_slow=2.0),
                dict(magnitude=float("inf")), dict(original_len=-1), dict(table=0)):
        assert table_status(ctx, **bad) in (1, 2), bad
    with pytest.raises(ValueError):
        ctx.rotary_table(4, 8, factors=[1.0] * 3)
    assert ctx.rotate(x[:0], table, pos[:0]).shape == (0, 3, 64)
    assert ctx.rotary_table(0, 8).shape == (0, 4, 2)
    ctx.sync_status()


def table_status(ctx, turn=8, n=4, first=0, base=10000.0, factor=1.0, factors=None, original_len=0, beta_fast=32.0, beta_slow=1.0,
                 magnitude=1.0, table=None):
    """The C call's status (refusals come before any launch)."""
    host = (ctypes.c_float * len(factors))(*factors) if factors else None
    spec = ggq.ggq_rotary_spec(turn, base, ctypes.cast(host, ctypes.c_void_p) if host else None, factor, original_len, beta_fast,
                               beta_slow, magnitude)
    room = torch.zeros(64, device="cuda")
    return ggq.load().ggq_rotary_table(ctx.handle, ctypes.byref(spec), first, n, room.data_ptr() if table is None else None, None)


def test_null_context():
    L = ggq.load()
    assert L.ggq_rotary_table(None, None, 0, 0, None, None) == 1
    assert L.ggq_rotate(None, None, ctypes.byref(ggq.ggq_rotate_args()), None) == 1
    assert L.ggq_kv_append(None, None, None, ctypes.byref(ggq.ggq_append_args()), None) == 1
