"""The block-quantized key/value cache: what ggq_kv_store writes (quants and
scales equal to the quantizers' arithmetic, every byte at its documented place),
what ggq_kv_load reads back, and the refusals of both."""
import numpy as np
import pytest

torch = pytest.importorskip("torch")

import gguf_block_quant_ggq_gb300 as ggq  # noqa: E402

gpu = pytest.mark.gpu
DTYPES = {"float32": torch.float32, "float16": torch.float16, "bfloat16": torch.bfloat16}


@pytest.fixture(scope="module")
def ctx():
    assert torch.cuda.is_available(), "GPU tests need a CUDA device"
    from gguf_block_quant_ggq_gb300 import _build
    _build.build()
    c = ggq.Context(0)
    yield c
    c.close()


def blob_bytes(fmt, D):
    return (17 if fmt == "Q8_0" else 9) * D


def decode(pool, fmt, value, n_pages, H, page, D):
    """(quants as stored [slots][H][D], fp16 scales [slots][H][D/32]) of a pool, place by place."""
    b = pool.reshape(n_pages, H, page // 16, blob_bytes(fmt, D))
    q = np.zeros((n_pages, H, page // 16, 16, D), dtype=np.int32)
    for r in range(16):
        for d in range(D):
            o = r // 8
            if not value:
                lane, j, i = 4 * (r % 8) + d % 16 // 4, d // 16, d % 4
                f = o * (D // 16) + j if fmt == "Q8_0" else o * (D // 32) + d // 32
                nib = 2 * i if fmt == "Q8_0" else 4 * (i & 1) + 2 * (j & 1) + (i >> 1)
            else:
                n, t, e = d // 8, r % 8 // 2, r % 2
                lane = 4 * (d % 8) + t
                f = n if fmt == "Q8_0" else n // 2
                nib = 2 * (2 * o + e) if fmt == "Q8_0" else 4 * e + 2 * o + (n & 1)
            byte = b[..., ((f // 4) * 32 + lane) * 16 + (f % 4) * 4 + nib // 2]
            q[..., r, d] = byte if fmt == "Q8_0" else (byte >> (4 * (nib & 1))) & 15
    sc = np.ascontiguousarray(b[..., -D:]).view(np.float16).reshape(n_pages, H, page // 16, 16, D // 32)
    order = (0, 2, 3, 1, 4)
    return q.transpose(order).reshape(n_pages * page, H, D), sc.transpose(order).reshape(n_pages * page, H, D // 32)


def quantize(x, fmt):
    """(stored quants, fp16 scales) of fp32 rows [..., D] by the fp32 sequence of the quantizers."""
    b = x.astype(np.float32).reshape(*x.shape[:-1], -1, 32)
    with np.errstate(divide="ignore", invalid="ignore", over="ignore"):
        if fmt == "Q8_0":
            d = (np.abs(b).max(-1, keepdims=True) * (np.float32(1) / np.float32(127))).astype(np.float32)
            inv = np.where(d != 0, np.float32(1) / d, np.float32(0)).astype(np.float32)
            r = (b * inv).astype(np.float32)
            q = np.clip(np.sign(r) * np.floor(np.abs(r.astype(np.float64)) + 0.5), -127, 127) + 128
        else:
            at = np.abs(b).argmax(-1)[..., None]
            d = (np.take_along_axis(b, at, -1) / np.float32(-8)).astype(np.float32)
            inv = np.where(d != 0, np.float32(1) / d, np.float32(0)).astype(np.float32)
            r = ((b * inv).astype(np.float32) + np.float32(8.5)).astype(np.float32)
            q = np.clip(np.floor(r), 0, 15)
        return q.astype(np.int32).reshape(x.shape), d[..., 0].astype(np.float16)


def rows(n, H, D, dtype, seed, stride=0):
    """n rows of H heads; stride: they are part of wider rows."""
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    w = torch.randn((n, H * D + stride), device="cuda", generator=g)
    w *= torch.exp2(torch.randint(-3, 4, (n, H * D + stride), device="cuda", generator=g).float())
    return w.to(DTYPES[dtype])[:, stride:].unflatten(1, (H, D))


SLOTS = {
    "one": lambda page, n: [page + 3],
    "run": lambda page, n: list(range(5, 5 + 53)),                 # a prompt from an odd place: groups and both ragged ends
    "aligned": lambda page, n: list(range(16, 16 + 48)),
    "scattered": lambda page, n: [(i * 37 + 11) % n for i in range(21)],
    "skips": lambda page, n: [-1, 7, -5] + list(range(32, 48)) + [-1] + list(range(64, 80)),
    "starts": lambda page, n: [16, 32, 48, 64] + list(range(80, 95)) + [0],  # aligned slots without their group
    "down": lambda page, n: list(range(60, 20, -1)),
}


@gpu
@pytest.mark.parametrize("where", sorted(SLOTS))
@pytest.mark.parametrize("k_type,v_type,H,D,dtype", [
    ("Q8_0", "Q8_0", 3, 128, "float32"), ("Q4_0", "Q4_0", 2, 64, "float32"), ("Q8_0", "Q4_0", 1, 256, "bfloat16"),
    ("Q4_0", "Q8_0", 5, 64, "float16"), ("Q4_0", "Q4_0", 2, 128, "bfloat16"), ("Q8_0", "Q8_0", 2, 64, "float16"),
    ("Q4_0", "Q4_0", 1, 256, "float32"),
])
def test_store_writes_the_blocks_and_load_reads_them(ctx, k_type, v_type, H, D, dtype, where):
    page, n_pages = 48, 3
    n_slots = page * n_pages
    slots = SLOTS[where](page, n_slots)
    n = len(slots)
    k, v = rows(n, H, D, dtype, 1, 8), rows(n, H, D, dtype, 2, 4)
    cache = ctx.kv_cache(k_type, v_type, n_pages, page, H, D)
    cache.k.fill_(0xA5)
    cache.v.fill_(0x5A)
    dslots = torch.tensor(slots, dtype=torch.int64, device="cuda")
    ctx.kv_store(cache, k, v, dslots)
    got = ctx.kv_load(cache, dslots)
    got16 = ctx.kv_load(cache, dslots, dtype=torch.bfloat16)
    ctx.sync_status()
    for x, pool, fmt, value, back, back16 in ((k, cache.k, k_type, False, got[0], got16[0]),
                                              (v, cache.v, v_type, True, got[1], got16[1])):
        q, sc = decode(pool.cpu().numpy(), fmt, value, n_pages, H, page, D)
        fill = np.full(1, 0x5A if value else 0xA5, dtype=np.uint8)
        want_q, want_sc = quantize(x.float().cpu().numpy(), fmt)
        live = [i for i, s in enumerate(slots) if s >= 0]
        at = [slots[i] for i in live]
        assert np.array_equal(q[at], want_q[live])
        assert np.array_equal(sc[at].view(np.uint16), want_sc[live].view(np.uint16))
        rest = np.setdiff1d(np.arange(n_slots), at)  # no other token's bytes moved
        byte = int(fill[0])
        assert np.isin(q[rest], [byte] if fmt == "Q8_0" else [byte & 15, byte >> 4]).all()
        assert (sc[rest].view(np.uint16) == byte * 257).all()
        vals = np.zeros((n, H, D), dtype=np.float32)
        vals[live] = (want_q[live] - (128 if fmt == "Q8_0" else 8)).astype(np.float32) * np.repeat(
            want_sc[live].astype(np.float32), 32, axis=-1)
        assert np.array_equal(back.cpu().numpy(), vals)
        assert torch.equal(back16, torch.from_numpy(vals).cuda().to(torch.bfloat16))


@gpu
def test_special_values(ctx):
    """Zeros, ties of the largest magnitude, values below fp16's scales and NaN."""
    D = 64
    x = torch.zeros((4, 1, D), device="cuda")
    x[1, 0, 3], x[1, 0, 9] = -2.0, 2.0          # a tie: the first one sets Q4_0's scale
    x[1, 0, 32:] = 1e-9
    x[2, 0] = torch.linspace(-1, 1, D)
    x[3, 0, 5], x[3, 0, 40] = float("nan"), 3.0
    slots = torch.arange(4, device="cuda") * 5
    for fmt in ("Q8_0", "Q4_0"):
        cache = ctx.kv_cache(fmt, fmt, 2, 16, 1, D)
        ctx.kv_store(cache, x, x, slots)
        k, v = ctx.kv_load(cache, slots)
        ctx.sync_status()
        assert torch.equal(k, v)
        y = x.clone()
        y[3, 0, 5] = 0.0
        q, sc = quantize(y.cpu().numpy(), fmt)
        q[3, 0, 5] = 1 if fmt == "Q8_0" else 0  # a NaN counts as the smallest quant
        want = (q - (128 if fmt == "Q8_0" else 8)).astype(np.float32) * np.repeat(sc.astype(np.float32), 32, axis=-1)
        assert np.array_equal(k.cpu().numpy(), want)
        assert (k[0] == 0).all()
        if fmt == "Q4_0":
            assert k[1, 0, 3] == -2.0 and k[1, 0, 9] == 1.75


@gpu
def test_places_beyond_32_bits(ctx):
    H, D, page = 8, 256, 256
    n_pages = (1 << 32) // (H * (page // 16) * 17 * D) + 40  # the K pool passes 4 GiB
    cache = ctx.kv_cache("Q8_0", "Q4_0", n_pages, page, H, D)
    assert cache.k.numel() > 1 << 32
    n = 37
    k, v = rows(n, H, D, "float32", 3), rows(n, H, D, "float32", 4)
    slots = torch.arange(n_pages * page - n, n_pages * page, device="cuda")
    ctx.kv_store(cache, k, v, slots)
    a, b = ctx.kv_load(cache, slots)
    ctx.sync_status()
    for x, fmt, y in ((k, "Q8_0", a), (v, "Q4_0", b)):
        q, sc = quantize(x.cpu().numpy(), fmt)
        assert np.array_equal(y.cpu().numpy(), (q - (128 if fmt == "Q8_0" else 8)).astype(np.float32)
                              * np.repeat(sc.astype(np.float32), 32, axis=-1))


@gpu
def test_slots_outside_the_cache_are_reported(ctx):
    cache = ctx.kv_cache("Q8_0", "Q8_0", 2, 16, 1, 64)
    x = rows(2, 1, 64, "float32", 5)
    slots = torch.tensor([3, 32], device="cuda")
    ctx.kv_store(cache, x, x, slots)
    with pytest.raises(ggq.GGQError, match="outside the key/value cache"):
        ctx.sync_status()
    k, _ = ctx.kv_load(cache, slots)
    with pytest.raises(ggq.GGQError, match="outside the key/value cache"):
        ctx.sync_status()
    assert (k[1] == 0).all() and (k[0] != 0).any()
    ctx.sync_status()


@gpu
def test_empty_and_refused_calls(ctx):
    cache = ctx.kv_cache("Q8_0", "Q4_0", 2, 16, 2, 64)
    none = torch.empty((0, 2, 64), device="cuda")
    ctx.kv_store(cache, none, none, torch.empty(0, dtype=torch.int64, device="cuda"))
    x = rows(1, 2, 64, "float32", 6)
    s = torch.zeros(1, dtype=torch.int64, device="cuda")
    with pytest.raises(ValueError, match="agree"):
        ctx.kv_store(cache, x, x.half(), s)
    with pytest.raises(ValueError, match="agree"):
        ctx.kv_store(cache, x, x, torch.zeros(2, dtype=torch.int64, device="cuda"))
    with pytest.raises(ValueError, match="int64"):
        ctx.kv_store(cache, x, x, s.int())
    with pytest.raises(ValueError, match="float32"):
        ctx.kv_store(cache, x.double(), x.double(), s)
    with pytest.raises(ValueError, match="tensor"):
        ctx.kv_store(cache, x[:, :1], x[:, :1], s)
    with pytest.raises(ValueError, match="dense"):
        y = torch.zeros((1, 2, 128), device="cuda")[..., ::2]
        ctx.kv_store(cache, y, y, s)
    with pytest.raises(ggq.GGQError, match="multiples of 4"):
        y = torch.zeros(1 * 2 * 64 + 1, device="cuda")[1:].view(1, 2, 64)
        ctx.kv_store(cache, y, y, s)
    with pytest.raises(ggq.GGQError, match="multiples of 4"):
        y = torch.zeros((1, 2, 66), device="cuda")[..., :64]
        ctx.kv_store(cache, y, y, s)
    for bad in (("Q4_K", "Q8_0", 2, 16, 2, 64), ("Q8_0", "Q8_0", 2, 16, 2, 96), ("Q8_0", "Q8_0", 2, 24, 2, 64)):
        with pytest.raises(ValueError, match="not supported"):
            ctx.kv_cache(*bad)
    with pytest.raises(ValueError, match="pool"):
        ctx.kv_cache("Q8_0", "Q8_0", 2, 16, 2, 64, k=torch.zeros(5, dtype=torch.uint8, device="cuda"))


def test_page_bytes_and_support_query():
    from gguf_block_quant_ggq_gb300 import _build
    _build.build()
    lib = ggq.load()
    for D in (64, 128, 256):
        assert lib.ggq_kv_page_bytes(ggq.TYPE["Q8_0"], 3, D, 32) == 3 * 2 * 17 * D
        assert lib.ggq_kv_page_bytes(ggq.TYPE["Q4_0"], 3, D, 32) == 3 * 2 * 9 * D
    for bad in ((ggq.TYPE["Q4_K"], 3, 64, 32), (8, 0, 64, 32), (8, 3, 96, 32), (8, 3, 64, 40), (8, 3, 64, 0)):
        assert lib.ggq_kv_page_bytes(*bad) == 0
    for w in ggq.TYPE:
        for a in ggq.TYPE:
            assert ggq.supported(w, a, "kv_cache") == (w in ("Q8_0", "Q4_0") and a in ("Q8_0", "Q4_0"))
    assert lib.ggq_kv_store(None, None, 0, None, 0, 0, None, 0, 0, None, 0, None) == 1
    assert lib.ggq_kv_load(None, None, 0, None, 0, None, 0, 0, None, 0, 0, None) == 1
    assert lib.ggq_attention(None, None, None, None) == 1
    assert lib.ggq_reserve_attention(None, None) == 1
    assert lib.ggq_moe_route(None, None, 0, None, 0, 1, None, None, None) == 1
