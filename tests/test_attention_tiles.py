"""ggq_attention where its tile kernels serve the call (many rows of many kv heads at
once: their waves then cost less than the streaming kernel's items), and where one
row's keys are shared by many CTAs.

The reference and the tolerance are test_attention's, with one more term: fp16
outputs below 2^-14 are rounded to multiples of 2^-24, which is 2^-25 off at most
whatever their size."""
import math

import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

import gguf_block_quant_ggq_gb300 as ggq  # noqa: E402
from test_attention import DTYPES, ROUND, SPLIT, Case, ctx  # noqa: E402,F401

# 24 sequences of 0 to 400 tokens: prompts from nothing, chunks, single tokens, none
# new, rows before the first key, ends on and beside every tile's and blob's edge
LENS = [400, 1, 15, 16, 17, 0, 127, 128, 129, 255, 256, 257, 33, 300, 90, 64, 65, 399, 31, 140, 2, 63, 200, 130]
NEWS = [130, 1, 15, 16, 5, 2, 127, 128, 129, 100, 33, 1, 40, 130, 90, 0, 65, 7, 31, 100, 2, 63, 128, 130]
HEADS = [(32, 8, 64), (14, 2, 64), (32, 8, 128), (8, 8, 128), (14, 2, 128), (16, 8, 256)]


def check(c, out, scale=None, cap=0.0, window=0, slopes=None):
    G, scale = c.H // c.Hkv, c.D ** -0.5 if scale is None else scale
    least = 1e-30 + (2.0 ** -25 if c.dtype == "f16" else 0.0)
    r0 = k0 = 0
    for length, new in zip(c.lens, c.news):
        q, got = (x[r0:r0 + new].double().transpose(0, 1) for x in (c.q, out))  # [heads][rows][D]
        k, v = (x[k0:k0 + length].transpose(0, 1).repeat_interleave(G, 0) for x in (c.k, c.v))
        pos = torch.arange(length - new, length, device="cuda")[:, None]
        key = torch.arange(length, device="cuda")[None]
        seen = (key <= pos) & (key > pos - window if window else True)
        x, size = scale * q @ k.transpose(1, 2), abs(scale) * q.abs() @ k.abs().transpose(1, 2)
        if cap > 0:
            x = cap * torch.tanh(x / cap)
        if slopes is not None:
            far = slopes.double()[:, None, None] * (key - pos)
            x, size = x + far, size + far.abs()
        p = torch.softmax(x.masked_fill(~seen, -math.inf), -1).nan_to_num(0.0)  # no key: 0
        S = (size * (p > 1e-9)).amax(-1, keepdim=True) if length else torch.zeros((c.H, new, 1), device="cuda")
        want, A = p @ v, p @ v.abs()
        bound = SPLIT[c.dtype] * (8 + 2 * S) * A + ROUND[c.dtype] * want.abs() + least
        err = (got - want).abs()
        assert torch.isfinite(got).all()
        assert (err <= bound).all(), f"{length} tokens: worst {float((err / bound).max()):.3g} of the bound"
        assert (got[:, ~seen.any(1)] == 0).all()
        r0 += new
        k0 += length


@pytest.mark.parametrize("k_type,v_type", [("Q8_0", "Q8_0"), ("Q4_0", "Q4_0"), ("Q8_0", "Q4_0"), ("Q4_0", "Q8_0")])
@pytest.mark.parametrize("dtype", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("H,Hkv,D", HEADS)
def test_many_rows(ctx, H, Hkv, D, dtype, k_type, v_type):  # noqa: F811
    c = Case(ctx, LENS, NEWS, H, Hkv, D, k_type, v_type, dtype, 16 if D == 64 else 48, seed=H + D)
    out = c.call()
    ctx.sync_status()
    check(c, out)


@pytest.mark.parametrize("opts", [dict(window=1), dict(window=50), dict(cap=5.0), dict(slopes=True), dict(scale=-0.3),
                                  dict(scale=0.0), dict(window=64, cap=30.0, slopes=True, scale=0.2)])
@pytest.mark.parametrize("dtype,D", [("f32", 64), ("f32", 128), ("f32", 256), ("bf16", 64), ("f16", 128), ("bf16", 256)])
def test_masks_caps_and_biases_of_many_rows(ctx, dtype, D, opts):  # noqa: F811
    c = Case(ctx, LENS, NEWS, 16, 8, D, "Q8_0", "Q4_0", dtype, 32, seed=D)
    opts = dict(opts)
    if opts.get("slopes"):
        opts["slopes"] = torch.exp2(-1.0 - torch.arange(16, device="cuda") / 2)
    out = c.call(**opts)
    ctx.sync_status()
    check(c, out, **opts)


@pytest.mark.parametrize("dtype,D", [("f32", 64), ("f32", 128), ("f32", 256), ("bf16", 128)])
def test_peaked_scores_of_many_rows(ctx, dtype, D):  # noqa: F811
    c = Case(ctx, LENS, NEWS, 32, 8, D, dtype=dtype, seed=3, q_mul=30.0)
    out = c.call()
    ctx.sync_status()
    check(c, out)


@pytest.mark.parametrize("what,bits", [("k", 0x7E00), ("v", 0x7E00), ("v", 0x7C00), ("v", 0xFC00)])
@pytest.mark.parametrize("dtype", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("window", [0, 40])
def test_bad_scales_reach_only_rows_that_see_them(ctx, D, dtype, window, what, bits):  # noqa: F811
    """One scale that is NaN or infinite in the middle of each sequence, for few rows and for many.

    Rows whose mask leaves the token out keep their results bit by bit.  Of those that see
    it, a NaN key makes the whole row NaN, a value's scale the outputs of its 32 channels
    (infinity times a quant of 0, or a probability of 0, is NaN)."""
    few = [min(x, 3) for x in NEWS]
    for news in (NEWS, few):
        c = Case(ctx, LENS, news, 16, 8, D, dtype=dtype, seed=11)
        clean = c.call(window=window)
        pool = (c.cache.k if what == "k" else c.cache.v).view(torch.uint8).view(-1, 17 * D)  # blobs of 16 tokens
        at, k0 = [], 0
        for length in LENS:
            at.append(length // 2)
            if length:
                slot = int(c.slots[k0 + length // 2])
                for head in range(8):  # pages hold 16 tokens here: one blob a head
                    scales = pool[slot // 16 * 8 + head, 16 * D:].view(torch.int16).view(16, D // 32)
                    scales[slot % 16, 1] = bits - (1 << 16 if bits >= 1 << 15 else 0)
            k0 += length
        out = c.call(window=window)
        ctx.sync_status()
        r0 = 0
        for length, new, bad in zip(LENS, news, at):
            pos = torch.arange(length - new, length, device="cuda")
            sees = (pos >= bad) & (length > 0)
            if window:
                sees &= pos - window < bad
            got, want = out[r0:r0 + new], clean[r0:r0 + new]
            assert torch.equal(got[~sees], want[~sees])
            spoilt = got[sees] if what == "k" else got[sees][..., 32:64]
            assert not torch.isfinite(spoilt.float()).any()
            if what == "v":
                assert torch.equal(got[sees][..., :32], want[sees][..., :32])
            r0 += new


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("H,Hkv,D,lens,news", [
    (1, 1, 64, [60001], [1]), (8, 1, 128, [40000, 7], [1, 1]), (4, 1, 256, [30011], [3]), (16, 1, 64, [3, 33333, 0], [3, 2, 0]),
])
def test_one_item_over_many_ctas(ctx, H, Hkv, D, lens, news, dtype):  # noqa: F811
    """Pieces of an item that fill the GPU are joined in two levels, the same way each time."""
    c = Case(ctx, lens, news, H, Hkv, D, dtype=dtype, page=256, seed=D)
    out = c.call()
    ctx.sync_status()
    check(c, out)
    for _ in range(3):
        assert torch.equal(out, c.call())


@pytest.mark.parametrize("dtype,D", [("f32", 64), ("f32", 128), ("f32", 256), ("f16", 64), ("bf16", 128)])
def test_strided_rows_of_many_tokens(ctx, dtype, D):  # noqa: F811
    c = Case(ctx, LENS, NEWS, 16, 8, D, dtype=dtype, seed=5)
    n = sum(NEWS)
    wide = torch.zeros((n, 3, 16, D + 32), dtype=DTYPES[dtype], device="cuda")
    wide[:, 1, :, 32:] = c.q
    out = torch.full((16, n + 1, D), 9.0, dtype=DTYPES[dtype], device="cuda")
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    with torch.cuda.stream(s):
        c.call(q=wide[:, 1, :, 32:], out=out[:, :n].transpose(0, 1))
    s.synchronize()
    ctx.sync_status()
    check(c, out[:, :n].transpose(0, 1))
    assert (out[:, n] == 9.0).all()


@pytest.mark.parametrize("dtype,D", [("f32", 64), ("f32", 256), ("bf16", 128)])
def test_bad_pages_of_many_rows_are_reported(ctx, dtype, D):  # noqa: F811
    c = Case(ctx, LENS, NEWS, 16, 8, D, dtype=dtype, seed=6)
    c.table[0, 2] = 10 ** 6
    c.call()
    with pytest.raises(ggq.GGQError, match="outside the key/value cache"):
        ctx.sync_status()
    c.table[0, 2] = 0
    c.call(max_len=399)
    with pytest.raises(ggq.GGQError, match="outside the key/value cache"):
        ctx.sync_status()
    c.call()
    ctx.sync_status()
