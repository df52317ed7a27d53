"""ggq_attention at the edges of its plan, its masks and its ranges: batches whose items meet in one CTA's
counters, and the rows that must not notice what they do not see.

The reference and the tolerance are those of test_attention_tiles."""
import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

import gguf_block_quant_ggq_gb300 as ggq  # noqa: E402
from test_attention import Case, ctx  # noqa: E402,F401
from test_attention_tiles import check  # noqa: E402


@pytest.mark.parametrize("dtype,news", [("f32", 1), ("bf16", 1), ("bf16", 2), ("f32", 3)])
@pytest.mark.parametrize("lens", [[38421, 6670], [96394, 1557, 13709], [1094, 5198, 50458, 1056]])
def test_long_sequences_beside_short_ones(ctx, lens, dtype, news):  # noqa: F811
    """The last group of one item's pieces begins with the CTA that begins the next item: every
    row is written, the same way in every call on the context."""
    c = Case(ctx, lens, [news] * len(lens), 32, 8, 128, dtype=dtype, page=64, seed=len(lens))
    out = torch.full_like(c.q, 7.0)
    c.call(out=out)
    ctx.sync_status()
    check(c, out)
    for _ in range(3):
        again = torch.full_like(c.q, 9.0)
        c.call(out=again)
        assert torch.equal(out, again)
    ctx.sync_status()


# prompts from nothing, so that rows lie before, at, between and behind two places of a sequence
PROMPTS = [300, 400, 257, 129, 90, 350, 200, 310, 33, 16, 399, 17] * 2


def set_scale(c, pool, type_, page, place, block, bits):
    """Writes `bits` as the scale of one block of 32 channels of the cache's slot `place`, of every kv head."""
    per = (17 if type_ == "Q8_0" else 9) * c.D
    blobs = pool.view(-1, per)
    first = (place // page * c.Hkv + torch.arange(c.Hkv, device="cuda")) * (page // 16) + place % page // 16
    at = per - c.D + 2 * (place % 16 * (c.D // 32) + block)
    blobs[first, at] = bits & 0xFF
    blobs[first, at + 1] = bits >> 8


@pytest.mark.parametrize("bits", [0x7E00, 0x7C00, 0xFC00])
@pytest.mark.parametrize("dtype", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("D,v_type,page", [(64, "Q8_0", 16), (128, "Q4_0", 48), (128, "Q8_0", 64), (256, "Q8_0", 16)])
@pytest.mark.parametrize("window", [0, 1, 40])
def test_rows_between_two_bad_values(ctx, D, v_type, page, dtype, window, bits):  # noqa: F811
    """Two value scales of a sequence that are not finite: rows that see neither keep their results bit by
    bit, those that see one have its 32 channels spoilt."""
    for news in (PROMPTS, [min(3, x) for x in PROMPTS]):
        c = Case(ctx, PROMPTS, news, 16, 8, D, v_type=v_type, dtype=dtype, page=page, seed=11)
        clean = c.call(window=window)
        k0, bad = 0, []
        for length in PROMPTS:
            bad.append([length // 4, length - 2 - length // 4])
            for at in bad[-1]:
                set_scale(c, c.cache.v, v_type, page, int(c.slots[k0 + at]), 1, bits)
            k0 += length
        out = c.call(window=window)
        ctx.sync_status()
        r0 = between = 0
        for length, new, two in zip(PROMPTS, news, bad):
            pos = torch.arange(length - new, length, device="cuda")
            sees = torch.zeros(new, dtype=torch.bool, device="cuda")
            for at in two:
                sees |= (pos >= at) & (pos < at + window if window else True)
            between += int((~sees & (pos > two[0]) & (pos < two[1])).sum())
            got, want = out[r0:r0 + new], clean[r0:r0 + new]
            assert torch.equal(got[~sees], want[~sees])
            assert not torch.isfinite(got[sees][..., 32:64].float()).any()
            assert torch.equal(got[sees][..., :32], want[sees][..., :32])
            r0 += new
        assert between > 0 or window == 0 or news is not PROMPTS


WIDE = [("k", "Q8_0", 512.0), ("k", "Q8_0", 516.0), ("k", "Q8_0", 60000.0), ("k", "Q4_0", 8192.0), ("k", "Q4_0", 60000.0),
        ("v", "Q8_0", 511.5), ("v", "Q8_0", 512.0), ("v", "Q8_0", 600.0), ("v", "Q4_0", 8192.0)]


@pytest.mark.parametrize("dtype,what,type_,scale", [(d, *w) for d in ("f32", "f16", "bf16") for w in WIDE if (d, w[0]) != ("bf16", "v")])
@pytest.mark.parametrize("D,page", [(64, 16), (128, 48), (256, 16)])
@pytest.mark.parametrize("window", [0, 40])
def test_keys_and_values_beyond_fp16(ctx, dtype, what, type_, scale, D, page, window):  # noqa: F811
    """One block of each sequence with a large finite scale, whose products leave fp16's range (an fp16 value
    of 65504 is stored with the scale 516): rows of prompts that do not see it keep their results bit by bit,
    those that see it, and single rows, are as close to 64 bits as any.

    Values of bf16 rows are not among the cases: prompts keep them and their probabilities in bf16, which
    holds every product but rounds each by up to 2^-8, more than the tolerance grants where one key is all."""
    types = {"k": dict(k_type=type_), "v": dict(v_type=type_)}[what]
    # scores of a few units beside a key of that size, nearly equal weights beside such a value
    q_mul = 0.08 / scale * (1.0 if type_ == "Q8_0" else 16.0) if what == "k" else 0.3
    for news in (PROMPTS, [min(3, x) for x in PROMPTS]):
        c = Case(ctx, PROMPTS, news, 16, 8, D, dtype=dtype, page=page, seed=13, q_mul=q_mul, **types)
        clean = c.call(window=window)
        bits = int(torch.tensor(scale, dtype=torch.float16).view(torch.int16))
        k0 = 0
        for length in PROMPTS:
            set_scale(c, c.cache.k if what == "k" else c.cache.v, type_, page, int(c.slots[k0 + length // 3]), 1, bits)
            k0 += length
        c.k, c.v = (x.double() for x in ctx.kv_load(c.cache, c.slots))
        out = c.call(window=window)
        ctx.sync_status()
        check(c, out, window=window)
        if news is PROMPTS:
            r0 = 0
            for length, new in zip(PROMPTS, news):
                pos = torch.arange(new, device="cuda")
                sees = (pos >= length // 3) & (pos < length // 3 + window if window else True)
                assert torch.equal(out[r0:r0 + new][~sees], clean[r0:r0 + new][~sees])
                r0 += new


def test_fp16_rows_at_the_end_of_their_range(ctx):  # noqa: F811
    """A value of 65504, stored by kv_store, behind every row of a prompt but the last."""
    c = Case(ctx, PROMPTS, PROMPTS, 16, 8, 128, dtype="f16", page=16, seed=2)
    clean = c.call()
    last = torch.tensor([sum(PROMPTS[:i + 1]) - 1 for i in range(len(PROMPTS))], device="cuda")
    k, v = (x[last].half() for x in (c.k, c.v))
    v[:, :, 5] = 65504.0
    ctx.kv_store(c.cache, k, v, c.slots[last])
    out = c.call()
    ctx.sync_status()
    before = torch.ones(sum(PROMPTS), dtype=torch.bool, device="cuda")
    before[last] = False
    assert torch.equal(out[before], clean[before])
    assert torch.isfinite(out).all()


def test_status_is_read_and_cleared_in_the_streams_order(ctx):  # noqa: F811
    """sync_status of a side stream neither waits for another stream's work nor leaves the clearing of the
    error word to it: calls that follow on the side stream are whole."""
    c = Case(ctx, [30000, 7, 900], [1, 1, 1], 8, 1, 128, page=64, seed=4)
    want = c.call()
    s, busy = torch.cuda.Stream(), torch.cuda.Event()
    outside = torch.full_like(c.slots[:1], c.cache.n_pages * c.cache.page_size)
    k, v = c.k[:1].float(), c.v[:1].float()
    outs = torch.zeros((20, *want.shape), device="cuda")
    torch.cuda.synchronize()
    for busily in (False, True):  # first a round in which nothing else runs: kernels are loaded
        outs.zero_()
        torch.cuda.synchronize()
        if busily:
            torch.cuda._sleep(2 * 10 ** 9)  # about a second of the default stream's time
            busy.record()
        with torch.cuda.stream(s):
            ctx.kv_store(c.cache, k, v, outside)
            with pytest.raises(ggq.GGQError, match="outside the key/value cache"):
                ctx.sync_status()
            for out in outs:
                c.call(out=out)
            ctx.sync_status()
            assert not busily or not busy.query()
        torch.cuda.synchronize()
        assert all(torch.equal(out, want) for out in outs)


@pytest.mark.parametrize("window", [2 ** 31 - 3, 2 ** 31 - 1, 2 ** 31, 2 ** 40])
@pytest.mark.parametrize("dtype,D", [("f32", 64), ("f32", 256), ("bf16", 128), ("f16", 256)])
def test_windows_of_any_size(ctx, dtype, D, window):  # noqa: F811
    """More new rows than cached tokens, and a window that stands for none: rows before the first key are zeros,
    the others see what they see without a window."""
    for lens, news in (([3, 17, 1], [6, 17, 5]), ([3, 17, 300, 5] * 6, [90, 170, 300, 6] * 6)):
        c = Case(ctx, lens, news, 16, 8, D, dtype=dtype, seed=D)
        out = c.call(window=window)
        ctx.sync_status()
        assert torch.equal(out, c.call())
        check(c, out)


@pytest.mark.parametrize("rows", [1, 300])
@pytest.mark.parametrize("dtype,D", [("f32", 64), ("f32", 256), ("bf16", 128)])
def test_lengths_up_to_the_bound(ctx, dtype, D, rows):  # noqa: F811
    """The longest sequence there is, on one page that its table names again and again, behind a window: the rows
    see what those of a short sequence see whose last tokens stand in the same places.  A longer one is cut to
    it and reported."""
    page, longest = 4096, 2 ** 31 - 2 ** 25
    c = Case(ctx, [page], [rows], 32, 8, D, dtype=dtype, page=page, seed=rows, spare_pages=0)
    start = torch.tensor([0, rows], dtype=torch.int32, device="cuda")

    def call(length, **kw):
        table = torch.zeros((1, (length + page - 1) // page), dtype=torch.int32, device="cuda")
        lens = torch.tensor([length], dtype=torch.int32, device="cuda")
        return ctx.attention(c.cache, c.q, lens, table, q_start=start, window=100, **kw)

    want = call(page)
    out = call(longest)
    ctx.sync_status()
    check(c, want, window=100)
    check(c, out, window=100)
    cut = call(2 ** 31 - 1)
    with pytest.raises(ggq.GGQError, match="outside the key/value cache"):
        ctx.sync_status()
    assert torch.equal(cut, out)


@pytest.mark.parametrize("cap", [1e-40, 1e-3, 1000.0, 3000.0, 1e5, 1e9, 1e30, 3e38])
@pytest.mark.parametrize("dtype,D,slopes", [("f32", 64, False), ("f32", 256, False), ("f16", 64, True), ("bf16", 128, False),
                                            ("f16", 256, False)])
def test_caps_of_any_size(ctx, dtype, D, slopes, cap):  # noqa: F811
    """A large cap leaves the scores as they are, a tiny one makes them equal; scores of both signs up to some hundreds."""
    for news in (PROMPTS, [min(3, x) for x in PROMPTS]):
        for q_mul in (1.0, 30.0):
            c = Case(ctx, PROMPTS, news, 16, 8, D, dtype=dtype, seed=21, q_mul=q_mul)
            opts = dict(cap=cap)
            if slopes:
                opts["slopes"] = torch.exp2(-1.0 - torch.arange(16, device="cuda") / 2)
            out = c.call(**opts)
            ctx.sync_status()
            check(c, out, **opts)


def test_scratch_is_what_a_call_can_use():
    """Two partial results of 16 rows of 256 channels for each of two CTAs an SM, no more."""
    own = ggq.Context(0)
    try:
        c = Case(own, [5000], [1], 2, 1, 256)
        c.call()
        own.sync_status()
        sms = torch.cuda.get_device_properties(0).multi_processor_count
        assert own.scratch_bytes() <= 2 * 2 * sms * (16 * 256 + 32) * 4 + 256
    finally:
        own.close()
