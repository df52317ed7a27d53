"""What the operators between the packed products of a decoding step cost: the norms around a block
(fused with its gate and its residual), the rotation of positions, alone and on the way into the
block-quantized key/value cache, low-rank adapters beside a shared projection, and the log
probabilities of given tokens behind the last projection.

`run` computes them in plain torch operations in 32 bits (`own` false) or through the library's
calls (`own` true).
"""
import math

import torch

own = False

FORMAT_BYTES = {"Q8_0": 17, "Q4_0": 9}  # bytes of 16 cached values
DTYPES = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}
_context = None


def _ctx():
    global _context
    if _context is None:
        import gguf_block_quant_ggq_gb300 as ggq

        _context = ggq.Context(torch.cuda.current_device())
    return _context


# ---------------------------------------------------------------- cases


def listed():
    norm = {"op": "norm", "after": False, "before": True, "gate": "none", "residual": True, "scale": 1.0, "strided": False}
    rotate = {"op": "rotate", "layout": "half", "first": 0}
    append = {"op": "append", "heads": 32, "kv_heads": 8, "dim": 128, "turn": 128, "layout": "half", "page": 64}
    adapt = {"op": "adapt", "ragged": False, "bank": "bf16"}
    return [
        # one user's token between two blocks: the residual is added and the sum normalised; latency counts
        dict(norm, name="norm 1 x 4096", dtype="f32", rows=1, width=4096),
        # a long prompt: the block's output is normalised, gated by channel, scaled, added and normalised again
        dict(norm, name="norm 4096 x 4096 gated", dtype="bf16", rows=4096, width=4096, after=True, gate="channel",
             scale=0.22),
        # a width that is no multiple of anything, rows inside wider ones, one gate a token, no second norm
        dict(norm, name="norm 300 x 2051", dtype="f16", rows=300, width=2051, after=True, before=False, gate="token",
             scale=0.5, strided=True),
        # the queries of a batch's tokens at far positions
        dict(rotate, name="rotate 64 tokens", dtype="f32", rows=64, heads=32, dim=128, turn=128, positions=131072),
        # a long prompt, interleaved pairs, the last half of each head only
        dict(rotate, name="rotate 8192 tokens", dtype="bf16", rows=8192, heads=40, dim=128, turn=64, layout="pairs",
             first=64, positions=32768),
        # one decode step of a batch: queries and keys rotated, keys and values into 64 pages of an 8-bit cache
        dict(append, name="append 64 tokens", dtype="f32", rows=64, k_type="Q8_0", v_type="Q8_0", prompt=False,
             positions=131072),
        # a long prompt into a cache of 8-bit keys and 4-bit values
        dict(append, name="append 16384 tokens", dtype="bf16", rows=16384, k_type="Q8_0", v_type="Q4_0", prompt=True,
             positions=32768),
        # one user's adapter beside the widest projection
        dict(adapt, name="adapt 1 x 4096 to 14336", dtype="f32", seqs=1, tokens=1, width=4096, out=14336, adapters=8,
             rank=16),
        # a decode batch whose users share some of 24 adapters
        dict(adapt, name="adapt 64 of 24 adapters", dtype="bf16", seqs=64, tokens=1, width=4096, out=6144, adapters=24,
             rank=64),
        # several prompts of different lengths, each with its adapter, 32-bit rows
        dict(adapt, name="adapt 5 x 1000 ragged", dtype="f32", seqs=5, tokens=1000, ragged=True, width=4096, out=4096,
             adapters=5, rank=32),
        # the sampled token of one user with the eight best
        {"name": "logprobs 1 of 131072", "op": "logprobs", "dtype": "f32", "rows": 1, "vocab": 131072, "given": 1,
         "top": 8, "masked": 0.0, "scale": 1.0},
        # scoring a prompt's tokens, 16-bit logits (many ties), an odd vocabulary
        {"name": "logprobs 2048 of 100003", "op": "logprobs", "dtype": "bf16", "rows": 2048, "vocab": 100003, "given": 1,
         "top": 5, "masked": 0.0, "scale": 1.0},
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op, dtype = rng.choice(["norm", "norm", "rotate", "append", "append", "adapt", "adapt", "logprobs"]), rng.choice(["f32", "f16", "bf16"])
    if op == "norm":
        width = _log(rng, 64, 16384)
        width -= rng.choice([0, width % 4, width % 32, width % 256 if width >= 256 else 0])
        after = rng.random() < 0.6
        return {"op": op, "dtype": dtype, "rows": _log(rng, 1, min(8192, 16777216 // width)), "width": width, "after": after,
                "before": not after or rng.random() < 0.6, "gate": rng.choice(["none", "channel", "token", "sigmoid"]),
                "residual": rng.random() < 0.8, "scale": rng.choice([1.0, 0.22]), "strided": rng.random() < 0.4}
    layout = rng.choice(["half", "pairs"])
    if op == "rotate":
        dim = rng.choice([64, 80, 96, 128, 192, 256])
        turn = rng.choice([dim, dim, dim // 2])
        heads = rng.choice([1, 4, 16, 28, 32, 40])
        return {"op": op, "dtype": dtype, "rows": _log(rng, 1, 41943040 // (heads * dim) if heads * dim > 5120 else 8192),
                "heads": heads, "dim": dim, "turn": turn, "layout": layout, "first": rng.choice([0, dim - turn]),
                "positions": _log(rng, 1024, 131072)}
    if op == "append":
        heads, kv_heads, dim = rng.choice([(32, 8, 128), (64, 8, 64), (16, 8, 256), (28, 4, 128), (24, 8, 128), (16, 1, 64)])
        types = rng.choice([("Q8_0", "Q8_0"), ("Q8_0", "Q8_0"), ("Q4_0", "Q4_0"), ("Q8_0", "Q4_0"), ("Q4_0", "Q8_0")])
        prompt = rng.random() < 0.5
        return {"op": op, "dtype": dtype, "heads": heads, "kv_heads": kv_heads, "dim": dim,
                "turn": rng.choice([dim, dim, dim // 2]), "layout": layout, "page": rng.choice([16, 32, 48, 64, 128]),
                "rows": _log(rng, 1, 8192 if prompt else 512), "k_type": types[0], "v_type": types[1], "prompt": prompt,
                "positions": _log(rng, 1024, 131072)}
    if op == "adapt":
        rank = rng.choice([4, 8, 16, 24, 32, 64, 128])
        width, out = rng.choice([(1024, 1024), (2048, 1536), (4096, 1024), (4096, 4096), (4096, 14336), (14336, 4096)])
        case = {"op": op, "dtype": dtype, "bank": rng.choice(["bf16", "f16"]), "width": width, "out": out, "rank": rank,
                "adapters": _log(rng, 1, 32)}
        if rng.random() < 0.5:
            return dict(case, seqs=_log(rng, 1, 256), tokens=1, ragged=False)
        tokens = _log(rng, 2, 2048)
        return dict(case, seqs=max(1, min(_log(rng, 1, 16), 4096 // tokens)), tokens=tokens, ragged=rng.random() < 0.7)
    vocab = _log(rng, 8192, 262144)
    return {"op": op, "dtype": dtype, "rows": _log(rng, 1, min(2048, 134217728 // vocab)), "vocab": vocab,
            "given": rng.choice([1, 1, 4]), "top": rng.choice([0, 1, 5, 8, 20]), "masked": rng.choice([0.0, 0.0, 0.4]),
            "scale": rng.choice([1.0, 0.7])}


def _news(case):
    """New tokens of each sequence: `tokens`, or spread below it."""
    n = case["seqs"]
    if not case["ragged"] or n == 1:
        return [case["tokens"]] * n
    return [max(1, int(case["tokens"] * (0.15 + 0.85 * ((i * 7 + 3) % n) / (n - 1)))) for i in range(n)]


def _users(case):
    """(adapter of each sequence, rank of each adapter): shared unevenly, one user in nine has none, ranks differ."""
    ids = [-1 if i % 9 == 8 else (i * i + 3 * i) % case["adapters"] for i in range(case["seqs"])]
    ranks = [case["rank"] if a % 3 else max(1, case["rank"] * 3 // 4) for a in range(case["adapters"])]
    return ids, ranks


def work(case):
    size = 4 if case["dtype"] == "f32" else 2
    if case["op"] == "norm":
        n = case["rows"] * case["width"]
        gate = n if case["gate"] == "channel" else case["width"] if case["gate"] == "sigmoid" else case["rows"] if case["gate"] == "token" else 0
        total = case["residual"] or not case["before"]
        moved = n * (1 + case["residual"] + total + case["before"]) + gate
        return {"bytes": moved * size + 4 * case["width"] * (case["after"] + case["before"]), "flops": 12.0 * n}
    if case["op"] == "rotate":
        n = case["rows"] * case["heads"]
        return {"bytes": 2 * n * case["dim"] * size + case["rows"] * (4 * case["turn"] + 4), "flops": 3.0 * n * case["turn"]}
    if case["op"] == "append":
        q, kv = case["rows"] * case["heads"] * case["dim"], case["rows"] * case["kv_heads"] * case["dim"]
        cache = kv * (FORMAT_BYTES[case["k_type"]] + FORMAT_BYTES[case["v_type"]]) / 16
        # written, and read back as the values that they stand for
        return {"bytes": 2 * q * size + 4 * kv * size + 2 * cache + case["rows"] * (4 * case["turn"] + 12), "flops": 3.0 * q + 11.0 * kv}
    if case["op"] == "adapt":
        ids, ranks = _users(case)
        both, news = case["width"] + case["out"], _news(case)
        used = sum(ranks[a] for a in set(ids) if a >= 0) * both
        return {"bytes": sum(news) * (case["width"] + 2 * case["out"]) * size + 2 * used,
                "flops": 2.0 * both * sum(n * ranks[a] for n, a in zip(news, ids) if a >= 0)}
    return {"bytes": case["rows"] * (case["vocab"] * size + 8 * case["given"] + 4 + 8 * case["top"]),
            "flops": 6.0 * case["rows"] * case["vocab"]}


# ---------------------------------------------------------------- inputs


def _table(case, dev):
    """fp32 [positions][turn / 2][2]: cosine and sine of each position's angles, slowed down fourfold where the table is long."""
    half = case["turn"] // 2
    freq = 10000.0 ** (-torch.arange(half, dtype=torch.float64, device=dev) / half)
    if case["positions"] > 32768:
        freq = freq / 4.0
    angle = torch.arange(case["positions"], dtype=torch.float64, device=dev)[:, None] * freq
    return torch.stack([angle.cos(), angle.sin()], -1).float()


def prepare(case, seed):
    dev = torch.device("cuda", torch.cuda.current_device())
    gen = torch.Generator(device=dev)
    gen.manual_seed(seed)
    dtype = DTYPES[case["dtype"]]
    s = {"case": case}

    def randn(*shape):
        return torch.randn(shape, device=dev, generator=gen)

    if case["op"] == "norm":
        n, w = case["rows"], case["width"]
        # some channels are far larger than the others, as in trained models
        size = torch.exp(randn(w))
        wide = (randn(n, w + 64 * case["strided"]) * torch.cat([size, size.new_ones(64 * case["strided"])])).to(dtype)
        s["x"] = wide[:, :w]
        s["residual"] = (randn(n, w) * 4 * size).to(dtype) if case["residual"] else None
        s["after"] = 1 + 0.3 * randn(w) if case["after"] else None
        s["before"] = 1 + 0.3 * randn(w) if case["before"] else None
        s["gate"] = None
        if case["gate"] != "none":
            s["gate"] = randn(*{"channel": (n, w), "token": (n, 1), "sigmoid": (w,)}[case["gate"]]).to(dtype)
        s["out"] = torch.empty((n, w), dtype=dtype, device=dev) if case["before"] else None
        s["total"] = torch.empty((n, w), dtype=dtype, device=dev) if case["residual"] or not case["before"] else None
        return s
    if case["op"] == "rotate":
        n = case["rows"]
        s["x"] = randn(n, case["heads"], case["dim"]).to(dtype)
        s["out"] = torch.empty_like(s["x"])
        s["table"] = _table(case, dev)
        s["positions"] = torch.randint(0, case["positions"], (n,), device=dev, generator=gen, dtype=torch.int32)
        return s
    if case["op"] == "append":
        n, H, D, page = case["rows"], case["kv_heads"], case["dim"], case["page"]
        # queries, keys and values are parts of the fused projection's rows
        row = randn(n, (case["heads"] + 2 * H) * D)
        row = (row * (0.25 + row.new_empty(row.shape[1]).exponential_(generator=gen))).to(dtype).unflatten(1, (-1, D))
        s["q"], s["k"], s["v"] = row.split([case["heads"], H, H], 1)
        s["q_out"] = torch.empty((n, case["heads"], D), dtype=dtype, device=dev)
        s["table"] = _table(case, dev)
        if case["prompt"]:  # consecutive places, from the middle of a page on
            at = torch.arange(n, device=dev) + page // 2
            pages = (n + page - 1) // page + 2
            first = int(torch.randint(0, max(1, case["positions"] - n), (1,), generator=torch.Generator().manual_seed(seed)))
            s["positions"] = ((first + torch.arange(n, device=dev)) % case["positions"]).int()
        else:  # a page of its own for each token
            pages = n + 1
            s["positions"] = torch.randint(0, case["positions"], (n,), device=dev, generator=gen, dtype=torch.int32)
            at = torch.arange(n, device=dev) * page + s["positions"].long() % page
        order = torch.randperm(pages, device=dev, generator=gen)
        s["slots"] = order[at // page] * page + at % page
        s["k_back"], s["v_back"] = (torch.empty((n, H, D), dtype=dtype, device=dev) for _ in range(2))
        if own:
            s["cache"] = _ctx().kv_cache(case["k_type"], case["v_type"], pages, page, H, D)
        return s
    if case["op"] == "adapt":
        ids, ranks = _users(case)
        news, R = _news(case), case["rank"]
        bank = DTYPES[case["bank"]]
        s["x"] = randn(sum(news), case["width"]).to(dtype)
        s["y"] = randn(sum(news), case["out"]).to(dtype)
        s["a"] = (randn(case["adapters"], R, case["width"]) / math.sqrt(case["width"])).to(bank)
        s["b"] = (randn(case["adapters"], case["out"], R) * 0.3).to(bank)
        s["ids"] = torch.tensor(ids, dtype=torch.int32, device=dev)
        s["ranks"] = torch.tensor(ranks, dtype=torch.int32, device=dev)
        s["scales"] = 16.0 / s["ranks"].float()
        s["q_start"], s["max_q"] = None, max(news)
        if case["tokens"] > 1:
            s["q_start"] = torch.tensor([sum(news[:i]) for i in range(len(news) + 1)], dtype=torch.int32, device=dev)
        s["out"] = torch.empty_like(s["y"])
        if own:
            s["adapters"] = _ctx().adapters(s["a"], s["b"], ranks=s["ranks"], scales=s["scales"])
        return s
    n, V = case["rows"], case["vocab"]
    x = torch.empty((n, V), dtype=dtype, device=dev)
    for i in range(0, n, 256):  # a few tokens of a row stand out
        part = randn(*x[i:i + 256].shape).mul_(2.0)
        best = torch.randint(0, V, (part.shape[0], 6), device=dev, generator=gen)
        part.scatter_add_(1, best, randn(*best.shape).abs() * 5)
        if case["masked"]:  # a grammar allows a part of the vocabulary
            part.masked_fill_(torch.rand(V, device=dev, generator=gen) < case["masked"], -math.inf)
        x[i:i + 256] = part
    s["logits"] = x
    s["tokens"] = torch.randint(0, V, (n, case["given"]), device=dev, generator=gen, dtype=torch.int32)
    s["logprobs"] = torch.empty((n, case["given"]), device=dev)
    s["entropy"] = torch.empty(n, device=dev)
    s["ids"] = torch.empty((n, case["top"]), dtype=torch.int32, device=dev)
    s["top"] = torch.empty((n, case["top"]), device=dev)
    return s


# ---------------------------------------------------------------- plain forms


def _plain_norm(s):
    case = s["case"]
    x = s["x"].float()
    if case["after"]:
        x = x * torch.rsqrt(x.square().mean(-1, keepdim=True) + 1e-6) * s["after"]
    if s["gate"] is not None:
        gate = s["gate"].float()
        x = x * (1.0 / (1.0 + torch.exp(-gate)) if case["gate"] == "sigmoid" else gate)
    x = x * case["scale"]
    if s["residual"] is not None:
        x = x + s["residual"].float()
    got = {}
    if s["total"] is not None:
        got["total"] = x.to(s["x"].dtype)
    if case["before"]:
        got["out"] = (x * torch.rsqrt(x.square().mean(-1, keepdim=True) + 1e-6) * s["before"]).to(s["x"].dtype)
    return got


def _turned(x, table, positions, layout, first):
    """fp32 rows [tokens][heads][D] with the channels from `first` on turned by the table's angles."""
    half = table.shape[1]
    c, sn = table[positions.long()][:, None].unbind(-1)
    part = x[..., first:first + 2 * half]
    a, b = part.unflatten(-1, (half, 2)).unbind(-1) if layout == "pairs" else part.split(half, -1)
    new = torch.stack([a * c - b * sn, a * sn + b * c], -1 if layout == "pairs" else -2).flatten(-2)
    return torch.cat([x[..., :first], new, x[..., first + 2 * half:]], -1)


def _plain_quantized(x, fmt):
    """The values that the cache's blocks of 32 stand for."""
    b = x.unflatten(-1, (-1, 32))
    if fmt == "Q8_0":
        d = b.abs().amax(-1, keepdim=True) * torch.tensor(1 / 127, dtype=torch.float32, device=x.device)
        r = b * torch.where(d != 0, 1.0 / d, 0.0)
        q = (torch.sign(r) * torch.floor(r.abs().double() + 0.5).float()).clamp(-127, 127)
    else:
        d = b.gather(-1, b.abs().argmax(-1, keepdim=True)) / -8.0  # the first of the largest magnitude
        q = (torch.floor(b * torch.where(d != 0, 1.0 / d, 0.0) + 8.5)).clamp(0, 15) - 8
    return (q * d.to(torch.float16).float()).flatten(-2)


def _plain_append(s):
    case, dtype = s["case"], s["q"].dtype
    q, k = (_turned(s[n].float(), s["table"], s["positions"], case["layout"], 0) for n in "qk")
    return {"q": q.to(dtype), "k": _plain_quantized(k, case["k_type"]).to(dtype),
            "v": _plain_quantized(s["v"].float(), case["v_type"]).to(dtype)}


def _plain_adapt(s):
    n, ids = s["x"].shape[0], s["ids"].long()
    start = s["q_start"].long() if s["q_start"] is not None else torch.arange(n + 1, device=ids.device)
    # rows padded to the most tokens of a sequence, a sequence's own bank
    i = torch.arange(s["max_q"], device=ids.device)
    there = i[None] < (start[1:] - start[:-1])[:, None]
    x = s["x"][torch.where(there, start[:-1, None] + i[None], 0)].float()
    own_bank = ids.clamp(min=0)
    rank = torch.where(ids >= 0, s["ranks"][own_bank], 0)
    a, b = s["a"][own_bank].float(), s["b"][own_bank].float()
    t = x @ a.transpose(1, 2) * s["scales"][own_bank][:, None, None]
    t = t.masked_fill(torch.arange(a.shape[1], device=ids.device)[None, None] >= rank[:, None, None], 0.0)
    return (s["y"].float() + (t @ b.transpose(1, 2))[there]).to(s["y"].dtype)


def _plain_logprobs(s):
    case = s["case"]
    x = s["logits"].float() * case["scale"]
    top = x.amax(-1, keepdim=True)
    e = torch.exp(x - top)
    total = e.sum(-1, keepdim=True)
    log = total.log()
    spread = torch.where(e > 0, (x - top) * e, 0.0).sum(-1, keepdim=True)
    got = {"logprobs": x.gather(1, s["tokens"].long()) - top - log, "entropy": (log - spread / total)[:, 0]}
    if case["top"]:
        ids = x.sort(dim=-1, descending=True, stable=True).indices[:, :case["top"]]
        got["ids"], got["top"] = ids.int(), x.gather(1, ids) - top - log
    return got


def _own(s):
    case, ctx = s["case"], _ctx()
    if case["op"] == "norm":
        out, total = ctx.norm(s["x"], after=s["after"], gate=s["gate"], gate_act="sigmoid" if case["gate"] == "sigmoid" else "none",
                              scale=case["scale"], residual=s["residual"], before=s["before"], out=s["out"], total=s["total"])
        return {"out": out, "total": total}
    if case["op"] == "rotate":
        return {"x": ctx.rotate(s["x"], s["table"], s["positions"], layout=case["layout"], first=case["first"], out=s["out"])}
    if case["op"] == "append":
        q = ctx.kv_append(s["cache"], s["k"], s["v"], s["slots"], s["table"], s["positions"], layout=case["layout"], q=s["q"],
                          q_out=s["q_out"])
        k, v = ctx.kv_load(s["cache"], s["slots"], k=s["k_back"], v=s["v_back"])
        return {"q": q, "k": k, "v": v}
    if case["op"] == "adapt":
        return {"y": ctx.adapt(s["adapters"], s["x"], s["y"], s["ids"], q_start=s["q_start"], out=s["out"])}
    top = case["top"]
    got = ctx.logprobs(s["logits"], s["tokens"], top_k=top, scale=case["scale"], logprobs=s["logprobs"], entropy=s["entropy"],
                       ids=s["ids"] if top else None, top=s["top"] if top else None)
    return dict(zip(("logprobs", "entropy", "ids", "top") if top else ("logprobs", "entropy"), got))


def run(s):
    case = s["case"]
    if own:
        return _own(s)
    if case["op"] == "norm":
        return _plain_norm(s)
    if case["op"] == "rotate":
        return {"x": _turned(s["x"].float(), s["table"], s["positions"], case["layout"], case["first"]).to(s["x"].dtype)}
    if case["op"] == "append":
        return _plain_append(s)
    if case["op"] == "adapt":
        return {"y": _plain_adapt(s)}
    return _plain_logprobs(s)


# ---------------------------------------------------------------- 64 bits


def _exact_rms(x, w):
    return x / (x.pow(2).sum(1, keepdim=True) / x.shape[1] + 1e-6).sqrt() * w.double()


def _exact_turned(x, s, layout, first):
    """Pairs of channels as complex numbers, turned by the table's complex ones."""
    x = x.double().clone()
    half = s["table"].shape[1]
    z = torch.view_as_complex(s["table"].double()[s["positions"].long()])[:, None]
    even = torch.arange(half, device=x.device) * (2 if layout == "pairs" else 1) + first
    odd = even + (1 if layout == "pairs" else half)
    w = torch.complex(x[..., even], x[..., odd]) * z
    x[..., even], x[..., odd] = w.real, w.imag
    return x


def _exact_quantized(x, fmt):
    b = x.reshape(*x.shape[:-1], -1, 32)
    if fmt == "Q8_0":
        d = b.abs().max(-1, keepdim=True).values / 127
        q = b / d
        q = torch.trunc(q + 0.5 * torch.sign(q)).clamp(-127, 127)
    else:
        d = b.gather(-1, b.abs().max(-1, keepdim=True).indices) / -8
        q = torch.trunc(b / d + 8.5).clamp(max=15) - 8
    return (torch.where(d == 0, 0.0, q) * d.half().double()).reshape(x.shape)


def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "norm":
        t = s["x"].double()
        if case["after"]:
            t = _exact_rms(t, s["after"])
        if s["gate"] is not None:
            t = t * (torch.sigmoid(s["gate"].double()) if case["gate"] == "sigmoid" else s["gate"].double())
        t = t * case["scale"] + (s["residual"].double() if case["residual"] else 0.0)
        return {"out": _exact_rms(t, s["before"]) if case["before"] else None, "total": t if s["total"] is not None else None}
    if case["op"] == "rotate":
        return {"x": _exact_turned(s["x"], s, case["layout"], case["first"])}
    if case["op"] == "append":
        return {"q": _exact_turned(s["q"], s, case["layout"], 0),
                "k": _exact_quantized(_exact_turned(s["k"], s, case["layout"], 0), case["k_type"]),
                "v": _exact_quantized(s["v"].double(), case["v_type"])}
    if case["op"] == "adapt":
        if work(case)["flops"] > 1e11:
            return None
        ids, ranks = _users(case)
        y, at = s["y"].double(), 0
        for a, n in zip(ids, _news(case)):
            if a >= 0:
                r = ranks[a]
                y[at:at + n] += float(s["scales"][a]) * ((s["x"][at:at + n].double() @ s["a"][a, :r].double().T) @ s["b"][a, :, :r].double().T)
            at += n
        return {"y": y}
    parts = []
    for i in range(0, case["rows"], 64):
        p = torch.log_softmax(s["logits"][i:i + 64].double() * case["scale"], -1)
        got = [p.gather(1, s["tokens"][i:i + 64].long()), -torch.xlogy(p.exp(), p.exp()).sum(-1)]
        parts.append(got + ([p.topk(case["top"], -1).values] if case["top"] else []))
    got = [torch.cat(x) for x in zip(*parts)]
    return {"logprobs": got[0], "entropy": got[1], "ids": None, "top": got[2] if case["top"] else None}
