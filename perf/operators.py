"""What the serving operators beside the packed products cost: the block-quantized
key/value cache (write, read back), the attention that reads it in its packed
form, and the router in front of the expert layer.

`run` computes them in plain torch operations in 32 bits (`own` false) or through
the library's calls (`own` true).  A cache pool is uint8
[n_pages][kv heads][page_size / 16][blob]; a blob holds 16 tokens of one head:
the quants in the order in which the matrix instruction takes them, then one
fp16 scale for each token and 32 channels ([16][D/32]).  With token
r = 8 o + g of the blob and channel d, quants are 32-bit words, four words of a
lane side by side: byte address ((f / 4) * 32 + lane) * 16 + (f % 4) * 4 + byte.
"""
import math

import torch

own = False

FORMAT_BYTES = {"Q8_0": 17, "Q4_0": 9}  # bytes of a blob for each channel (16 quants and half a scale)
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
    llm = {"op": "attention", "heads": 32, "kv_heads": 8, "dim": 128, "k_type": "Q8_0", "v_type": "Q8_0", "tokens": 1,
           "ragged": False, "window": 0, "cap": 0.0, "slopes": False, "page": 64}
    return [
        # one user, a short conversation: the call's latency counts
        dict(llm, name="decode 1 x 777", dtype="f32", seqs=1, length=777, page=32),
        # a serving batch in the middle of its answers
        dict(llm, name="decode 64 x 4096 ragged", dtype="bf16", seqs=64, length=4096, ragged=True),
        # few users with book-length contexts: the cache is all there is to read
        dict(llm, name="decode 4 x 131072", dtype="f32", seqs=4, length=131072),
        # 4-bit cache, narrow heads, eight query heads on one kv head, the smallest pages
        dict(llm, name="decode 33 x 16384 4-bit", dtype="f16", seqs=33, length=16384, ragged=True, heads=64, dim=64,
             k_type="Q4_0", v_type="Q4_0", page=16),
        # five drafted tokens of each user verified at once, wide heads, capped scores and a sliding window
        dict(llm, name="verify 16 x 5 capped", dtype="bf16", seqs=16, length=9001, tokens=5, ragged=True, heads=16,
             dim=256, v_type="Q4_0", window=4096, cap=50.0, page=128),
        # the second half of an 8192-token prompt
        dict(llm, name="prompt 4096 of 8192", dtype="bf16", seqs=1, length=8192, tokens=4096),
        # several prompts of different lengths in one call, fp32 activations, distance bias, an odd group of heads
        dict(llm, name="prompts 5 x 1000 ragged", dtype="f32", seqs=5, length=1231, tokens=1000, ragged=True, heads=28,
             kv_heads=4, v_type="Q4_0", slopes=True, page=16),
        # the cache's write and read-back: one decode step of a batch, and a long prompt
        {"name": "cache 64 tokens", "op": "cache", "rows": 64, "kv_heads": 8, "dim": 128, "k_type": "Q8_0",
         "v_type": "Q8_0", "dtype": "f32", "page": 64},
        {"name": "cache 16384 tokens", "op": "cache", "rows": 16384, "kv_heads": 8, "dim": 128, "k_type": "Q8_0",
         "v_type": "Q4_0", "dtype": "bf16", "page": 64},
        # routers: one token of the 128-expert layer, a batch of tokens with 16-bit logits (many ties), and the
        # 4096-token prompt with sigmoid scores, a balance bias and groups of experts
        {"name": "route 1 of 128", "op": "route", "rows": 1, "experts": 128, "top_k": 8, "scoring": "softmax",
         "groups": 1, "top_groups": 1, "dtype": "f32"},
        {"name": "route 512 of 128", "op": "route", "rows": 512, "experts": 128, "top_k": 8, "scoring": "softmax",
         "groups": 1, "top_groups": 1, "dtype": "bf16"},
        {"name": "route 4096 of 256 grouped", "op": "route", "rows": 4096, "experts": 256, "top_k": 8,
         "scoring": "sigmoid", "groups": 8, "top_groups": 4, "dtype": "f32"},
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    kind = rng.choice(["decode", "decode", "decode", "verify", "prompt", "prompt", "cache", "cache", "route", "route"])
    types = rng.choice([("Q8_0", "Q8_0"), ("Q8_0", "Q8_0"), ("Q4_0", "Q4_0"), ("Q8_0", "Q4_0"), ("Q4_0", "Q8_0")])
    dtype, page = rng.choice(["f32", "f16", "bf16"]), rng.choice([16, 32, 48, 64, 128, 256])
    if kind == "cache":
        return {"op": "cache", "rows": _log(rng, 1, 16384), "kv_heads": rng.choice([1, 2, 4, 5, 8]),
                "dim": rng.choice([64, 128]), "k_type": types[0], "v_type": types[1], "dtype": dtype, "page": page}
    if kind == "route":
        experts, groups, top = rng.choice([(8, 1, 1), (60, 1, 1), (64, 8, 3), (128, 1, 1), (160, 8, 3), (256, 8, 4),
                                           (512, 1, 1)])
        return {"op": "route", "rows": _log(rng, 1, 8192), "experts": experts, "top_k": rng.randint(1, 8),
                "scoring": "sigmoid" if groups > 1 else rng.choice(["softmax", "sigmoid"]), "groups": groups,
                "top_groups": top, "dtype": dtype}
    heads, kv_heads, dim = rng.choice([(32, 8, 128), (64, 8, 64), (16, 8, 256), (28, 4, 128), (8, 1, 128), (24, 8, 128),
                                       (12, 12, 64), (16, 1, 64)])
    case = {"op": "attention", "heads": heads, "kv_heads": kv_heads, "dim": dim, "k_type": types[0],
            "v_type": types[1], "dtype": dtype, "page": page, "ragged": rng.random() < 0.6, "tokens": 1,
            "window": rng.choice([0, 0, _log(rng, 100, 5000)]), "cap": rng.choice([0.0, 0.0, 30.0]),
            "slopes": rng.random() < 0.25}
    if kind == "prompt":
        tokens = _log(rng, 16, 4096)
        seqs = max(1, min(_log(rng, 1, 16), 4096 // tokens))
        return dict(case, tokens=tokens, seqs=seqs, length=min(8192, tokens + rng.choice([0, 0, _log(rng, 1, 4096)])))
    length = _log(rng, 16, 131072)
    most = max(1, min(256, 524288 * 1024 // (length * kv_heads * dim)))
    tokens = rng.randint(2, 6) if kind == "verify" else 1
    return dict(case, tokens=tokens, seqs=_log(rng, 1, most), length=length)


def _spread(case):
    """Cached tokens and new tokens of each sequence: `length` and `tokens`, or spread below them."""
    n = case["seqs"]
    lens, news = [], []
    for i in range(n):
        if case["ragged"] and n > 1:
            part = ((i * 7 + 3) % n) / (n - 1)  # 0 .. 1 in a mixed order
            new = case["tokens"] if case["tokens"] <= 8 else max(1, int(case["tokens"] * (0.15 + 0.85 * part)))
            old = case["length"] - case["tokens"]
            lens.append(int(old * (0.1 + 0.9 * ((i * 5 + 1) % n) / (n - 1))) + new)
            news.append(new)
        else:
            lens.append(case["length"])
            news.append(case["tokens"])
    return lens, news


def _pairs(case):
    """(keys read, query-key pairs) over all sequences, for one head."""
    keys = pairs = 0
    w = case["window"]
    for length, new in zip(*_spread(case)):
        first = length - new
        keys += length - (max(0, first + 1 - w) if w else 0)
        if not w:
            pairs += new * first + new * (new + 1) // 2
        else:
            pairs += sum(min(w, first + i + 1) for i in range(new))
    return keys, pairs


def work(case):
    size = 4 if case["dtype"] == "f32" else 2
    if case["op"] == "attention":
        keys, pairs = _pairs(case)
        tokens = sum(_spread(case)[1])
        row = case["dim"] * (FORMAT_BYTES[case["k_type"]] + FORMAT_BYTES[case["v_type"]]) / 16
        return {"bytes": keys * case["kv_heads"] * row + 2 * tokens * case["heads"] * case["dim"] * size,
                "flops": 4.0 * pairs * case["heads"] * case["dim"]}
    if case["op"] == "cache":
        values = case["rows"] * case["kv_heads"] * case["dim"]
        cache = values * (FORMAT_BYTES[case["k_type"]] + FORMAT_BYTES[case["v_type"]]) / 16
        return {"bytes": 2 * values * size + 2 * cache + 2 * values * 4 + 8 * case["rows"], "flops": 8.0 * values}
    return {"bytes": case["rows"] * (case["experts"] * size + 8 * case["top_k"]),
            "flops": 4.0 * case["rows"] * case["experts"]}


# ---------------------------------------------------------------- inputs


def _pool(fmt, groups, dim, gen):
    """Packed cache bytes of `groups` blobs: normally distributed quants, as blocks of activations have, and scales."""
    dev = gen.device
    quants = 16 * dim if fmt == "Q8_0" else 8 * dim
    pool = torch.empty((groups, FORMAT_BYTES[fmt] * dim), dtype=torch.uint8, device=dev)
    step = max(1, (1 << 27) // quants)
    for i in range(0, groups, step):
        part = pool[i:i + step]
        n = part.shape[0]
        if fmt == "Q8_0":
            part[:, :quants] = (torch.randn((n, quants), device=dev, generator=gen).mul_(50).round_()
                                .clamp_(-127, 127) + 128).to(torch.uint8)
        else:
            q = (torch.randn((n, quants, 2), device=dev, generator=gen).mul_(3).round_().clamp_(-8, 7) + 8).to(torch.uint8)
            part[:, :quants] = q[:, :, 0] | (q[:, :, 1] << 4)
        d = torch.rand((n, dim // 2), device=dev, generator=gen) + 0.5
        part[:, quants:] = (d / (50 if fmt == "Q8_0" else 3)).to(torch.float16).view(torch.uint8)
    return pool


def prepare(case, seed):
    dev = torch.device("cuda", torch.cuda.current_device())
    gen = torch.Generator(device=dev)
    gen.manual_seed(seed)
    dtype = DTYPES[case["dtype"]]
    s = {"case": case}
    if case["op"] == "route":
        s["logits"] = (torch.randn((case["rows"], case["experts"]), device=dev, generator=gen) * 1.5).to(dtype)
        s["bias"] = None
        if case["scoring"] == "sigmoid":
            s["bias"] = torch.randn(case["experts"], device=dev, generator=gen) * 0.05
        return s
    H, D, page = case["kv_heads"], case["dim"], case["page"]
    if case["op"] == "cache":
        T = case["rows"]
        # keys and values are parts of the fused projection's rows: strided
        row = torch.randn((T, 3 * H * D), device=dev, generator=gen)
        row = (row * (0.25 + row.new_empty(3 * H * D).exponential_(generator=gen))).to(dtype)
        s["k"], s["v"] = row[:, H * D:2 * H * D].view(T, H, D), row[:, 2 * H * D:].view(T, H, D)
        pages = (T + page - 1) // page + 2
        order = torch.randperm(pages, device=dev, generator=gen)
        at = torch.arange(T, device=dev) + page // 2  # the first page is half full already
        s["slots"] = order[at // page] * page + at % page
        pools = [torch.zeros((pages * H * page // 16, FORMAT_BYTES[case[t]] * D), dtype=torch.uint8, device=dev)
                 for t in ("k_type", "v_type")]
    else:
        lens, news = _spread(case)
        n = case["seqs"]
        cols = max((x + page - 1) // page for x in lens)
        used = sum((x + page - 1) // page for x in lens)
        pages = used + 1
        order = torch.randperm(pages, device=dev, generator=gen).to(torch.int32).tolist()
        table = torch.full((n, cols), order[-1], dtype=torch.int32)  # the unused entries name a page of others
        for i, x in enumerate(lens):
            c = (x + page - 1) // page
            table[i, :c] = torch.tensor(order[:c], dtype=torch.int32)
            order = order[c:]
        s["table"] = table.to(dev)
        s["lens"] = torch.tensor(lens, dtype=torch.int32, device=dev)
        s["q_start"] = torch.tensor([sum(news[:i]) for i in range(n + 1)], dtype=torch.int32, device=dev)
        s["max_len"], s["max_q"] = max(lens), max(news)
        s["q"] = (torch.randn((sum(news), case["heads"], D), device=dev, generator=gen) * 1.3).to(dtype)
        s["out"] = torch.empty_like(s["q"])
        s["slopes"] = None
        if case["slopes"]:
            s["slopes"] = torch.exp2(-8.0 * torch.arange(1, case["heads"] + 1, device=dev) / case["heads"])
        pools = [_pool(case[t], pages * H * page // 16, D, gen) for t in ("k_type", "v_type")]
    s["k_pool"], s["v_pool"], s["pages"] = pools[0], pools[1], pages
    if own:
        s["cache"] = _ctx().kv_cache(case["k_type"], case["v_type"], pages, page, H, D, k=pools[0], v=pools[1])
    return s


# ---------------------------------------------------------------- plain forms


def _places(fmt, dim, value, dev):
    """(byte, shift) of each (token, channel) of a blob of 16 tokens."""
    r, d = torch.arange(16, device=dev)[:, None], torch.arange(dim, device=dev)[None, :]
    o = r // 8
    if not value:
        lane, j, i = 4 * (r % 8) + d % 16 // 4, d // 16, d % 4
        if fmt == "Q8_0":
            f, nib = o * (dim // 16) + j, 2 * i
        else:
            f, nib = o * (dim // 32) + j // 2, i % 2 * 4 + i // 2 + 2 * (j % 2)
    else:
        lane, n = 4 * (d % 8) + r % 8 // 2, d // 8
        if fmt == "Q8_0":
            f, nib = n + 0 * r, 2 * (2 * o + r % 2) + 0 * d
        else:
            f, nib = n // 2 + 0 * r, r % 2 * 4 + 2 * o + n % 2
    return (f // 4 * 32 + lane) * 16 + f % 4 * 4 + nib // 2, nib % 2 * 4


def _values(pool, case, which, groups):
    """fp32 [..., 16, D] values of the blobs `groups`."""
    fmt, dim = case[which], case["dim"]
    byte, shift = _places(fmt, dim, which == "v_type", pool.device)
    blob = pool[groups]
    quants = 16 * dim if fmt == "Q8_0" else 8 * dim
    q = blob[..., byte.reshape(-1)].unflatten(-1, (16, dim))
    q = q.float() - 128 if fmt == "Q8_0" else (q >> shift.to(torch.uint8) & 15).float() - 8
    scale = blob[..., quants:].contiguous().view(torch.float16).float().unflatten(-1, (16, dim // 32))
    return (q.unflatten(-1, (dim // 32, 32)) * scale[..., None]).flatten(-2)


def _plain_attention(s):
    case = s["case"]
    n, H, D, page = case["seqs"], case["kv_heads"], case["dim"], case["page"]
    G = case["heads"] // H
    per = page // 16
    # blobs of each sequence and head in the order of the tokens: [seqs][heads][cols * page / 16]
    dev = s["q"].device
    blobs = (s["table"].long()[:, None, :, None] * H + torch.arange(H, device=dev)[None, :, None, None]) * per
    blobs = (blobs + torch.arange(per, device=dev)).flatten(2)
    used = (s["max_len"] + 15) // 16
    k = _values(s["k_pool"], case, "k_type", blobs[:, :, :used]).flatten(2, 3)  # [seqs][H][tokens][D]
    v = _values(s["v_pool"], case, "v_type", blobs[:, :, :used]).flatten(2, 3)
    # queries, padded to the most tokens of a sequence
    start, lens = s["q_start"].long(), s["lens"].long()
    news = start[1:] - start[:-1]
    i = torch.arange(s["max_q"], device=dev)
    there = i[None] < news[:, None]
    token = torch.where(there, start[:-1, None] + i[None], 0)
    q = s["q"][token].float().unflatten(2, (H, G)).permute(0, 2, 3, 1, 4).flatten(2, 3)  # [seqs][H][G * new][D]
    x = (q @ k.transpose(2, 3)).mul_(1.0 / math.sqrt(D)).unflatten(2, (G, -1))
    if case["cap"] > 0:
        x = x.div_(case["cap"]).tanh_().mul_(case["cap"])
    pos = lens[:, None] - news[:, None] + i[None]  # [seqs][new]
    far = pos[:, None, None, :, None] - torch.arange(used * 16, device=dev)
    if s["slopes"] is not None:
        x = x - s["slopes"].view(1, H, G, 1, 1) * far
    seen = far >= 0
    if case["window"]:
        seen &= far < case["window"]
    x = x.masked_fill_(~seen, -math.inf)
    top = x.amax(-1, keepdim=True)
    p = (x - torch.where(top == -math.inf, 0.0, top)).exp_()
    total = p.sum(-1, keepdim=True)
    # values beyond a sequence's end are no part of it, whatever the page holds
    v = v.masked_fill_((torch.arange(used * 16, device=dev)[None] >= lens[:, None])[:, None, :, None], 0.0)
    out = (p.flatten(2, 3) @ v).unflatten(2, (G, -1))
    out = torch.where(total > 0, out / total, 0.0)
    out = out.permute(0, 3, 1, 2, 4).flatten(2, 3)  # [seqs][new][heads][D]
    return out[there].to(s["q"].dtype)


def _plain_quantized(x, fmt):
    """The values that the cache's blocks of 32 stand for."""
    b = x.float().unflatten(-1, (-1, 32))
    if fmt == "Q8_0":
        d = b.abs().amax(-1, keepdim=True) / 127.0
        r = b * torch.where(d != 0, 1.0 / d, 0.0)
        q = (torch.sign(r) * torch.floor(r.abs() + 0.5)).clamp(-127, 127)
    else:
        d = b.gather(-1, b.abs().argmax(-1, keepdim=True)) / -8.0  # the first of the largest magnitude
        q = (torch.floor(b * torch.where(d != 0, 1.0 / d, 0.0) + 8.5)).clamp(0, 15) - 8
    return (q * d.to(torch.float16).float()).flatten(-2)


def _plain_route(s):
    case, k = s["case"], s["case"]["top_k"]
    x = s["logits"].float()
    if case["scoring"] == "sigmoid":
        score = 1.0 / (1.0 + torch.exp(-x))
        choice = score + s["bias"]
    else:
        e = torch.exp(x - x.amax(-1, keepdim=True))
        score = e / e.sum(-1, keepdim=True)
        choice = x  # the order of the scores
    if case["groups"] > 1:
        g = choice.unflatten(1, (case["groups"], -1))
        best = g.sort(dim=-1, descending=True).values
        kept = (best[..., 0] + best[..., 1]).sort(dim=-1, descending=True, stable=True).indices[:, :case["top_groups"]]
        open_ = torch.zeros(g.shape[:2], dtype=torch.bool, device=x.device).scatter_(1, kept, True)
        choice = g.masked_fill(~open_[..., None], -math.inf).flatten(1)
    ids = choice.sort(dim=-1, descending=True, stable=True).indices[:, :k]
    w = score.gather(1, ids)
    total = w.sum(-1, keepdim=True)
    return {"ids": ids.to(torch.int32), "weights": torch.where(total > 0, w / total, 0.0) * 2.5}


def run(s):
    case = s["case"]
    if case["op"] == "attention":
        if not own:
            return _plain_attention(s)
        return _ctx().attention(s["cache"], s["q"], s["lens"], s["table"], q_start=s["q_start"], max_q=s["max_q"],
                                max_len=s["max_len"], cap=case["cap"], window=case["window"], slopes=s["slopes"],
                                out=s["out"])
    if case["op"] == "cache":
        if not own:
            return {"k": _plain_quantized(s["k"], case["k_type"]), "v": _plain_quantized(s["v"], case["v_type"])}
        _ctx().kv_store(s["cache"], s["k"], s["v"], s["slots"])
        k, v = _ctx().kv_load(s["cache"], s["slots"])
        return {"k": k, "v": v}
    if not own:
        return _plain_route(s)
    ids, weights = _ctx().moe_route(s["logits"], case["top_k"], scoring=case["scoring"], bias=s["bias"],
                                    n_groups=case["groups"], top_groups=case["top_groups"], group_best=2, scale=2.5)
    return {"ids": ids, "weights": weights}


# ---------------------------------------------------------------- 64 bits


def _exact_blobs(pool, fmt, dim, value):
    """fp64 [blobs][16][D] by undoing the order of a blob's words with views."""
    quants = 16 * dim if fmt == "Q8_0" else 8 * dim
    w = pool[:, :quants].reshape(-1, quants // 512, 8, 4, 4, 4)  # [four words][g][t][word][byte]
    w = w.permute(0, 1, 4, 2, 3, 5).reshape(-1, quants // 128, 8, 4, 4)  # [word][g][t][byte]
    if fmt == "Q8_0":
        x = w.double() - 128
        if value:  # word = 8 channels, byte = (octet, odd token)
            x = x.reshape(-1, dim // 8, 8, 4, 2, 2).permute(0, 4, 3, 5, 1, 2)
        else:  # word = (octet, 16 channels)
            x = x.reshape(-1, 2, dim // 16, 8, 4, 4).permute(0, 1, 3, 2, 4, 5)
    else:
        x = torch.stack([w & 15, w >> 4], -1).double() - 8  # nibble p = 2 byte + high: three bits
        if value:  # p = (odd token, octet, odd eight of channels)
            x = x.reshape(-1, dim // 16, 8, 4, 2, 2, 2).permute(0, 5, 3, 4, 1, 6, 2)
        else:  # p = (odd channel, odd sixteen of channels, channel pair)
            x = x.reshape(-1, 2, dim // 32, 8, 4, 2, 2, 2).permute(0, 1, 3, 2, 6, 4, 7, 5)
    x = x.reshape(-1, 16, dim // 32, 32)
    d = pool[:, quants:].contiguous().view(torch.float16).double().reshape(-1, 16, dim // 32, 1)
    return (x * d).reshape(-1, 16, dim)


def _exact_attention(case, s):
    H, G, D, per = case["kv_heads"], case["heads"] // case["kv_heads"], case["dim"], case["page"] // 16
    out = torch.zeros(s["q"].shape, dtype=torch.float64, device=s["q"].device)
    t0 = 0
    for b, (length, new) in enumerate(zip(*_spread(case))):
        pages = s["table"][b, :(length + case["page"] - 1) // case["page"]].tolist()
        pos = torch.arange(length - new, length, device=out.device)
        key = torch.arange(length, device=out.device)
        for h in range(H):
            at = torch.tensor([(p * H + h) * per + i for p in pages for i in range(per)], device=out.device)
            k = _exact_blobs(s["k_pool"][at], case["k_type"], D, False).reshape(-1, D)[:length]
            v = _exact_blobs(s["v_pool"][at], case["v_type"], D, True).reshape(-1, D)[:length]
            for i in range(h * G, h * G + G):
                x = s["q"][t0:t0 + new, i].double() @ k.T / math.sqrt(D)
                if case["cap"] > 0:
                    x = torch.tanh(x / case["cap"]) * case["cap"]
                if s["slopes"] is not None:
                    x += float(s["slopes"][i]) * (key[None] - pos[:, None])
                no = key[None] > pos[:, None]
                if case["window"]:
                    no |= key[None] <= pos[:, None] - case["window"]
                x[no] = -math.inf
                out[t0:t0 + new, i] = torch.softmax(x, -1) @ v
        t0 += new
    return out


def _exact_quantized(x, fmt):
    b = x.double().reshape(*x.shape[:-1], -1, 32)
    if fmt == "Q8_0":
        d = b.abs().max(-1, keepdim=True).values / 127
        q = b / d
        q = torch.trunc(q + 0.5 * torch.sign(q)).clamp(-127, 127)
    else:
        d = b.gather(-1, b.abs().max(-1, keepdim=True).indices) / -8
        q = torch.trunc(b / d + 8.5).clamp(max=15) - 8
    return (torch.where(d == 0, 0.0, q) * d.half().double()).reshape(x.shape)


def _exact_route(case, s):
    x = s["logits"].double()
    score = torch.sigmoid(x) if case["scoring"] == "sigmoid" else torch.softmax(x, -1)
    choice = score + s["bias"].double() if s["bias"] is not None else score
    if case["groups"] > 1:
        g = choice.reshape(len(x), case["groups"], -1)
        limit = g.topk(2, -1).values.sum(-1)
        limit = limit >= limit.topk(case["top_groups"], -1).values[:, -1:]
        choice = torch.where(limit[..., None], g, -math.inf).reshape(x.shape)
    w = score.gather(1, choice.sort(dim=-1, descending=True, stable=True).indices[:, :case["top_k"]])
    return {"ids": None, "weights": 2.5 * w / w.sum(-1, keepdim=True)}


def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "attention":
        if work(case)["flops"] > 2e12:
            return None
        return _exact_attention(case, s)
    if case["op"] == "cache":
        return {"k": _exact_quantized(s["k"], case["k_type"]), "v": _exact_quantized(s["v"], case["v_type"])}
    return _exact_route(case, s)
