"""Whole decoding steps of a small packed model: every operation of a step is a call of the library.

Each layer: norm (rows for the adapters, Q8_K blocks for the products), the fused query/key/value projection with
a low-rank adapter of each user beside it, rotation of positions on the way into the cache, attention, output
projection, norms around the residual, router, experts; after the last layer a norm, the vocabulary projection,
and the log probabilities of the chosen token with its alternatives.  Prompts of several users go through in one
pass; after that a step takes one token of each user, as a CUDA graph.  Weights are synthetic.

    python examples/decode_step.py [steps]
"""
import os
import sys
import time

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

import torch  # noqa: E402

import ggq_synth as syn  # noqa: E402
import gguf_block_quant_ggq_gb300 as ggq  # noqa: E402

LAYERS, HIDDEN, HEADS, KV_HEADS, DIM, VOCAB = 2, 1024, 16, 4, 64, 2048
EXPERTS, INTER, TOP_K, PAGE, ADAPTERS, RANK, BEST = 32, 256, 4, 64, 3, 8, 5
SPREAD = 2.0  # of the scaled logits
QKV = (HEADS + 2 * KV_HEADS) * DIM


class Model:
    def __init__(self, ctx, users, max_len, seed=23):
        self.ctx, g = ctx, syn.rng(seed, 0)
        pack = lambda a: torch.from_numpy(a).cuda()  # noqa: E731
        gen = torch.Generator(device="cuda")
        gen.manual_seed(seed)
        rand = lambda *s: torch.randn(s, device="cuda", generator=gen)  # noqa: E731
        self.embed = rand(VOCAB, HIDDEN)
        self.head = pack(syn.weights("Q4_K", VOCAB, HIDDEN, g))
        self.scale = 1.0  # of the logits (1 / temperature)
        self.layers = []
        for _ in range(LAYERS):
            banks = [pack(syn.expert_bank(f, EXPERTS, *s, g)) for f, s in (("Q4_K", (INTER, HIDDEN)), ("Q4_K", (INTER, HIDDEN)),
                                                                           ("Q6_K", (HIDDEN, INTER)))]
            self.layers.append(dict(
                qkv=pack(syn.weights("Q4_K", QKV, HIDDEN, g)), out=pack(syn.weights("Q4_K", HIDDEN, HEADS * DIM, g)),
                router=pack(syn.weights("Q4_K", EXPERTS, HIDDEN, g)), banks=banks,
                experts=ctx.moe_weights("Q4_K", banks[0], "Q4_K", banks[1], "Q6_K", banks[2]),
                adapters=ctx.adapters((rand(ADAPTERS, RANK, HIDDEN) * HIDDEN ** -0.5).half(), rand(ADAPTERS, QKV, RANK).half(),
                                      scales=torch.full((ADAPTERS,), 0.5, device="cuda")),
                norms=[1 + 0.1 * rand(HIDDEN) for _ in range(4)],  # before attention, after it, before the experts, after them
                cache=ctx.kv_cache("Q8_0", "Q4_0", users * ((max_len + PAGE - 1) // PAGE), PAGE, KV_HEADS, DIM)))
        self.last = 1 + 0.1 * rand(HIDDEN)
        pages = (max_len + PAGE - 1) // PAGE
        self.max_len = max_len
        # pages are handed out in turn, so that a user's are scattered over the pool
        self.table = (torch.arange(pages, device="cuda")[None] * users + torch.arange(users, device="cuda")[:, None]).int().contiguous()
        self.turns = ctx.rotary_table(max_len, DIM, factor=2.0, original_len=max_len // 2 + 1)
        self.adapter = (torch.arange(users, device="cuda", dtype=torch.int32) % (ADAPTERS + 1)) - 1  # the first user has none

    def product(self, W, rows, packed):
        """Packed rows (Q8_K) times a Q4_K matrix, eight tokens a call."""
        T = packed.shape[0]
        y = torch.empty((T, rows), device="cuda")
        for i in range(0, T, 8):
            n = min(8, T - i)
            self.ctx.mul_mat_vec_q("Q4_K", W, rows, HIDDEN, packed[i:i + n], n, Y=y[i:i + n])
        return y

    def forward(self, tokens, positions, slots, lens, q_start=None, max_q=1):
        """(hidden rows, logits) of the users' new tokens, which are already counted in lens."""
        ctx, x, y, after = self.ctx, self.embed[tokens], None, None
        for L in self.layers:
            w = L["norms"]
            rows = torch.empty_like(x)
            if y is None:
                packed, _ = ctx.norm(x, before=w[0], act="Q8_K", out=rows)
            else:
                packed, x = ctx.norm(y, after=after, residual=x, before=w[0], act="Q8_K", out=rows)
            qkv = self.product(L["qkv"], QKV, packed)
            ctx.adapt(L["adapters"], rows, qkv, self.adapter, q_start=q_start, out=qkv)
            q, k, v = qkv.view(-1, HEADS + 2 * KV_HEADS, DIM).split([HEADS, KV_HEADS, KV_HEADS], 1)
            ctx.kv_append(L["cache"], k, v, slots, self.turns, positions, q=q, q_out=q)
            a = ctx.attention(L["cache"], q, lens, self.table, q_start=q_start, max_q=max_q, max_len=self.max_len)
            o = self.product(L["out"], HIDDEN, ctx.quantize_act("Q8_K", a.view(-1, HEADS * DIM)))
            packed, x = ctx.norm(o, after=w[1], residual=x, before=w[2], act="Q8_K", out=rows)
            ids, weights = ctx.moe_route(self.product(L["router"], EXPERTS, packed), TOP_K)
            y = ctx.moe_experts(L["experts"], EXPERTS, HIDDEN, INTER, TOP_K, rows, ids=ids, route_w=weights)
            after = w[3]
        packed, x = ctx.norm(y, after=after, residual=x, before=self.last, act="Q8_K")
        return x, self.product(self.head, VOCAB, packed)

    def slots_of(self, user, pos):
        return self.table[user, pos // PAGE].long() * PAGE + pos % PAGE

    def prompts(self, tokens):
        """Prompts of all users (a list of int64 tensors) in one pass."""
        n = [t.numel() for t in tokens]
        user = torch.cat([torch.full((m,), i, device="cuda") for i, m in enumerate(n)])
        pos = torch.cat([torch.arange(m, device="cuda") for m in n])
        start = torch.tensor([sum(n[:i]) for i in range(len(n) + 1)], dtype=torch.int32, device="cuda")
        self.lens = torch.tensor(n, dtype=torch.int32, device="cuda")
        return self.forward(torch.cat(tokens), pos.int(), self.slots_of(user, pos), self.lens, start, max(n))

    def step(self):
        """One token of each user: reads self.tokens and self.lens, leaves the best next token in self.tokens."""
        user = torch.arange(self.lens.numel(), device="cuda")
        slots, pos = self.slots_of(user, self.lens.long()), self.lens.clone()
        self.lens += 1
        x, logits = self.forward(self.tokens, pos, slots, self.lens)
        best = self.ctx.logprobs(logits, top_k=1)[2]
        lp, entropy, ids, top = self.ctx.logprobs(logits, best, top_k=BEST, scale=self.scale)
        self.tokens.copy_(best[:, 0])
        return x, lp, entropy, ids, top, logits * self.scale

    def capture(self):
        lens, tokens = self.lens.clone(), self.tokens.clone()
        s = torch.cuda.Stream()
        s.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(s):  # workspaces grow before the capture; the places written are written again
            self.step()
        torch.cuda.current_stream().wait_stream(s)
        self.graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(self.graph):
            self.result = self.step()
        self.lens.copy_(lens)
        self.tokens.copy_(tokens)


def main(steps=32, prompts=(37, 200, 5, 90)):
    """(hidden rows of the prompts in one pass, the same token by token, results of the graph's steps, the same steps without
    a graph, us a graph step)"""
    torch.cuda.set_device(0)
    ctx = ggq.Context(0)
    gen = torch.Generator(device="cuda")
    gen.manual_seed(5)
    users, max_len = len(prompts), max(prompts) + steps + 1
    tokens = [torch.randint(0, VOCAB, (n,), device="cuda", generator=gen) for n in prompts]
    runs = []
    for graph in (True, False):
        model = Model(ctx, users, max_len)
        x, logits = model.prompts(tokens)
        ends = torch.tensor(prompts, device="cuda").cumsum(0) - 1
        model.scale = SPREAD / float(logits.std())  # synthetic weights know no temperature
        model.tokens = ctx.logprobs(logits[ends], top_k=1)[2][:, 0].long()
        results = []
        if graph:
            model.capture()
        torch.cuda.synchronize()
        t0 = time.perf_counter()
        for _ in range(steps):
            if graph:
                model.graph.replay()
                results.append([r.clone() for r in model.result])
            else:
                results.append(model.step())
        torch.cuda.synchronize()
        runs.append((x, results, (time.perf_counter() - t0) / max(steps, 1) * 1e6))
    # the prompts again, each user's tokens one at a time from an empty cache
    check, single = Model(ctx, users, max_len), []
    for u, t in enumerate(tokens):
        for i in range(t.numel()):
            lens = torch.zeros(users, dtype=torch.int32, device="cuda")
            lens[u] = i + 1
            start = (torch.arange(users + 1, device="cuda") > u).int()
            at = torch.tensor([i], device="cuda")
            single.append(check.forward(t[i:i + 1], at.int(), check.slots_of(torch.tensor([u], device="cuda"), at), lens, start)[0])
    ctx.sync_status()
    ctx.close()
    return runs[0][0], torch.cat(single), runs[0][1], runs[1][1], runs[0][2]


if __name__ == "__main__":
    both, alone, graph, eager, us = main(int(sys.argv[1]) if len(sys.argv) > 1 else 32)
    print(f"{both.shape[0]} prompt tokens, one pass against token by token: NMSE {float((both - alone).square().sum() / alone.square().sum()):.1e}")
    print(f"{len(graph)} steps as a graph and without: {'the same' if all(torch.equal(a, b) for g, e in zip(graph, eager) for a, b in zip(g, e)) else 'DIFFERENT'}")
    print(f"a step of 4 users: {us:.0f} us; last log probabilities {[round(float(v), 3) for v in graph[-1][1][:, 0]]}")
