"""One attention + expert layer, packed from end to end, as a serving loop runs it.

Prompts of several users go through the layer in one call each of kv_store,
attention, moe_route and moe_experts; after that every step takes one token of each
user, as a CUDA graph that reads the lengths and the page table from device memory.
Projections are matrix-vector products on Q4_K weights (8 tokens a call), the cache is
Q8_0 keys and Q4_0 values, the experts Q4_K and Q6_K.  Weights are synthetic.

    python examples/decode_layer.py [steps]
"""
import os
import sys
import time

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

import torch  # noqa: E402

import ggq_synth as syn  # noqa: E402
import gguf_block_quant_ggq_gb300 as ggq  # noqa: E402

HIDDEN, HEADS, KV_HEADS, DIM = 1024, 16, 4, 64
EXPERTS, INTER, TOP_K, PAGE = 32, 256, 4, 64


class Layer:
    def __init__(self, ctx, users, max_len, seed=17):
        self.ctx, g = ctx, syn.rng(seed, 0)
        pack = lambda a: torch.from_numpy(a).cuda()  # noqa: E731
        qkv = (HEADS + 2 * KV_HEADS) * DIM
        self.w_qkv, self.w_out = pack(syn.weights("Q4_K", qkv, HIDDEN, g)), pack(syn.weights("Q4_K", HIDDEN, HEADS * DIM, g))
        self.w_router = pack(syn.weights("Q4_K", EXPERTS, HIDDEN, g))
        self.banks = [pack(syn.expert_bank("Q4_K", EXPERTS, INTER, HIDDEN, g)), pack(syn.expert_bank("Q4_K", EXPERTS, INTER, HIDDEN, g)),
                      pack(syn.expert_bank("Q6_K", EXPERTS, HIDDEN, INTER, g))]
        self.experts = ctx.moe_weights("Q4_K", self.banks[0], "Q4_K", self.banks[1], "Q6_K", self.banks[2])
        pages = (max_len + PAGE - 1) // PAGE
        self.max_len = max_len
        self.cache = ctx.kv_cache("Q8_0", "Q4_0", users * pages, PAGE, KV_HEADS, DIM)
        # pages are handed out in turn, so that a user's are scattered over the pool
        self.table = (torch.arange(pages, device="cuda")[None] * users + torch.arange(users, device="cuda")[:, None]).int().contiguous()
        self.slopes = torch.exp2(-8.0 * torch.arange(1, HEADS + 1, device="cuda") / HEADS)  # positions enter as a distance bias

    def project(self, W, rows, x):
        y = torch.empty((x.shape[0], rows), device=x.device)
        for i in range(0, x.shape[0], 8):
            self.ctx.mul_mat_vec("Q4_K", W, rows, x.shape[1], x[i:i + 8], Y=y[i:i + 8])
        return y

    @staticmethod
    def norm(x):
        return x * torch.rsqrt(x.square().mean(-1, keepdim=True) + 1e-6)

    def forward(self, x, lens, slots, q_start=None, max_q=1):
        """x [tokens][hidden]: each user's new tokens, already counted in lens; slots: their places in the cache."""
        qkv = self.project(self.w_qkv, (HEADS + 2 * KV_HEADS) * DIM, self.norm(x)).view(-1, HEADS + 2 * KV_HEADS, DIM)
        q, k, v = qkv.split([HEADS, KV_HEADS, KV_HEADS], 1)
        self.ctx.kv_store(self.cache, k, v, slots)
        a = self.ctx.attention(self.cache, q, lens, self.table, q_start=q_start, max_q=max_q, max_len=self.max_len,
                               slopes=self.slopes)
        x = x + self.norm(self.project(self.w_out, HIDDEN, a.view(-1, HEADS * DIM)))
        n = self.norm(x)
        ids, weights = self.ctx.moe_route(self.project(self.w_router, EXPERTS, n), TOP_K)
        return x + self.norm(self.ctx.moe_experts(self.experts, EXPERTS, HIDDEN, INTER, TOP_K, n, ids=ids, route_w=weights))

    def slots_of(self, user, pos):
        """Cache places of positions pos of users (int64 tensors of one shape)."""
        return self.table[user, pos // PAGE].long() * PAGE + pos % PAGE

    def prompts(self, xs):
        """Prompts of all users (a list of [tokens][hidden]) in one pass; their outputs, one after another."""
        n = [x.shape[0] for x in xs]
        user = torch.cat([torch.full((m,), i, device="cuda") for i, m in enumerate(n)])
        pos = torch.cat([torch.arange(m, device="cuda") for m in n])
        start = torch.tensor([sum(n[:i]) for i in range(len(n) + 1)], dtype=torch.int32, device="cuda")
        self.lens = torch.tensor(n, dtype=torch.int32, device="cuda")
        return self.forward(torch.cat(xs), self.lens, self.slots_of(user, pos), start, max(n))

    def capture(self, users):
        """The decode step as a graph: self.x holds each user's token, self.y receives the layer's output."""
        self.x = torch.zeros((users, HIDDEN), device="cuda")
        self.user = torch.arange(users, device="cuda")

        def step():
            slots = self.slots_of(self.user, self.lens.long())
            self.lens += 1
            return self.forward(self.x, self.lens, slots)

        lens = self.lens.clone()
        s = torch.cuda.Stream()
        s.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(s):  # workspaces grow before the capture; the place written is written again
            step()
        torch.cuda.current_stream().wait_stream(s)
        self.lens.copy_(lens)
        self.graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(self.graph):
            self.y = step()
        self.lens.copy_(lens)


def main(steps=64, prompts=(37, 200, 5, 90)):
    """(outputs of all positions through prompts and graph, the same token by token, us a graph step)"""
    torch.cuda.set_device(0)
    ctx = ggq.Context(0)
    g = torch.Generator(device="cuda")
    g.manual_seed(3)
    users, max_len = len(prompts), max(prompts) + steps
    xs = [torch.randn((n + steps, HIDDEN), device="cuda", generator=g) for n in prompts]
    layer = Layer(ctx, users, max_len)
    y = layer.prompts([x[:n] for x, n in zip(xs, prompts)]).split(list(prompts))
    outs = [[part] for part in y]
    layer.capture(users)
    torch.cuda.synchronize()
    t0 = time.perf_counter()
    for i in range(steps):
        layer.x.copy_(torch.stack([x[n + i] for x, n in zip(xs, prompts)]))
        layer.graph.replay()
        for u in range(users):
            outs[u].append(layer.y[u:u + 1].clone())
    torch.cuda.synchronize()
    us = (time.perf_counter() - t0) / steps * 1e6
    # the same, each user's tokens one at a time from an empty cache
    check = Layer(ctx, users, max_len)
    single = []
    for u, x in enumerate(xs):
        rows = []
        for i in range(x.shape[0]):
            lens = torch.zeros(users, dtype=torch.int32, device="cuda")
            lens[u] = i + 1
            start = (torch.arange(users + 1, device="cuda") > u).int()
            rows.append(check.forward(x[i:i + 1], lens, check.slots_of(torch.tensor([u], device="cuda"), torch.tensor([i], device="cuda")), start))
        single.append(torch.cat(rows))
    ctx.sync_status()
    ctx.close()
    return [torch.cat(o) for o in outs], single, us


if __name__ == "__main__":
    both, alone, us = main(int(sys.argv[1]) if len(sys.argv) > 1 else 64)
    for u, (a, b) in enumerate(zip(both, alone)):
        print(f"user {u}: {a.shape[0]} tokens, prompt + graph against token by token: "
              f"NMSE {float((a - b).square().sum() / b.square().sum()):.1e}")
    print(f"decode step of {len(both)} users: {us:.0f} us")
