"""Text generation with slot-pool MoE layers: prefill and decode steps of a small random transformer.

Each step runs the library's serving operators in the order a server does:

    tables   once a step: pages for the new tokens, row starts, positions, cache slots
    qkv      per layer: norm + rotation of queries and keys, K and V into the paged cache
    forward  per layer: attention of the new tokens over the cache
    (pool)   per layer: the routed experts from the slot pool
    sample   once a step: the next token of every request

The plain projections, the residual norms and the embedding are torch calls.  Run it with

    python examples/generate.py [--requests 4] [--tokens 24] [--temperature 0.8]
"""
import argparse
import os
import sys

import numpy as np
import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import expert_offload_slot_gb300 as moe  # noqa: E402

LAYERS, HIDDEN, EXPERTS, TOP_K, INTER, VOCAB = 2, 256, 8, 2, 128, 1000
Q_HEADS, KV_HEADS, HEAD_DIM, PAGE = 8, 2, 64, 16


def rms(x):
    return x * torch.rsqrt(x.square().mean(-1, keepdim=True) + 1e-6)


class Server:
    """The weights, the expert pool, the paged cache and the requests' state of a small fp32 model."""

    def __init__(self, requests, max_len, max_rows=1024, seed=0):
        self.R, self.max_len = requests, max_len
        gen = torch.Generator("cuda").manual_seed(seed)

        def weight(*shape, scale):
            return torch.randn(*shape, generator=gen, device="cuda") * scale
        width = (Q_HEADS + 2 * KV_HEADS) * HEAD_DIM
        self.embed = weight(VOCAB, HIDDEN, scale=1.0)
        self.unembed = weight(HIDDEN, VOCAB, scale=0.2)
        self.wqkv = [weight(HIDDEN, width, scale=HIDDEN ** -0.5) for _ in range(LAYERS)]
        self.wo = [weight(Q_HEADS * HEAD_DIM, HIDDEN, scale=(Q_HEADS * HEAD_DIM) ** -0.5) for _ in range(LAYERS)]
        self.q_norm = [1 + weight(HEAD_DIM, scale=0.1) for _ in range(LAYERS)]
        self.k_norm = [1 + weight(HEAD_DIM, scale=0.1) for _ in range(LAYERS)]
        self._experts(np.random.default_rng(seed), max_rows)
        # attention: one handle for all layers, one cache pair per layer, and the page list
        self.attn = moe.Attention(moe.make_attn_config(Q_HEADS, KV_HEADS, HEAD_DIM, PAGE, moe.MOE_F32))
        self.width = -(-max_len // PAGE)
        pages = requests * self.width
        self.k_cache, self.v_cache = ([torch.empty(pages, KV_HEADS, PAGE, HEAD_DIM, device="cuda") for _ in range(LAYERS)]
                                      for _ in range(2))
        self.free_pages = torch.randperm(pages, device="cuda", generator=gen).int()
        half = HEAD_DIM // 2
        angle = torch.arange(max_len, device="cuda")[:, None] * 10000.0 ** (-torch.arange(half, device="cuda") / half)
        self.rope = torch.cat([angle.cos(), angle.sin()], 1).contiguous()
        self.reset()

    def _experts(self, rng, max_rows):
        """Half of the experts have a slot; the others stay in the pinned host pool until a step needs them."""
        slots = LAYERS * EXPERTS // 2
        self.cfg = moe.make_config(LAYERS, EXPERTS, TOP_K, HIDDEN, INTER, slots, moe.MOE_F32, moe.MOE_F32, max_tokens=max_rows)
        record = moe.moe_expert_layout(self.cfg)[4]
        self.host = moe.HostPool(LAYERS * EXPERTS * record)
        for i in range(LAYERS * EXPERTS):
            mats = [rng.standard_normal(s, np.float32) * 0.05 for s in ((INTER, HIDDEN), (INTER, HIDDEN), (HIDDEN, INTER))]
            self.host.numpy()[i * record:(i + 1) * record] = moe.moe_pack_expert_record(self.cfg, *mats)
        self.router = torch.from_numpy(rng.standard_normal((LAYERS, EXPERTS, HIDDEN), np.float32) * 0.05).cuda()
        self.router_bias = torch.zeros(LAYERS, EXPERTS, device="cuda")
        self.pool = moe.Pool(self.cfg, self.host.ptr, self.host.nbytes, self.router, self.router_bias)
        lut = np.full((LAYERS, EXPERTS), -1, np.int32)
        for slot in range(slots):
            lut[slot % LAYERS, slot // LAYERS] = slot
        self.pool.set_lut(lut)

    def reset(self):
        """Forget every request: empty tables, all pages free."""
        ints = dict(dtype=torch.int32, device="cuda")
        self.table = torch.zeros(self.R, self.width, **ints)
        self.ctx = torch.zeros(self.R, **ints)
        self.head = torch.zeros(1, **ints)
        self.row_start, self.seq = torch.zeros(self.R + 1, **ints), torch.zeros(self.R, **ints)

    def step(self, tokens, new):
        """tokens: the new tokens of all requests, one request after another; new: how many of each (host list).
        Returns the logits after each request's last token, [R, VOCAB]."""
        ints = dict(dtype=torch.int32, device="cuda")
        rows = len(tokens)
        positions, slots = torch.empty(rows, **ints), torch.empty(rows, **ints)
        self.attn.tables(self.ctx, torch.tensor(new, **ints), self.table, self.free_pages, self.head, self.head,
                         self.row_start, self.seq, positions, slots)
        x = self.embed[tokens]
        q = torch.empty(rows, Q_HEADS, HEAD_DIM, device="cuda")
        out, ffn = torch.empty_like(q), torch.empty_like(x)
        for l in range(LAYERS):
            self.attn.qkv(rms(x) @ self.wqkv[l], self.q_norm[l], self.k_norm[l], self.rope, positions, slots, q,
                          self.k_cache[l], self.v_cache[l])
            self.attn.forward(q, self.row_start, self.seq, max(new), self.k_cache[l], self.v_cache[l], self.table, out)
            x = x + out.flatten(1) @ self.wo[l]
            self.pool.forward(l, rms(x), ffn)
            x = x + ffn
        self.ctx.copy_(self.seq)
        last = self.row_start[1:].long() - 1
        return rms(x[last]) @ self.unembed

    def close(self):
        self.attn.close()
        self.pool.close()
        self.host.free()


def generate(server, prompts, count, temperature=0.8, top_k=50, top_p=0.95, min_p=0.0, seed=0):
    """Token ids [R, count] that follow the prompts (lists of ids, none empty: a first token follows its prompt's last)."""
    R = len(prompts)
    if R != server.R or not all(prompts):
        raise ValueError(f"{server.R} prompts of one token or more are wanted, got lengths {[len(p) for p in prompts]}")
    per = lambda v, t: torch.full((R,), v, dtype=t, device="cuda")  # noqa: E731
    knobs = dict(temperature=per(temperature, torch.float32), top_k=per(top_k, torch.int32),
                 top_p=per(top_p, torch.float32), min_p=per(min_p, torch.float32))
    gen = torch.Generator("cuda").manual_seed(seed)
    ids, logp, made = per(0, torch.int32), per(0.0, torch.float32), []
    server.reset()
    tokens, new = torch.tensor(sum(prompts, []), device="cuda"), [len(p) for p in prompts]
    for _ in range(count):
        logits = server.step(tokens, new)
        moe.moe_sample(logits, torch.rand(R, generator=gen, device="cuda"), ids, logp, **knobs)
        made.append(ids.clone())
        tokens, new = ids.long(), [1] * R
    if server.attn.status() or server.pool.status():
        raise RuntimeError(f"device status {server.attn.status()} (attention), {server.pool.status()} (experts)")
    return torch.stack(made, 1)


def main():
    ap = argparse.ArgumentParser()
    ap.add_argument("--requests", type=int, default=4)
    ap.add_argument("--tokens", type=int, default=24)
    ap.add_argument("--temperature", type=float, default=0.8)
    a = ap.parse_args()
    rng = np.random.default_rng(1)
    prompts = [rng.integers(0, VOCAB, int(n)).tolist() for n in rng.integers(1, 70, a.requests)]
    server = Server(a.requests, max_len=128 + a.tokens)
    for prompt, ids in zip(prompts, generate(server, prompts, a.tokens, a.temperature).tolist()):
        print(f"prompt of {len(prompt):3d} tokens -> {ids}")
    print("experts:", {k: v for k, v in server.pool.stats().items() if k in ("steps", "hits", "misses", "evictions")})
    server.close()


if __name__ == "__main__":
    main()
