"""Text generation with slot-pool MoE layers: prefill and decode steps of a small random transformer.

Each step runs the library's serving operators in the order a server does:

    tables   once a step: pages for the new tokens, row starts, positions, cache slots
    norm     before and after each block: the block's output into the residual stream, the next block's norm
    linear   per layer, with --q4: the projections with 4-bit weights; once a step the logits
    qkv      per layer: norm + rotation of queries and keys, K and V into the paged cache
    forward  per layer: attention of the new tokens over the cache
    (pool)   per layer: the routed experts from the slot pool
    sample   once a step: the next token of every request
    logprobs once a step, with --top: the tokens' log probabilities and the best alternatives

The embedding and, without --q4, the projections are torch calls.  Run it with

    python examples/generate.py [--requests 4] [--tokens 24] [--temperature 0.8] [--q4] [--top 3]
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


GROUP = 64                                     # inputs that share a scale, with --q4


class Projection:
    """y = x W, W [in, out] in fp32 or, packed, 4-bit codes with group scales."""

    def __init__(self, w, q4):
        self.w, self.q4 = w, q4
        if q4:
            codes, scales = moe.moe_q4_pack(w.t().cpu().numpy(), GROUP)
            self.codes, self.scales = torch.from_numpy(codes).cuda(), torch.from_numpy(scales).cuda()

    def __call__(self, x):
        if not self.q4:
            return x @ self.w
        out = torch.empty(x.shape[0], self.w.shape[1], device="cuda")
        moe.moe_linear_q4(x, self.codes, self.scales, out, group=GROUP)
        return out


class Server:
    """The weights, the expert pool, the paged cache and the requests' state of a small fp32 model."""

    def __init__(self, requests, max_len, max_rows=1024, seed=0, q4=False):
        self.R, self.max_len = requests, max_len
        gen = torch.Generator("cuda").manual_seed(seed)

        def weight(*shape, scale):
            return torch.randn(*shape, generator=gen, device="cuda") * scale
        width = (Q_HEADS + 2 * KV_HEADS) * HEAD_DIM
        self.embed = weight(VOCAB, HIDDEN, scale=1.0)
        self.unembed = Projection(weight(HIDDEN, VOCAB, scale=0.2), q4)
        self.wqkv = [Projection(weight(HIDDEN, width, scale=HIDDEN ** -0.5), q4) for _ in range(LAYERS)]
        self.wo = [Projection(weight(Q_HEADS * HEAD_DIM, HIDDEN, scale=(Q_HEADS * HEAD_DIM) ** -0.5), q4) for _ in range(LAYERS)]
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
        out, ffn, h = torch.empty_like(q), torch.empty_like(x), torch.empty_like(x)
        moe.moe_residual_norm(None, x, None, h)
        for l in range(LAYERS):
            self.attn.qkv(self.wqkv[l](h), self.q_norm[l], self.k_norm[l], self.rope, positions, slots, q,
                          self.k_cache[l], self.v_cache[l])
            self.attn.forward(q, self.row_start, self.seq, max(new), self.k_cache[l], self.v_cache[l], self.table, out)
            moe.moe_residual_norm(self.wo[l](out.flatten(1)), x, x, h)           # x += attention, h its norm
            self.pool.forward(l, h, ffn)
            moe.moe_residual_norm(ffn, x, x, h)                                  # x += experts
        self.ctx.copy_(self.seq)
        return self.unembed(h[self.row_start[1:].long() - 1])

    def close(self):
        self.attn.close()
        self.pool.close()
        self.host.free()


def check(server):
    """Raise where a kernel of the steps so far gave up: its output, and the tokens made of it, are undefined."""
    status = {"attention": server.attn.status(), "experts": server.pool.status()}
    if server.unembed.q4:
        status["projections"] = moe.moe_step_status()          # of the device, and reset by this
    if any(status.values()):
        raise RuntimeError("device status " + ", ".join(f"{v} ({n})" for n, v in status.items()))


def generate(server, prompts, count, temperature=0.8, top_k=50, top_p=0.95, min_p=0.0, seed=0, scores=None, top=0):
    """Token ids [R, count] that follow the prompts (lists of ids, none empty: a first token follows its prompt's last).

    scores: a list that gets, for each step, the model's own view of the tokens before temperature and filters: a dict
    of logp, entropy, rank [R] and top_ids, top_logp [R, top]."""
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
        if scores is not None:
            row = {n: per(0, torch.int32 if n == "rank" else torch.float32) for n in ("logp", "entropy", "rank")}
            row.update(top_ids=torch.empty(R, top, dtype=torch.int32, device="cuda"), top_logp=torch.empty(R, top, device="cuda"))
            moe.moe_logprobs(logits, ids, **row)
            scores.append(row)
        tokens, new = ids.long(), [1] * R
    check(server)
    return torch.stack(made, 1)


def main():
    ap = argparse.ArgumentParser()
    ap.add_argument("--requests", type=int, default=4)
    ap.add_argument("--tokens", type=int, default=24)
    ap.add_argument("--temperature", type=float, default=0.8)
    ap.add_argument("--q4", action="store_true", help="projections with 4-bit weights")
    ap.add_argument("--top", type=int, default=0, help="print the first tokens' log probabilities and this many alternatives")
    a = ap.parse_args()
    rng = np.random.default_rng(1)
    prompts = [rng.integers(0, VOCAB, int(n)).tolist() for n in rng.integers(1, 70, a.requests)]
    server = Server(a.requests, max_len=128 + a.tokens, q4=a.q4)
    scores = [] if a.top > 0 else None
    for r, (prompt, ids) in enumerate(zip(prompts, generate(server, prompts, a.tokens, a.temperature, scores=scores, top=a.top).tolist())):
        print(f"prompt of {len(prompt):3d} tokens -> {ids}")
        if scores:
            s = scores[0]
            print(f"    first: logp {float(s['logp'][r]):.3f}, rank {int(s['rank'][r])}, entropy {float(s['entropy'][r]):.3f}, best",
                  ", ".join(f"{int(i)} ({float(p):.3f})" for i, p in zip(s["top_ids"][r], s["top_logp"][r])))
    print("experts:", {k: v for k, v in server.pool.stats().items() if k in ("steps", "hits", "misses", "evictions")})
    server.close()


if __name__ == "__main__":
    main()
