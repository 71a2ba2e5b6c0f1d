"""Measured cases of the operators around the MoE layer in a serving step.

Four operators, in the order a step runs them: the page tables of the step, the
query/key norm + rotation + cache write, the attention of the new tokens over
the paged cache, and the choice of the next tokens.  Each case runs either in
plain torch operations in 32 bits or (``own``) through the package's public
entry points, on the same inputs.
"""
import functools
import math
import random

import torch

own = False

F32, BF16 = torch.float32, torch.bfloat16
TYPES = {"f32": F32, "bf16": BF16}


# ------------------------------------------------------------------------------------------ cases
def _heads(q_heads, kv_heads, head_dim, page, dtype="bf16", window=0, rotary=None, pairs=False, norm=True):
    return {"q_heads": q_heads, "kv_heads": kv_heads, "head_dim": head_dim, "page": page, "dtype": dtype,
            "window": window, "rotary": head_dim if rotary is None else rotary, "pairs": pairs, "norm": norm}


def _lens(lens, decodes, chunks, ctx_lo, ctx_hi, new_lo=1, new_hi=1):
    """`decodes` requests with one new token and `chunks` with new_lo..new_hi, over ctx_lo..ctx_hi cached ones."""
    return {"lens": lens, "decodes": decodes, "chunks": chunks, "ctx_lo": ctx_lo, "ctx_hi": ctx_hi,
            "new_lo": new_lo, "new_hi": new_hi}


def listed():
    return [
        # the tables of a decode step of 16 requests: a handful of integers, latency only
        {"name": "tables_decode_16", "op": "tables", "page": 16, **_lens(1, 16, 0, 1, 8191)},
        # the tables of a mixed step: 360 decodes and 24 prompt chunks, ~25k rows
        {"name": "tables_mixed_384", "op": "tables", "page": 16, **_lens(2, 360, 24, 1, 8191, 65, 2048)},
        # one decoded token of one request: the latency of norm + rotation + cache write
        {"name": "qkv_one", "op": "qkv", **_heads(32, 4, 128, 16), **_lens(3, 1, 0, 700, 2000)},
        # a 2048-token prefill, half-split rotation over the whole head
        {"name": "qkv_prefill_2048", "op": "qkv", **_heads(32, 8, 128, 64), **_lens(4, 0, 1, 0, 0, 2048, 2048)},
        # an odd number of fp32 rows, partial rotation of neighbouring pairs, 64-wide heads
        {"name": "qkv_f32_1333", "op": "qkv", **_heads(12, 3, 64, 16, "f32", rotary=32, pairs=True),
         **_lens(5, 36, 1, 0, 900, 1297, 1297)},
        # one decoded token over a short context: latency
        {"name": "attend_one", "op": "attend", **_heads(32, 4, 128, 16), **_lens(6, 1, 0, 900, 1100)},
        # the decode step of a batch of 16 with ragged contexts
        {"name": "attend_decode_16", "op": "attend", **_heads(32, 4, 128, 16), **_lens(7, 16, 0, 60, 8191)},
        # four long contexts decoded together: the stream of the cache
        {"name": "attend_decode_long", "op": "attend", **_heads(32, 8, 128, 64), **_lens(8, 4, 0, 90000, 110000)},
        # prompts of ragged lengths from an empty cache
        {"name": "attend_prefill", "op": "attend", **_heads(32, 4, 128, 16), **_lens(9, 0, 3, 0, 0, 700, 2048)},
        # a chunk of a long prompt over what is cached of it
        {"name": "attend_chunk_long", "op": "attend", **_heads(32, 8, 128, 64), **_lens(10, 0, 1, 30000, 32000, 1024, 1024)},
        # the next token of one request
        {"name": "sample_one", "op": "sample", "rows": 1, "vocab": 131072, "dtype": "bf16", "pad": 0, "filters": "all"},
        # the next tokens of a batch, fp32 logits of an odd vocabulary in padded rows
        {"name": "sample_batch_48", "op": "sample", "rows": 48, "vocab": 100277, "dtype": "f32", "pad": 11, "filters": "mixed"},
    ]


def _log(rng, lo, hi):
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["tables", "qkv", "qkv", "attend", "attend", "attend", "attend", "sample", "sample"])
    seed = rng.randrange(1 << 30)
    if op == "tables":
        chunks = rng.choice([0, 0, rng.randint(1, 20)])
        return {"op": op, "page": rng.choice([16, 32, 64, 128]),
                **_lens(seed, _log(rng, 1, 400), chunks, rng.randint(0, 100), _log(rng, 200, 8191), 2, 2048)}
    if op == "sample":
        return {"op": op, "rows": _log(rng, 1, 48), "vocab": _log(rng, 1000, 131072), "dtype": rng.choice(["bf16", "f32"]),
                "pad": rng.choice([0, 0, 1, 24]), "filters": rng.choice(["all", "mixed", "greedy", "none"])}
    kv = rng.choice([1, 2, 4, 8])
    dtype = rng.choice(["bf16", "bf16", "bf16", "f32"])
    dim = rng.choice([64, 128, 128])
    heads = _heads(kv * rng.choice([1, 3, 4, 8]), kv, dim, rng.choice([16, 32, 64, 128]), dtype,
                   window=rng.choice([0, 0, 0, _log(rng, 16, 4096)]), rotary=rng.choice([dim, dim // 2]),
                   pairs=rng.random() < 0.3, norm=rng.random() < 0.8)
    if op == "qkv":
        heads["window"] = 0
        return {"op": op, **heads, **_lens(seed, rng.randint(0, 60), rng.randint(0, 2) + (rng.random() < 0.5), 0,
                                           _log(rng, 100, 2000), 2, 800)} if rng.random() < 0.7 else \
               {"op": op, **heads, **_lens(seed, _log(rng, 1, 64), 0, 0, 2000)}
    kind = rng.choice(["decode", "decode", "prefill", "chunk", "mixed"])
    small = dtype == "f32"
    if kind == "decode":
        requests = _log(rng, 1, 64)
        lens = _lens(seed, requests, 0, 0, _log(rng, 100, min(100000, (80000 if small else 400000) // requests)))
    elif kind == "prefill":
        lens = _lens(seed, 0, rng.randint(1, 3), 0, 0, 2, _log(rng, 40, 500 if small else 2000))
    elif kind == "chunk":
        lens = _lens(seed, 0, rng.randint(1, 2), 0, _log(rng, 100, 2000 if small else 7000), 2,
                     _log(rng, 8, 200 if small else 1000))
    else:
        lens = _lens(seed, rng.randint(1, 10), 1, 0, _log(rng, 100, 1000 if small else 3000), 2,
                     _log(rng, 8, 200 if small else 600))
    return {"op": op, **heads, **lens}


def _lengths(case):
    """Cached and new tokens of every request: part of the case, the same for every seed."""
    rng = random.Random(case["lens"])
    n = case["decodes"] + case["chunks"]
    ctx = [rng.randint(case["ctx_lo"], case["ctx_hi"]) for _ in range(n)]
    new = [1] * case["decodes"] + [rng.randint(case["new_lo"], case["new_hi"]) for _ in range(case["chunks"])]
    if not n:
        ctx, new = [case["ctx_hi"]], [1]
    order = list(range(len(ctx)))
    rng.shuffle(order)
    return [ctx[i] for i in order], [new[i] for i in order]


# ----------------------------------------------------------------------------------------- inputs
def _device():
    return "cuda"


def _ints(values):
    return torch.tensor(values, dtype=torch.int32, device=_device())


def _requests(case, seed):
    """Lengths, pages and rows of a step, as a serving program holds them on the GPU."""
    ctx, new = _lengths(case)
    page = case["page"]
    have = [-(-c // page) for c in ctx]
    need = [-(-(c + n) // page) for c, n in zip(ctx, new)]
    pages = sum(need) + 5
    order = list(range(pages))
    random.Random(seed).shuffle(order)                  # pages in no order, as after hours of serving
    width = max(need) + 1
    tables, at = [], 0
    for h in have:
        tables.append(order[at:at + h] + [-1] * (width - h))
        at += h
    rows = sum(new)
    return {"ctx_host": ctx, "new_host": new, "ctx": _ints(ctx), "new": _ints(new), "table": _ints(tables),
            "free": _ints(order[at:]), "free_head": _ints([0]), "pages": pages, "rows": rows, "width": width,
            "requests": len(ctx), "max_new": max(new), "page": page}


def _grown(s):
    """The same step after its tables were built: full tables, row starts, positions, slots."""
    t = _plain_tables(s)
    return {**s, "table": t["table"], "row_start": t["row_start"], "seq_len": t["seq_len"],
            "positions": t["positions"], "slots": t["slots"]}


def _normal(gen, shape, dtype, scale=1.0):
    return torch.randn(shape, generator=gen, device=_device(), dtype=F32).mul_(scale).to(dtype)


def prepare(case, seed):
    gen = torch.Generator(device=_device())
    gen.manual_seed(seed)
    op = case["op"]
    if op == "sample":
        return _sample_state(case, seed, gen)
    s = _requests(case, seed)
    s["op"] = op
    if op == "tables":
        s["rows"] = -(-s["rows"] // 8) * 8              # rows of a captured step are padded
        for name, n in (("row_start", s["requests"] + 1), ("seq_len", s["requests"]), ("positions", s["rows"]),
                        ("slots", s["rows"]), ("head_out", 1)):
            s[name] = torch.empty(n, dtype=torch.int32, device=_device())
        return s
    s = _grown(s)
    dtype, dim, hq, hkv = TYPES[case["dtype"]], case["head_dim"], case["q_heads"], case["kv_heads"]
    s.update(dtype=dtype, dim=dim, q_heads=hq, kv_heads=hkv, window=case["window"], rotary=case["rotary"],
             pairs=case["pairs"], eps=1e-6, scale=dim ** -0.5)
    cache = (s["pages"], hkv, case["page"], dim)
    if op == "qkv":
        s["qkv"] = _normal(gen, (s["rows"], (hq + 2 * hkv) * dim), dtype)
        s["q_norm"] = 1 + _normal(gen, (dim,), F32, 0.1) if case["norm"] else None
        s["k_norm"] = 1 + _normal(gen, (dim,), F32, 0.1) if case["norm"] else None
        if case["norm"]:
            s["q_norm"], s["k_norm"] = s["q_norm"].to(dtype), s["k_norm"].to(dtype)
        length = max(c + n for c, n in zip(s["ctx_host"], s["new_host"]))
        half = case["rotary"] // 2
        freq = 10000.0 ** (-torch.arange(half, device=_device(), dtype=torch.float64) / half)
        angle = torch.arange(length, device=_device(), dtype=torch.float64)[:, None] * freq
        s["rope"] = torch.cat([angle.cos(), angle.sin()], 1).to(F32)
        s["k_cache"] = torch.zeros(cache, dtype=dtype, device=_device())
        s["v_cache"] = torch.zeros(cache, dtype=dtype, device=_device())
        s["q"] = torch.empty((s["rows"], hq, dim), dtype=dtype, device=_device())
    else:
        # normalised, rotated keys have unit mean square; query norm weights near 2 peak the softmax
        s["q"] = _normal(gen, (s["rows"], hq, dim), dtype, 2.0)
        s["k_cache"] = _normal(gen, cache, dtype)
        s["v_cache"] = _normal(gen, cache, dtype)
        s["out"] = torch.empty((s["rows"], hq, dim), dtype=dtype, device=_device())
    return s


def _sample_state(case, seed, gen):
    rng = random.Random(seed)
    rows, vocab, kind = case["rows"], case["vocab"], case["filters"]
    wide = _normal(gen, (rows, vocab + case["pad"]), F32, 3.0)
    logits = wide.to(TYPES[case["dtype"]])[:, :vocab]
    on = {"all": lambda: True, "none": lambda: False, "greedy": lambda: False, "mixed": lambda: rng.random() < 0.6}[kind]
    temp = [0.0 if kind == "greedy" or (kind == "mixed" and rng.random() < 0.1) else rng.uniform(0.5, 1.2) for _ in range(rows)]
    top_k = [rng.choice([20, 40, 50, 100, 1000]) if on() else 0 for _ in range(rows)]
    top_p = [rng.uniform(0.7, 0.99) if on() else 1.0 for _ in range(rows)]
    min_p = [rng.uniform(0.01, 0.1) if on() else 0.0 for _ in range(rows)]
    floats = functools.partial(torch.tensor, dtype=F32, device=_device())
    return {"op": "sample", "logits": logits, "temperature": floats(temp), "top_k": _ints(top_k), "top_p": floats(top_p),
            "min_p": floats(min_p), "u": torch.rand(rows, generator=gen, device=_device(), dtype=F32),
            "ids": torch.empty(rows, dtype=torch.int32, device=_device()),
            "logp": torch.empty(rows, dtype=F32, device=_device())}


# ------------------------------------------------------------------------------------ plain forms
def _plain_tables(s):
    page, width, rows = s["page"], s["width"], s["rows"]
    ctx, new = s["ctx"].long(), s["new"].long()
    seq = ctx + new
    have, need = (ctx + page - 1) // page, (seq + page - 1) // page
    grow = need - have
    off = grow.cumsum(0) - grow + s["free_head"].long()
    col = torch.arange(width, device=ctx.device)[None, :]
    fresh = (col >= have[:, None]) & (col < need[:, None])
    source = (off[:, None] + col - have[:, None]).clamp(0, s["free"].numel() - 1)
    table = torch.where(fresh, s["free"][source], s["table"])
    ends = new.cumsum(0)
    row = torch.arange(rows, device=ctx.device)
    live = row < ends[-1]
    req = torch.searchsorted(ends, row, right=True).clamp(max=s["requests"] - 1)
    pos = torch.where(live, ctx[req] + row - (ends - new)[req], 0)
    slot = table[req, pos // page].long() * page + pos % page
    return {"table": table, "row_start": torch.cat([ends.new_zeros(1), ends]).int(), "seq_len": seq.int(),
            "positions": pos.int(), "slots": torch.where(live, slot, -1).int(),
            "free_head": s["free_head"] + grow.sum().int()}


def _plain_rotate(x, s, cos, sin):
    half = s["rotary"] // 2
    head, rest = x[..., :2 * half], x[..., 2 * half:]
    a, b = (head[..., 0::2], head[..., 1::2]) if s["pairs"] else (head[..., :half], head[..., half:])
    ra, rb = a * cos - b * sin, b * cos + a * sin
    turned = torch.stack([ra, rb], -1).flatten(-2) if s["pairs"] else torch.cat([ra, rb], -1)
    return torch.cat([turned, rest], -1)


def _plain_qkv(s):
    rows, hq, hkv, dim, page = s["rows"], s["q_heads"], s["kv_heads"], s["dim"], s["page"]
    x = s["qkv"].float().view(rows, hq + 2 * hkv, dim)
    q, k, v = x[:, :hq], x[:, hq:hq + hkv], x[:, hq + hkv:]
    if s["q_norm"] is not None:
        q = q * torch.rsqrt(q.square().mean(-1, keepdim=True) + s["eps"]) * s["q_norm"].float()
        k = k * torch.rsqrt(k.square().mean(-1, keepdim=True) + s["eps"]) * s["k_norm"].float()
    half = s["rotary"] // 2
    turn = s["rope"][s["positions"].long()]
    cos, sin = turn[:, None, :half], turn[:, None, half:]
    q, k = _plain_rotate(q, s, cos, sin), _plain_rotate(k, s, cos, sin)
    slot = s["slots"].long()
    s["k_cache"][slot // page, :, slot % page] = k.to(s["dtype"])
    s["v_cache"][slot // page, :, slot % page] = v.to(s["dtype"])
    return {"q": q.to(s["dtype"]), "k_cache": s["k_cache"], "v_cache": s["v_cache"]}


def _gathered(cache, s):
    """[requests, kv_heads, width * page, dim] in 32 bits."""
    got = cache[s["table"].clamp(min=0).long()]                       # [R, W, Hkv, P, D]
    return got.permute(0, 2, 1, 3, 4).reshape(s["requests"], s["kv_heads"], -1, s["dim"]).float()


def _plain_attend(s):
    R, hkv, dim, new_max = s["requests"], s["kv_heads"], s["dim"], s["max_new"]
    group = s["q_heads"] // hkv
    start, new, seq = s["row_start"][:-1].long(), s["new"].long(), s["seq_len"].long()
    i = torch.arange(new_max, device=new.device)
    live = i[None, :] < new[:, None]
    row = (start[:, None] + i).clamp(max=s["rows"] - 1)
    q = s["q"][row].float().view(R, new_max, hkv, group, dim).permute(0, 2, 1, 3, 4).reshape(R, hkv, new_max * group, dim)
    k, v = _gathered(s["k_cache"], s), _gathered(s["v_cache"], s)
    key = torch.arange(k.shape[2], device=new.device)
    pos = (seq - new)[:, None] + i                                    # [R, new_max]
    seen = (key <= pos[..., None]) & live[..., None]
    if s["window"]:
        seen &= key > pos[..., None] - s["window"]
    score = (q @ k.transpose(-1, -2)).mul_(s["scale"]).view(R, hkv, new_max, group, -1)
    score = score.masked_fill_(~seen[:, None, :, None, :], -math.inf)
    top = score.amax(-1, keepdim=True).clamp(min=-3e38)
    p = score.sub_(top).exp_()
    total = p.sum(-1, keepdim=True)
    out = (p.view(R, hkv, new_max * group, -1) @ v).view(R, hkv, new_max, group, dim) / total.clamp(min=1e-30)
    out = out.permute(0, 2, 1, 3, 4).reshape(R, new_max, s["q_heads"], dim)
    flat = (torch.arange(s["rows"], device=new.device))
    req = torch.searchsorted(s["row_start"][1:].long(), flat, right=True)
    return {"out": out[req, flat - start[req]].to(s["dtype"])}


def _plain_sample(s):
    x = s["logits"].float()
    vocab = x.shape[1]
    best = x.amax(1, keepdim=True)
    temp = s["temperature"][:, None]
    greedy = temp == 0
    z = (x - best) / torch.where(greedy, 1.0, temp)
    w = (torch.exp(z) * 2.0 ** 40).to(torch.int64)
    order = torch.sort(x, dim=1, descending=True, stable=True).indices
    ws = w.gather(1, order)
    rank = torch.arange(vocab, device=x.device)
    k = torch.where(s["top_k"] > 0, s["top_k"], vocab)[:, None]
    ws = torch.where(rank < k, ws, 0)
    inc = ws.cumsum(1)
    limit = (s["top_p"][:, None].double() * inc[:, -1:].double()).ceil().to(torch.int64).clamp(min=1)
    keep = (rank < k) & ((inc - ws < limit) | (s["top_p"][:, None] >= 1)) & (ws.double() >= s["min_p"][:, None].double() * 2.0 ** 40)
    kept = torch.zeros_like(w).scatter_(1, order, torch.where(keep, ws, 0))
    run_ = kept.cumsum(1)
    mass = run_[:, -1:]
    goal = (s["u"][:, None].double() * mass.double()).to(torch.int64)
    drawn = (run_ <= goal).sum(1, keepdim=True).clamp(max=vocab - 1)
    ids = torch.where(greedy, order[:, :1], drawn)
    logp = torch.where(greedy, 0.0, torch.log(kept.gather(1, ids).float() / mass.float()))
    return {"ids": ids[:, 0].int(), "logp": logp[:, 0]}


# ---------------------------------------------------------------------------- the package's calls
@functools.lru_cache(maxsize=None)
def _attention(q_heads, kv_heads, dim, page, f32, rotary, pairs, window, scale, eps):
    """The handle (workspaces only) that a program makes once for its layers' shape."""
    import expert_offload_slot_gb300 as moe
    return moe.Attention(moe.make_attn_config(
        q_heads, kv_heads, dim, page, moe.MOE_F32 if f32 else moe.MOE_BF16, rotary_dim=rotary,
        rotary_style=moe.MOE_ROTARY_PAIRS if pairs else moe.MOE_ROTARY_HALF, window=window, softmax_scale=scale, norm_eps=eps))


def _handle(s):
    return _attention(s["q_heads"], s["kv_heads"], s["dim"], s["page"], s["dtype"] is F32, s["rotary"], s["pairs"], s["window"],
                      s["scale"], s["eps"])


def _own_tables(s):
    _attention(32, 4, 128, s["page"], False, 128, False, 0, 128 ** -0.5, 1e-6).tables(
        s["ctx"], s["new"], s["table"], s["free"], s["free_head"], s["head_out"], s["row_start"], s["seq_len"], s["positions"],
        s["slots"])
    return {"table": s["table"], "row_start": s["row_start"], "seq_len": s["seq_len"], "positions": s["positions"],
            "slots": s["slots"], "free_head": s["head_out"]}


def _own_qkv(s):
    _handle(s).qkv(s["qkv"], s["q_norm"], s["k_norm"], s["rope"], s["positions"], s["slots"], s["q"], s["k_cache"], s["v_cache"])
    return {"q": s["q"], "k_cache": s["k_cache"], "v_cache": s["v_cache"]}


def _own_attend(s):
    _handle(s).forward(s["q"], s["row_start"], s["seq_len"], s["max_new"], s["k_cache"], s["v_cache"], s["table"], s["out"])
    return {"out": s["out"]}


def _own_sample(s):
    import expert_offload_slot_gb300 as moe
    moe.moe_sample(s["logits"], s["u"], s["ids"], s["logp"], temperature=s["temperature"], top_k=s["top_k"], top_p=s["top_p"],
                   min_p=s["min_p"])
    return {"ids": s["ids"], "logp": s["logp"]}


PLAIN = {"tables": _plain_tables, "qkv": _plain_qkv, "attend": _plain_attend, "sample": _plain_sample}
OWN = {"tables": _own_tables, "qkv": _own_qkv, "attend": _own_attend, "sample": _own_sample}


def run(state):
    return (OWN if own else PLAIN)[state["op"]](state)


# ------------------------------------------------------------------------------------- the floors
def work(case):
    if case["op"] == "sample":
        size = 2 if case["dtype"] == "bf16" else 4
        return {"bytes": case["rows"] * (case["vocab"] * size + 28), "flops": case["rows"] * case["vocab"] * 4}
    ctx, new = _lengths(case)
    page, rows = case["page"], sum(new)
    pages = sum(-(-(c + n) // page) for c, n in zip(ctx, new))
    if case["op"] == "tables":
        fresh = pages - sum(-(-c // page) for c in ctx)
        return {"bytes": 4 * (4 * len(ctx) + 2 * fresh + 2 * rows), "flops": 0}
    size = 2 if case["dtype"] == "bf16" else 4
    hq, hkv, dim = case["q_heads"], case["kv_heads"], case["head_dim"]
    if case["op"] == "qkv":
        return {"bytes": rows * (2 * (hq + 2 * hkv) * dim * size + 8 + case["rotary"] * 4), "flops": rows * (hq + hkv) * dim * 8}
    window = case["window"] or 1 << 60
    keys = sum(min(c + n, window + n - 1) for c, n in zip(ctx, new))
    pairs = 0
    for c, n in zip(ctx, new):
        ramp = max(0, min(n, window - c))               # rows that still see every key before them
        pairs += ramp * c + ramp * (ramp + 1) // 2 + (n - ramp) * window if window < 1 << 60 else n * c + n * (n + 1) // 2
    return {"bytes": 2 * keys * hkv * dim * size + 2 * rows * hq * dim * size + 4 * pages, "flops": 4 * dim * hq * pairs}


# ------------------------------------------------------------------- the definitions in 64 bits
def exact(case, seed):
    s = prepare(case, seed)
    return {"tables": _exact_tables, "qkv": _exact_qkv, "attend": _exact_attend, "sample": _exact_sample}[case["op"]](s)


def _exact_tables(s):
    page, head = s["page"], int(s["free_head"][0])
    table, free = s["table"].tolist(), s["free"].tolist()
    starts, pos, slot = [0], [], []
    for r, (c, n) in enumerate(zip(s["ctx_host"], s["new_host"])):
        for j in range(-(-c // page), -(-(c + n) // page)):
            table[r][j] = free[head]
            head += 1
        starts.append(starts[-1] + n)
        pos += range(c, c + n)
        slot += [table[r][p // page] * page + p % page for p in range(c, c + n)]
    pad = s["rows"] - len(pos)
    return {"table": _ints(table), "row_start": _ints(starts), "seq_len": _ints([c + n for c, n in zip(s["ctx_host"], s["new_host"])]),
            "positions": _ints(pos + [0] * pad), "slots": _ints(slot + [-1] * pad), "free_head": _ints([head])}


def _exact_qkv(s):
    hq, hkv, dim, half, page = s["q_heads"], s["kv_heads"], s["dim"], s["rotary"] // 2, s["page"]
    heads = s["qkv"].double().reshape(s["rows"], hq + 2 * hkv, dim)
    angles = s["rope"].double()[s["positions"].long()]

    def turned(x, weight):
        if weight is not None:
            x = x / torch.sqrt((x * x).sum(-1, keepdim=True) / dim + s["eps"]) * weight.double()
        y = x.clone()
        for i in range(half):
            a, b = (2 * i, 2 * i + 1) if s["pairs"] else (i, i + half)
            c, d = angles[:, None, i], angles[:, None, half + i]
            y[..., a] = x[..., a] * c - x[..., b] * d
            y[..., b] = x[..., a] * d + x[..., b] * c
        return y

    k = torch.zeros(s["pages"], hkv, page, dim, dtype=torch.float64, device=heads.device)
    v = torch.zeros_like(k)
    for h in range(hkv):
        flat = k[:, h].reshape(-1, dim), v[:, h].reshape(-1, dim)
        flat[0][s["slots"].long()] = turned(heads[:, hq + h:hq + h + 1], s["k_norm"])[:, 0]
        flat[1][s["slots"].long()] = heads[:, hq + hkv + h]
        k[:, h], v[:, h] = flat[0].view(-1, page, dim), flat[1].view(-1, page, dim)
    return {"q": turned(heads[:, :hq], s["q_norm"]), "k_cache": k, "v_cache": v}


def _exact_attend(s):
    out = torch.zeros(s["rows"], s["q_heads"], s["dim"], dtype=torch.float64, device=s["q"].device)
    group, at = s["q_heads"] // s["kv_heads"], 0
    for r, (c, n) in enumerate(zip(s["ctx_host"], s["new_host"])):
        used = s["table"][r, :-(-(c + n) // s["page"])].long()
        for h in range(s["q_heads"]):
            k = s["k_cache"][used, h // group].reshape(-1, s["dim"])[:c + n].double()
            v = s["v_cache"][used, h // group].reshape(-1, s["dim"])[:c + n].double()
            t = s["q"][at:at + n, h].double() @ k.T * s["scale"]
            gap = torch.arange(c, c + n, device=t.device)[:, None] - torch.arange(c + n, device=t.device)[None, :]
            t[(gap < 0) | ((gap >= s["window"]) if s["window"] else (gap < 0))] = -math.inf
            out[at:at + n, h] = torch.softmax(t, -1) @ v
        at += n
    return {"out": out}


def _exact_sample(s):
    ids, logp = [], []
    rows = zip(s["logits"].double(), s["temperature"].tolist(), s["top_k"].tolist(), s["top_p"].tolist(), s["min_p"].tolist(), s["u"].tolist())
    for x, temp, k, p, m, u in rows:
        order = torch.sort(x, descending=True, stable=True).indices
        if temp == 0:
            ids.append(int(order[0]))
            logp.append(0.0)
            continue
        weight = torch.exp((x - x.max()) / temp)
        kept = order[:k] if k > 0 else order
        before = weight[kept].cumsum(0) - weight[kept]
        if p < 1:
            kept = kept[before < p * weight[kept].sum()]
        kept = kept[weight[kept] >= m].sort().values
        mass = weight[kept].cumsum(0)
        at = int(torch.searchsorted(mass, u * mass[-1], right=True).clamp(max=len(kept) - 1))
        ids.append(int(kept[at]))
        logp.append(float(torch.log(weight[kept[at]] / mass[-1])))
    return {"ids": _ints(ids), "logp": torch.tensor(logp, dtype=torch.float64, device=s["u"].device)}
