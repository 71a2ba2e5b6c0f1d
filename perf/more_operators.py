"""Measured cases of the operators between the attention and the experts of a serving step.

Three operators: the join of a block's output into the residual stream with the
norms on either side of it, the projections with 4-bit weights, and the scores of
given tokens (log probability, entropy, rank and the best alternatives).  Each
case runs either in plain torch operations in 32 bits or (``own``) through the
package's public entry points, on the same inputs.
"""
import math
import random

import torch

own = False

F32, BF16 = torch.float32, torch.bfloat16
TYPES = {"f32": F32, "bf16": BF16}
SIZE = {"f32": 4, "bf16": 2}
MAX_ELEMENTS = 8192 * 4096                              # of a norm
MAX_FLOPS, MAX_WEIGHTS = 2 * 2048 * 4096 * 6144, 2048 * 131072      # of a projection
MAX_LOGITS = 2048 * 131072


# ------------------------------------------------------------------------------------------ cases
def _norm(rows, hidden, dtype="bf16", stream=None, post=False, gate="none", sigmoid=False, scale=1.0, offset=0.0, block=True,
          pad=0):
    """`stream`: type of the residual; `block` False: the step's first norm, which has no block before it."""
    return {"op": "norm", "rows": rows, "hidden": hidden, "dtype": dtype, "stream": stream or dtype, "post": post, "gate": gate,
            "sigmoid": sigmoid, "scale": scale, "offset": offset, "block": block, "pad": pad}


def _linear(rows, k, n, group=128, dtype="bf16", out=None, scales="f32", bias=False, pad=0):
    return {"op": "linear", "rows": rows, "k": k, "n": n, "group": group, "dtype": dtype, "out": out or dtype,
            "scales": scales, "bias": bias, "pad": pad}


def _score(rows, vocab, dtype="bf16", top=5, pad=0, masked=False, skipped=False):
    """`masked`: a grammar bars some tokens with -inf; `skipped`: some rows ask for no token."""
    return {"op": "score", "rows": rows, "vocab": vocab, "dtype": dtype, "top": top, "pad": pad, "masked": masked,
            "skipped": skipped}


def listed():
    return [
        # one decoded token between attention and experts: latency
        {"name": "norm_one", **_norm(1, 2048)},
        # a decode batch of a model with norms on both sides of a block and a gate per token
        {"name": "norm_decode_48", **_norm(48, 7168, post=True, gate="row", sigmoid=True, scale=0.22, offset=1.0)},
        # an odd fp32 width, rows of a wider buffer, one gate per channel
        {"name": "norm_f32_777", **_norm(777, 1537, "f32", gate="channel", pad=3)},
        # long prompts, the residual stream held in 32 bits
        {"name": "norm_prefill_8192", **_norm(8192, 4096, stream="f32", post=True)},
        # query, key and value projection of one decoded token
        {"name": "linear_one", **_linear(1, 2048, 5120)},
        # the logits of a decode batch of 16
        {"name": "linear_head_16", **_linear(16, 2048, 131072, out="f32", scales="bf16")},
        # odd sizes in fp32, short groups, a bias
        {"name": "linear_f32_5", **_linear(5, 1120, 3001, 32, "f32", bias=True, pad=8)},
        # a projection of a whole prompt
        {"name": "linear_prompt_2048", **_linear(2048, 4096, 6144)},
        # the score of one sampled token with its alternatives
        {"name": "score_one", **_score(1, 131072, top=20)},
        # the tokens of a batch, fp32 logits of an odd vocabulary in padded rows, some tokens barred
        {"name": "score_batch_48", **_score(48, 100277, "f32", pad=11, masked=True)},
        # a prompt of odd length over an odd vocabulary, no alternatives asked for
        {"name": "score_odd_333", **_score(333, 50257, top=0, skipped=True)},
        # every token of a prompt scored
        {"name": "score_prompt_2048", **_score(2048, 131072)},
    ]


def _log(rng, lo, hi):
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["norm", "norm", "linear", "linear", "linear", "score", "score"])
    dtype = rng.choice(["bf16", "bf16", "f32"])
    if op == "norm":
        hidden = rng.choice([_log(rng, 64, 16384), 8 * _log(rng, 8, 2048)])
        gate = rng.choice(["none", "none", "row", "channel", "element"])
        return _norm(_log(rng, 1, min(8192, MAX_ELEMENTS // 2 // hidden)), hidden, dtype, rng.choice([dtype, "f32"]),
                     rng.random() < 0.5, gate, gate != "none" and rng.random() < 0.5, rng.choice([1.0, 0.22]),
                     rng.choice([0.0, 1.0]), rng.random() < 0.85, rng.choice([0, 0, 8, 3]))
    if op == "linear":
        group = rng.choice([32, 64, 128, 128])
        k = 32 * _log(rng, 4, 384)
        n = _log(rng, 64, min(131072, MAX_WEIGHTS // 2 // k))
        top = MAX_FLOPS // 2 // (2 * k * n)
        rows = rng.choice([_log(rng, 1, 64), _log(rng, 1, 64), _log(rng, 33, 2048 if dtype == "bf16" else 300)])
        return _linear(max(1, min(rows, top)), k, n, group, dtype, rng.choice([dtype, dtype, "f32"]), rng.choice(["f32", "bf16"]),
                       rng.random() < 0.3, rng.choice([0, 0, 8]))
    vocab = _log(rng, 1000, 131072)
    return _score(_log(rng, 1, min(2048, MAX_LOGITS // 2 // vocab)), vocab, dtype, rng.choice([0, 1, 5, 20, 32]),
                  rng.choice([0, 0, 1, 24]), rng.random() < 0.3, rng.random() < 0.3)


# ----------------------------------------------------------------------------------------- inputs
def _device():
    return "cuda"


def _normal(gen, shape, dtype, scale=1.0):
    return torch.randn(shape, generator=gen, device=_device(), dtype=F32).mul_(scale).to(dtype)


def _empty(shape, dtype):
    return torch.empty(shape, dtype=dtype, device=_device())


def prepare(case, seed):
    gen = torch.Generator(device=_device())
    gen.manual_seed(seed)
    return {"norm": _norm_state, "linear": _linear_state, "score": _score_state}[case["op"]](case, gen)


def _norm_state(case, gen):
    rows, hidden, pad = case["rows"], case["hidden"], case["pad"]
    dtype, stream = TYPES[case["dtype"]], TYPES[case["stream"]]
    wide = lambda t, scale: _normal(gen, (rows, hidden + pad), t, scale)[:, :hidden]  # noqa: E731
    # norm weights lie near 1: stored less the offset that the operator adds
    weight = lambda: ((1 - case["offset"]) + _normal(gen, (hidden,), F32, 0.1)).to(dtype)  # noqa: E731
    gate = {"none": None, "row": (rows, 1), "channel": (hidden,), "element": (rows, hidden)}[case["gate"]]
    return {"op": "norm", "eps": 1e-6, "scale": case["scale"], "offset": case["offset"], "sigmoid": case["sigmoid"],
            "x": wide(dtype, 1.5) if case["block"] else None, "residual": wide(stream, 6.0),
            "post": weight() if case["post"] and case["block"] else None, "pre": weight(),
            "gate": _normal(gen, gate, dtype) if gate and case["block"] else None,
            "sum": _empty((rows, hidden), stream) if case["block"] else None, "y": _empty((rows, hidden), dtype)}


def _linear_state(case, gen):
    rows, k, n, group = case["rows"], case["k"], case["n"], case["group"]
    groups = -(-k // group)
    # activations after a norm: near unit, a few channels far above the others
    x = _normal(gen, (rows, k + case["pad"]), F32)
    x[:, ::61] *= 8
    codes = _empty((n, k // 2), torch.uint8)
    scales = _empty((n, groups), TYPES[case["scales"]])
    for at in range(0, n, 8192):                                    # weights of deviation 0.02, quantised group by group
        w = torch.zeros(min(8192, n - at), groups * group, device=_device())
        w[:, :k] = _normal(gen, (w.shape[0], k), F32, 0.02)
        w = w.view(w.shape[0], groups, group)
        s = (w.abs().amax(2) / 7).clamp_(min=1e-8).to(scales.dtype)
        c = torch.round(w / s.float()[..., None]).clamp_(-7, 7).to(torch.int32).view(w.shape[0], -1)[:, :k] & 15
        codes[at:at + 8192] = (c[:, 0::2] | (c[:, 1::2] << 4)).to(torch.uint8)
        scales[at:at + 8192] = s
    dtype = TYPES[case["dtype"]]
    return {"op": "linear", "x": x.to(dtype)[:, :k], "codes": codes, "scales": scales, "group": group,
            "bias": _normal(gen, (n,), dtype, 0.1) if case["bias"] else None, "out": _empty((rows, n), TYPES[case["out"]])}


def _score_state(case, gen):
    rows, vocab, top = case["rows"], case["vocab"], case["top"]
    wide = _normal(gen, (rows, vocab + case["pad"]), F32)
    heat = torch.rand(rows, 1, generator=gen, device=_device())
    x = wide.mul_(1.5 + 2.5 * heat).to(TYPES[case["dtype"]])[:, :vocab]         # flat rows and peaked ones
    if case["masked"]:
        bar = torch.rand(vocab, generator=gen, device=_device()) < 0.3
        x[::2, bar] = -math.inf
    # half of the tokens near the top, as sampled ones are, half anywhere
    near = x.float().argmax(1)
    far = torch.randint(0, vocab, (rows,), generator=gen, device=_device())
    pick = torch.rand(rows, generator=gen, device=_device())
    target = torch.where(pick < 0.5, near, far)
    if case["skipped"]:
        target = torch.where(pick > 0.8, -1, target)
    return {"op": "score", "logits": x, "target": target.int(), "top": top, "logp": _empty(rows, F32), "entropy": _empty(rows, F32),
            "rank": _empty(rows, torch.int32), "top_ids": _empty((rows, top), torch.int32), "top_logp": _empty((rows, top), F32)}


# ------------------------------------------------------------------------------------ plain forms
def _plain_norm(s):
    def normed(v, weight):
        return v * torch.rsqrt(v.square().mean(-1, keepdim=True) + s["eps"]) * (s["offset"] + weight.float())

    r = s["residual"].float()
    out = {}
    if s["x"] is not None:
        n = s["x"].float()
        if s["post"] is not None:
            n = normed(n, s["post"])
        if s["gate"] is not None:
            g = s["gate"].float()
            n = n * (1 / (1 + torch.exp(-g)) if s["sigmoid"] else g)
        r = r + s["scale"] * n
        out["sum"] = r.to(s["residual"].dtype)
    out["y"] = normed(r, s["pre"]).to(s["y"].dtype)
    return out


def _plain_linear(s):
    k = s["x"].shape[1]
    low = (s["codes"] & 15).to(torch.int8)
    high = (s["codes"] >> 4).to(torch.int8)
    c = torch.stack([low, high], -1).flatten(1)
    w = torch.where(c > 7, c - 16, c).float()
    w *= s["scales"].float().repeat_interleave(s["group"], 1)[:, :k]
    out = s["x"].float() @ w.t()
    if s["bias"] is not None:
        out = out + s["bias"].float()
    return {"out": out.to(s["out"].dtype)}


def _plain_score(s):
    x = s["logits"].float()
    rows, vocab = x.shape
    best = x.amax(1, keepdim=True)
    e = torch.exp(x - best)
    total = e.sum(1, keepdim=True)
    lse = best + torch.log(total)
    entropy = torch.log(total[:, 0]) - torch.where(e > 0, e * (x - best), 0).sum(1) / total[:, 0]
    wanted = s["target"] >= 0
    t = s["target"].clamp(min=0).long()[:, None]
    xt = x.gather(1, t)
    index = torch.arange(vocab, device=x.device)
    rank = ((x > xt) | ((x == xt) & (index < t))).sum(1)
    # unique keys: ordered logits above, the lower index first among equal ones
    bits = (x + 0.0).view(torch.int32)
    order = torch.where(bits < 0, bits ^ 0x7fffffff, bits).long()
    keys = torch.topk(order * (1 << 32) + (vocab - index), s["top"], dim=1).values
    ids = vocab - (keys & 0xffffffff)
    return {"logp": torch.where(wanted, (xt - lse)[:, 0], 0.0), "entropy": entropy, "rank": torch.where(wanted, rank, -1).int(),
            "top_ids": ids.int(), "top_logp": x.gather(1, ids) - lse}


# ---------------------------------------------------------------------------- the package's calls
def _own_norm(s):
    import expert_offload_slot_gb300 as moe
    moe.moe_residual_norm(s["x"], s["residual"], s["sum"], s["y"], post_weight=s["post"], pre_weight=s["pre"], gate=s["gate"],
                          gate_sigmoid=s["sigmoid"], residual_scale=s["scale"], eps=s["eps"], weight_offset=s["offset"])
    return {"y": s["y"]} if s["sum"] is None else {"sum": s["sum"], "y": s["y"]}


def _own_linear(s):
    import expert_offload_slot_gb300 as moe
    moe.moe_linear_q4(s["x"], s["codes"], s["scales"], s["out"], group=s["group"], bias=s["bias"])
    return {"out": s["out"]}


def _own_score(s):
    import expert_offload_slot_gb300 as moe
    moe.moe_logprobs(s["logits"], s["target"], s["logp"], entropy=s["entropy"], rank=s["rank"], top_ids=s["top_ids"],
                     top_logp=s["top_logp"])
    return {n: s[n] for n in ("logp", "entropy", "rank", "top_ids", "top_logp")}


PLAIN = {"norm": _plain_norm, "linear": _plain_linear, "score": _plain_score}
OWN = {"norm": _own_norm, "linear": _own_linear, "score": _own_score}


def run(state):
    return (OWN if own else PLAIN)[state["op"]](state)


# ------------------------------------------------------------------------------------- the floors
def work(case):
    size = SIZE[case["dtype"]]
    if case["op"] == "norm":
        n = case["rows"] * case["hidden"]
        gates = {"none": 0, "row": case["rows"], "channel": case["hidden"], "element": n}[case["gate"]]
        block = n * (size + SIZE[case["stream"]]) + (gates + case["post"] * case["hidden"]) * size if case["block"] else 0
        return {"bytes": block + n * (SIZE[case["stream"]] + size) + case["hidden"] * size, "flops": 10 * n}
    if case["op"] == "linear":
        rows, k, n = case["rows"], case["k"], case["n"]
        return {"bytes": n * (k // 2 + -(-k // case["group"]) * SIZE[case["scales"]] + case["bias"] * size) + rows * k * size +
                rows * n * SIZE[case["out"]], "flops": 2 * rows * k * n}
    return {"bytes": case["rows"] * (case["vocab"] * size + 16 + 8 * case["top"]), "flops": 5 * case["rows"] * case["vocab"]}


# ------------------------------------------------------------------- the definitions in 64 bits
def exact(case, seed):
    return {"norm": _exact_norm, "linear": _exact_linear, "score": _exact_score}[case["op"]](prepare(case, seed))


def _exact_norm(s):
    def length(v):
        return torch.sqrt((v * v).sum(1) / v.shape[1] + s["eps"])[:, None]

    total, out = s["residual"].double(), {}
    if s["x"] is not None:
        branch = s["x"].double()
        if s["post"] is not None:
            branch = branch / length(branch) * (s["post"].double() + s["offset"])
        if s["gate"] is not None:
            branch = branch * (torch.sigmoid(s["gate"].double()) if s["sigmoid"] else s["gate"].double())
        total = out["sum"] = total + branch * s["scale"]
    out["y"] = total / length(total) * (s["pre"].double() + s["offset"])
    return out


def _exact_linear(s):
    x, group = s["x"].double(), s["group"]
    rows, k = x.shape
    parts = []
    for codes, scales in zip(s["codes"].split(16384), s["scales"].double().split(16384)):
        values = torch.empty(codes.shape[0], k, dtype=torch.float64, device=x.device)
        for odd in (0, 1):
            nibble = (codes.int() >> 4 * odd) & 15
            values[:, odd::2] = ((nibble + 8) % 16 - 8).double()
        for g in range(scales.shape[1]):
            values[:, g * group:(g + 1) * group] *= scales[:, g:g + 1]
        parts.append(x @ values.T)
    out = torch.cat(parts, 1)
    return {"out": out if s["bias"] is None else out + s["bias"].double()}


def _exact_score(s):
    made = {n: [] for n in ("logp", "entropy", "rank", "top_ids", "top_logp")}
    for x, target in zip(s["logits"].split(64), s["target"].split(64)):
        x = x.double()
        logs = torch.log_softmax(x, 1)
        p = torch.exp(logs)
        made["entropy"].append(-torch.where(p > 0, p * logs, 0).sum(1))
        order = torch.sort(x, dim=1, descending=True, stable=True).indices
        at = (order == target[:, None]).int().argmax(1)
        asked = target >= 0
        made["rank"].append(torch.where(asked, at, -1).int())
        made["logp"].append(torch.where(asked, logs.gather(1, target.clamp(min=0).long()[:, None])[:, 0], 0.0))
        made["top_ids"].append(order[:, :s["top"]].int())
        made["top_logp"].append(logs.gather(1, order[:, :s["top"]]))
    return {n: torch.cat(v) for n, v in made.items()}
