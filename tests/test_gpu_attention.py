"""Page tables, norm + rotation + cache write, and attention over the paged cache against the 64-bit oracle.

Tolerances.  Attention, bf16: the probabilities and the output are each rounded to bf16 (at most
2^-8 of their size, the probabilities' errors averaging out over the keys) and the fp32 scores are
off by at most D 2^-24 sum|q k| scale (about 2e-4 here): 2^-7 sum p|v| is allowed.  fp32: the
scores' error alone, 2e-4 sum p|v|.  Norm + rotation: the reduction and the products keep 1e-6 of
|a| + |b|; bf16 adds one rounding, 2^-8 |y|.
"""
import numpy as np
import pytest
import torch

import expert_offload_slot_gb300 as moe
from oracle import attention as oracle

pytestmark = pytest.mark.gpu
DT = {"f32": (torch.float32, moe.MOE_F32), "bf16": (torch.bfloat16, moe.MOE_BF16)}


def ints(v):
    return torch.tensor(np.asarray(v), dtype=torch.int32, device="cuda")


class Step:
    """A step's requests with their tables, built by the library."""

    def __init__(self, ctx, new, dtype="bf16", hq=8, hkv=2, dim=128, page=16, window=0, pad=0, spare=3, seed=0, scale=None,
                 **cfg):
        self.ctx, self.new, self.page, self.hq, self.hkv, self.dim, self.window = ctx, new, page, hq, hkv, dim, window
        self.dtype = DT[dtype][0]
        self.scale = dim ** -0.5 if scale is None else scale
        rng = np.random.default_rng(seed)
        have = [-(-c // page) for c in ctx]
        need = [-(-(c + n) // page) for c, n in zip(ctx, new)]
        self.pages, self.width, self.rows = sum(need) + spare, max(need + [1]) + 1, sum(new) + pad
        order = rng.permutation(self.pages)
        table, at = np.full((len(ctx), self.width), 1 << 30), 0           # entries in no use hold no page
        for r, h in enumerate(have):
            table[r, :h] = order[at:at + h]
            at += h
        self.free, self.head0, self.table0 = order[at:], 0, table
        self.handle = moe.Attention(moe.make_attn_config(hq, hkv, dim, page, DT[dtype][1], window=window, softmax_scale=self.scale,
                                                         **cfg))
        self.table, self.free_d = ints(table), ints(self.free)
        self.head = ints([0])
        self.start, self.seq = ints(np.zeros(len(ctx) + 1)), ints(np.zeros(len(ctx)))
        self.pos, self.slot = ints(np.zeros(self.rows)), ints(np.zeros(self.rows))
        self.handle.tables(ints(ctx), ints(new), self.table, self.free_d, self.head, self.head, self.start, self.seq,
                           self.pos, self.slot)

    def cache(self, gen):
        shape = (self.pages, self.hkv, self.page, self.dim)
        return [torch.randn(shape, generator=gen, device="cuda").to(self.dtype) for _ in range(2)]

    def lines(self, cache, r):
        """Cached rows of request r as [Hkv, seq, D] in 64 bits."""
        table = self.table.cpu().numpy()[r]
        n = self.ctx[r] + self.new[r]
        used = table[:-(-n // self.page)] if n else table[:0]
        got = cache[torch.tensor(used, dtype=torch.long, device="cuda")]       # [pages, Hkv, P, D]
        return got.permute(1, 0, 2, 3).reshape(self.hkv, -1, self.dim)[:, :n].double().cpu().numpy()


def check_attention(s, seed=1, q_pad=0, poison=True, spike=1.0):
    gen = torch.Generator("cuda").manual_seed(seed)
    kc, vc = s.cache(gen)
    if poison:                      # what no token sees: the rest of last pages, spare pages
        seen = torch.zeros(s.pages, s.page, dtype=torch.bool)
        table = s.table.cpu().numpy()
        for r, (c, n) in enumerate(zip(s.ctx, s.new)):
            first = max(0, c - s.window + 1) if s.window and n else 0
            for p in range(first if n else 0, c + n if n else 0):
                seen[table[r][p // s.page], p % s.page] = True
        hide = ~seen.cuda()
        kc.permute(0, 2, 1, 3)[hide] = float("nan")
        vc.permute(0, 2, 1, 3)[hide] = float("inf")
    wide = torch.randn(s.rows, s.hq * s.dim + q_pad, generator=gen, device="cuda").mul_(2 * spike).to(s.dtype)
    q = wide[:, :s.hq * s.dim].view(s.rows, s.hq, s.dim) if not q_pad else wide[:, :s.hq * s.dim].unflatten(1, (s.hq, s.dim))
    out = torch.full((s.rows, s.hq, s.dim), 7.0, device="cuda", dtype=s.dtype)
    args = (q, s.start, s.seq, max(s.new), kc, vc, s.table)
    s.handle.forward(*args, out)
    again = torch.full_like(out, 7.0)
    s.handle.forward(*args, again)
    assert torch.equal(out, again)                         # the same bits whatever the CTAs' order
    assert s.handle.status() == moe.MOE_OK
    got, qh, row = out.double().cpu().numpy(), q.double().cpu().numpy(), 0
    tol = 2.0 ** -7 if s.dtype is torch.bfloat16 else 2e-4
    rng = np.random.default_rng(seed)
    for r, (c, n) in enumerate(zip(s.ctx, s.new)):
        if n:
            k, v = s.lines(kc, r), s.lines(vc, r)
            if s.window:                                   # keys before every window may be anything
                k[:, :max(0, c - s.window + 1)], v[:, :max(0, c - s.window + 1)] = 0, 0
        some = range(n) if n <= 40 else sorted({0, 1, n - 2, n - 1, *rng.integers(0, n, 24).tolist()})
        for i in some:
            for h in range(s.hq):
                ref, size = oracle.attend(qh[row + i, h], k[h // (s.hq // s.hkv)], v[h // (s.hq // s.hkv)], c + i, s.scale,
                                          s.window)
                err = np.abs(got[row + i, h] - ref)
                assert (err <= tol * size + 1e-30).all(), (r, i, h, float((err / (size + 1e-30)).max()))
        row += n
    assert (out[row:] == 7.0).all()                        # rows of no request are not written


# ------------------------------------------------------------------------------------------ tables
@pytest.mark.parametrize("page", [16, 32, 64, 128])
@pytest.mark.parametrize("ctx,new,pad", [
    ([0], [1], 0), ([15], [1], 0), ([16], [1], 3), ([0], [0], 2), ([5, 8, 0, 128, 127], [4, 0, 3, 1, 2], 5),
    (list(range(300)), [1 + i % 3 for i in range(300)], 1), ([0, 7000, 3], [5000, 1, 700], 0),
    ([i * 7 for i in range(1024)], [i % 2 for i in range(1024)], 16)])
def test_tables(ctx, new, pad, page):
    s = Step(ctx, new, page=page, pad=pad)
    table, start, seq, pos, slot, head = oracle.tables(ctx, new, s.table0, s.free.tolist(), 0, page, s.rows)
    assert s.table.cpu().tolist() == table.tolist()
    assert s.start.cpu().tolist() == start.tolist() and s.seq.cpu().tolist() == seq.tolist()
    assert s.pos.cpu().tolist() == pos.tolist() and s.slot.cpu().tolist() == slot.tolist()
    assert int(s.head) == head                             # free_head_out is free_head here
    assert s.handle.status() == moe.MOE_OK


def test_tables_without_a_free_list_only_map():
    s = Step([30, 5], [2, 7])
    table, pos, slot = s.table.clone(), s.pos.clone(), s.slot.clone()
    h2 = ints([9])
    full = ints([-(-32 // 16) * 16 - 0, 16])
    # the same rows with every page in the tables already: lengths whose pages are all there
    s.handle.tables(ints([30, 5]), ints([2, 7]), s.table, s.free_d, ints([0]), h2, s.start, s.seq, s.pos, s.slot)
    assert torch.equal(table, s.table) and torch.equal(pos, s.pos) and torch.equal(slot, s.slot)
    s.handle.tables(full, ints([0, 0]), s.table, s.free_d[:0], ints([4]), h2, s.start, s.seq, s.pos, s.slot)
    assert int(h2) == 4 and s.handle.status() == moe.MOE_OK


@pytest.mark.parametrize("what", ["free", "width", "rows", "negative"])
def test_tables_report_what_does_not_fit(what):
    s = Step([10, 3], [30, 5])
    table, slot, rows = s.table.clone(), s.slot, s.rows
    new, free, want = [30, 5], s.free_d, moe.MOE_ERR_CAPACITY
    if what == "free":
        free = free[:1]
    elif what == "width":
        table = table[:, :2].contiguous()
    elif what == "rows":
        rows -= 1
    else:
        new, want = [-4, 5], moe.MOE_ERR_BOUNDS
    pos, slot = ints(np.zeros(rows)), ints(np.full(rows, 99))
    s.handle.tables(ints([10, 3]), ints(new), table, free, ints([0]), s.head, s.start, s.seq, pos, slot)
    assert s.handle.status() == want
    assert slot.max() < s.pages * s.page
    s.handle.clear_status()
    assert s.handle.status() == moe.MOE_OK


# --------------------------------------------------------------------------------------------- qkv
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("dim,rotary,pairs,norm,heads", [
    (128, 128, False, True, (8, 2)), (128, 64, False, True, (3, 1)), (64, 64, True, True, (4, 4)), (64, 32, True, False, (6, 2)),
    (128, 0, False, True, (2, 2)), (128, 16, False, False, (5, 1)), (64, 48, False, True, (1, 1))])
def test_qkv(dtype, dim, rotary, pairs, norm, heads):
    hq, hkv = heads
    s = Step([0, 20, 3], [1, 5, 30], dtype, hq, hkv, dim, pad=3, rotary_dim=rotary,
             rotary_style=moe.MOE_ROTARY_PAIRS if pairs else moe.MOE_ROTARY_HALF, norm_eps=1e-5)
    gen = torch.Generator("cuda").manual_seed(3)
    width = (hq + 2 * hkv) * dim
    wide = torch.randn(s.rows, width + 16, generator=gen, device="cuda").to(s.dtype)
    qkv = wide[:, 8:8 + width] if dtype == "bf16" else wide[:, 4:4 + width]       # strided rows
    wq, wk = [(1 + 0.3 * torch.randn(dim, generator=gen, device="cuda")).to(s.dtype) if norm else None for _ in range(2)]
    rope = torch.randn(40, rotary, generator=gen, device="cuda") if rotary else None
    kc, vc = s.cache(gen)
    k0, v0 = kc.clone(), vc.clone()
    q = torch.empty(s.rows, hq, dim, device="cuda", dtype=s.dtype)
    s.handle.qkv(qkv, wq, wk, rope, s.pos, s.slot, q, kc, vc)
    assert s.handle.status() == moe.MOE_OK
    x = qkv.double().cpu().numpy().reshape(s.rows, hq + 2 * hkv, dim)
    pos, slot = s.pos.cpu().numpy(), s.slot.cpu().numpy()
    table = rope.double().cpu().numpy() if rotary else np.zeros((40, 0))
    weights = [None if w is None else w.double().cpu().numpy() for w in (wq, wk)]
    one = 2.0 ** -8 if dtype == "bf16" else 0.0
    half = rotary // 2
    written = np.zeros((s.pages, s.page), bool)
    for t in range(s.rows):
        for h in range(hq + 2 * hkv):
            if h >= hq and slot[t] < 0:
                continue
            w = weights[0 if h < hq else 1]
            plain = oracle.norm_rotate(x[t, h], w, 1e-5, np.ones(0), np.ones(0), pairs)
            ref = oracle.norm_rotate(x[t, h], w, 1e-5, table[pos[t], :half], table[pos[t], half:], pairs)
            if h >= hq + hkv:
                ref = plain = x[t, h]
            if h < hq:
                got = q[t, h]
            else:
                c = kc if h < hq + hkv else vc
                got = c[slot[t] // s.page, (h - hq) % hkv, slot[t] % s.page]
                written[slot[t] // s.page, slot[t] % s.page] = True
            size = 4 * np.abs(plain).max()
            err = np.abs(got.double().cpu().numpy() - ref)
            assert (err <= one * np.abs(ref) + 1e-6 * size).all(), (t, h, err.max())
    keep = torch.tensor(~written).cuda()
    for c, c0 in ((kc, k0), (vc, v0)):
        assert torch.equal(c.permute(0, 2, 1, 3)[keep], c0.permute(0, 2, 1, 3)[keep])


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("dim,rotary,pairs,norm,heads,rows", [
    (128, 128, False, True, (32, 8), 2100), (128, 64, True, False, (60, 10), 1003), (64, 64, False, True, (96, 32), 1200),
    (64, 16, True, True, (7, 7), 7500), (128, 0, False, True, (20, 1), 3700), (128, 128, False, True, (300, 100), 170)])
def test_qkv_of_many_rows(dtype, dim, rotary, pairs, norm, heads, rows):
    # one request's rows, every 97th of them padding, over a pool with the slots in no order
    hq, hkv = heads
    s = Step([0], [4], dtype, hq, hkv, dim, rotary_dim=rotary, rotary_style=moe.MOE_ROTARY_PAIRS if pairs else moe.MOE_ROTARY_HALF,
             norm_eps=1e-5)
    gen = torch.Generator("cuda").manual_seed(rows)
    wide = torch.randn(rows, (hq + 2 * hkv) * dim + 8, generator=gen, device="cuda").mul_(3).to(s.dtype)
    qkv = wide[:, :(hq + 2 * hkv) * dim]
    w = [torch.randn(dim, generator=gen, device="cuda").to(s.dtype) if norm else None for _ in range(2)]
    rope = torch.randn(2 * rows, rotary, generator=gen, device="cuda") if rotary else None
    pos = torch.randint(0, 2 * rows, (rows,), generator=gen, device="cuda").int()
    pages = -(-rows // s.page) + 2
    slot = torch.randperm(pages * s.page, generator=gen, device="cuda")[:rows].int()
    slot[::97] = -1
    q = torch.full((rows, hq, dim), 7.0, device="cuda", dtype=s.dtype)
    caches = [torch.full((pages, hkv, s.page, dim), 7.0, device="cuda", dtype=s.dtype) for _ in range(2)]
    s.handle.qkv(qkv, *w, rope, pos, slot, q, *caches)
    assert s.handle.status() == moe.MOE_OK
    x = qkv.double().view(rows, hq + 2 * hkv, dim)
    size = x.abs().amax(-1, keepdim=True)
    if norm:
        scale = torch.cat([w[0].double().expand(hq, dim), w[1].double().expand(hkv, dim)])
        y = x[:, :hq + hkv] / (x[:, :hq + hkv].square().mean(-1, keepdim=True) + 1e-5).sqrt() * scale
        size = torch.cat([y.abs().amax(-1, keepdim=True), size[:, hq + hkv:]], 1)
    else:
        y = x[:, :hq + hkv].clone()
    if rotary:
        cos, sin = rope.double()[pos.long()].split(rotary // 2, -1)
        cos, sin = cos[:, None], sin[:, None]
        a, b = (y[..., 0:rotary:2], y[..., 1:rotary:2]) if pairs else (y[..., :rotary // 2], y[..., rotary // 2:rotary])
        a, b = a * cos - b * sin, b * cos + a * sin
        size = size * 2 * rope.abs().max().double()                      # bounds |a cos| + |b sin|
        y[..., :rotary] = torch.stack([a, b], -1).flatten(-2) if pairs else torch.cat([a, b], -1)
    one = 2.0 ** -8 if s.dtype is torch.bfloat16 else 2.0 ** -24
    ref = torch.cat([y, x[:, hq + hkv:]], 1)

    def close(got, ref, size):
        return bool(((got.double() - ref).abs() <= one * ref.abs() + 1e-6 * size).all())
    assert close(q, ref[:, :hq], size[:, :hq])
    live = slot >= 0
    at = slot[live].long()
    for c, h in zip(caches, (hq, hq + hkv)):
        assert close(c[at // s.page, :, at % s.page], ref[live, h:h + hkv], size[live, h:h + hkv])
        flat = c.permute(0, 2, 1, 3).reshape(-1, hkv, dim)
        rest = torch.ones(len(flat), dtype=torch.bool, device="cuda")
        rest[at] = False
        assert (flat[rest] == 7.0).all()
    # a position and a slot outside are reported, the rest is done
    pos[rows // 2], slot[rows // 3] = 2 * rows, pages * s.page
    s.handle.qkv(qkv, *w, rope, pos, slot, q, *caches)
    assert s.handle.status() == moe.MOE_ERR_BOUNDS


def test_qkv_reports_positions_and_slots_out_of_range():
    s = Step([0], [4], hq=2, hkv=1)
    gen = torch.Generator("cuda").manual_seed(3)
    qkv = torch.randn(4, 4 * 128, generator=gen, device="cuda").bfloat16()
    rope = torch.randn(3, 128, generator=gen, device="cuda")              # position 3 is outside
    kc, vc = s.cache(gen)
    q = torch.empty(4, 2, 128, device="cuda", dtype=torch.bfloat16)
    s.handle.qkv(qkv, None, None, rope, s.pos, s.slot, q, kc, vc)
    assert s.handle.status() == moe.MOE_ERR_BOUNDS
    s.handle.clear_status()
    before = kc.clone()
    s.handle.qkv(qkv, None, None, torch.cat([rope, rope]), s.pos, ints([s.pages * s.page, 1 << 30, -1, -7]), q, kc, vc)
    assert s.handle.status() == moe.MOE_ERR_BOUNDS and torch.equal(before, kc)


# --------------------------------------------------------------------------------------- attention
LENGTHS = [
    ([0], [1]), ([15], [1]), ([16], [1]), ([1], [1]), ([127], [1]), ([128], [1]), ([0], [17]), ([3], [33]), ([200], [2]),
    ([0, 31, 300, 5, 64], [1, 1, 1, 1, 1]), ([40, 0, 129, 7], [0, 5, 1, 130]), ([2000], [1]), ([513, 1], [70, 0]),
]


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("ctx,new", LENGTHS)
def test_attention_lengths(dtype, ctx, new):
    check_attention(Step(ctx, new, dtype, pad=2))


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("dim", [64, 128])
@pytest.mark.parametrize("heads", [(1, 1), (3, 1), (8, 1), (16, 1), (6, 2), (20, 4), (8, 8), (40, 2)])
def test_attention_heads(dtype, dim, heads):
    check_attention(Step([70, 0, 17], [1, 20, 3], dtype, *heads, dim))


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("page", [16, 32, 64, 128])
@pytest.mark.parametrize("window", [0, 1, 16, 50, 129])
def test_attention_pages_and_windows(dtype, page, window):
    check_attention(Step([300, 0, 64, 10], [1, 40, 1, 150], dtype, page=page, window=window))
    check_attention(Step([700, 3], [1, 1], dtype, page=page, window=window))


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_attention_strided_queries_and_sharp_scores(dtype):
    check_attention(Step([90, 4], [3, 65], dtype), q_pad=8)
    check_attention(Step([500], [1], dtype, scale=0.02), spike=20.0)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_attention_long_rows_are_split(dtype):
    check_attention(Step([9000, 17, 4000], [1, 1, 1], dtype, 8, 1, page=64), poison=False)
    check_attention(Step([30011], [1], dtype, 4, 1, page=32), poison=False)
    check_attention(Step([6000], [9], dtype, 8, 2), poison=False)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("dim", [64, 128])
@pytest.mark.parametrize("hq", [1, 2, 3, 4, 8, 16])
def test_attention_of_few_rows_in_many_pieces(dtype, dim, hq):
    check_attention(Step([20500], [1], dtype, hq, 1, dim, page=128), poison=False)
    check_attention(Step([2100], [3], dtype, hq, 1, dim), poison=False)


@pytest.mark.parametrize("new", [40, 100, 203])
def test_attention_of_a_chunk_in_many_pieces(new):
    check_attention(Step([5000], [new], "bf16", 8, 1), poison=False)
    check_attention(Step([2000, 30], [new, 7], "bf16", 4, 1, 64, window=700))


def test_attention_prefill_of_many_rows():
    check_attention(Step([0, 100], [700, 333], "bf16", 8, 2), poison=True)
    check_attention(Step([1500], [600], "bf16", 16, 2, page=64), poison=True)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("count", [31, 33, 260, 500, 1024])
@pytest.mark.parametrize("most", [1, 5, 60])
def test_attention_of_many_requests(dtype, count, most):
    rng = np.random.default_rng(count + most)
    new = rng.integers(0, most + 1, count)
    new[count // 2], new[-1] = most, 0
    if most > 1:                                           # most requests add one token or none
        new[rng.random(count) < 0.8] = 1
        new[rng.random(count) < 0.1] = 0
        new[0] = most
    ctx = rng.integers(0, 40, count)
    ctx[rng.integers(0, count, 3)] = 500
    check_attention(Step(ctx.tolist(), new.tolist(), dtype, 4, 2, 64, pad=1))


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("new", [2, 3, 4, 5, 63, 64, 65])
@pytest.mark.parametrize("window", [0, 37])
def test_attention_of_row_tiles_full_and_not(dtype, new, window):
    check_attention(Step([333, 4], [new, 1], dtype, 8, 1, window=window))


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_offsets_past_32_bits(dtype):
    # pages of 2 heads x 16 x 128 elements: 2^32 elements lie below page 2^20
    s = Step([100, 7], [1, 40], dtype)
    far = (1 << 20) + 9
    need = torch.unique(s.table[(s.table < s.pages)])
    kc, vc = (torch.empty(far + s.pages, s.hkv, s.page, s.dim, device="cuda", dtype=s.dtype) for _ in range(2))
    gen = torch.Generator("cuda").manual_seed(4)
    near = s.cache(gen)
    for c, n in zip((kc, vc), near):
        c[far:] = n
    moved = torch.where(s.table < s.pages, s.table + far, s.table)
    assert need.numel() and kc.numel() > 1 << 32
    q = torch.randn(s.rows, s.hq, s.dim, generator=gen, device="cuda").to(s.dtype)
    for start, seq, new, table, rows in ((s.start, s.seq, 40, moved, slice(0, None)),                       # a chunk
                                         (ints([0, 1]), s.seq[:1].contiguous(), 1, moved[:1].contiguous(), slice(0, 1))):
        out, ref = torch.zeros_like(q), torch.zeros_like(q)
        s.handle.forward(q, start, seq, new, kc, vc, table, out)
        s.handle.forward(q, start, seq, new, *near, s.table[:len(seq)].contiguous(), ref)
        assert torch.equal(out[rows], ref[rows]) and ref[rows].any()
    # and the write of new rows there
    qkv = torch.randn(s.rows, (s.hq + 2 * s.hkv) * s.dim, generator=gen, device="cuda").to(s.dtype)
    rope = torch.randn(200, s.dim, generator=gen, device="cuda")
    outs = []
    for c, slot in (((kc, vc), s.slot + far * s.page), (near, s.slot)):
        q2 = torch.empty_like(q)
        s.handle.qkv(qkv, None, None, rope, s.pos, slot, q2, *c)
        outs.append(q2)
    assert torch.equal(*outs) and torch.equal(kc[far:], near[0]) and torch.equal(vc[far:], near[1])
    assert s.handle.status() == moe.MOE_OK


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_rows_before_the_first_key_are_zero(dtype):
    s = Step([0], [6], dtype)
    gen = torch.Generator("cuda").manual_seed(1)
    kc, vc = s.cache(gen)
    q = torch.randn(6, s.hq, s.dim, generator=gen, device="cuda").to(s.dtype)
    out = torch.full_like(q, 7.0)
    s.handle.forward(q, s.start, ints([2]), 6, kc, vc, s.table, out)      # six rows, two keys: four rows see none
    assert (out[:4] == 0).all() and torch.isfinite(out).all() and (out[4:] != 0).any()
    out.fill_(7.0)
    s.handle.forward(q, s.start, ints([0]), 6, kc, vc, s.table, out)
    assert (out == 0).all() and s.handle.status() == moe.MOE_OK


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_attention_reports_bad_tables_and_lengths(dtype):
    s = Step([40], [1], dtype)
    gen = torch.Generator("cuda").manual_seed(1)
    kc, vc = s.cache(gen)
    q = torch.randn(1, s.hq, s.dim, generator=gen, device="cuda").to(s.dtype)
    out = torch.empty_like(q)
    for table, seq, start in ((ints([[0, s.pages, 1, 0]]), [41], [0, 1]), (ints([[0, -1, 1, 0]]), [41], [0, 1]),
                              (s.table, [1 << 30], [0, 1]), (s.table, [-5], [0, 1]), (s.table, [41], [0, 9]),
                              (s.table, [41], [-1, 1]), (s.table, [41], [1, 0])):
        s.handle.forward(q, ints(start), ints(seq), 1, kc, vc, table, out)
        assert s.handle.status() == moe.MOE_ERR_BOUNDS, (seq, start)
        s.handle.clear_status()
    s.handle.forward(q, s.start, s.seq, 1, kc, vc, s.table, out)
    assert s.handle.status() == moe.MOE_OK


def test_attention_on_another_stream_and_in_a_graph():
    s = Step([300, 20], [1, 1])
    gen = torch.Generator("cuda").manual_seed(1)
    kc, vc = s.cache(gen)
    q = torch.randn(2, s.hq, s.dim, generator=gen, device="cuda").to(s.dtype)
    out, ref = torch.empty_like(q), torch.empty_like(q)
    s.handle.forward(q, s.start, s.seq, 1, kc, vc, s.table, ref)
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    s.handle.forward(q, s.start, s.seq, 1, kc, vc, s.table, out, stream=side)
    side.synchronize()
    assert torch.equal(out, ref)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        s.handle.forward(q, s.start, s.seq, 1, kc, vc, s.table, out)
    out.zero_()
    q.mul_(0.5)
    graph.replay()
    s.handle.forward(q, s.start, s.seq, 1, kc, vc, s.table, ref)
    assert torch.equal(out, ref)


def test_refusals():
    good = dict(num_q_heads=8, num_kv_heads=2, head_dim=128, page_size=16)
    for bad in (dict(num_q_heads=7), dict(num_kv_heads=0), dict(head_dim=96), dict(page_size=8), dict(page_size=48),
                dict(rotary_dim=24), dict(rotary_dim=256), dict(rotary_style=2), dict(window=-1), dict(softmax_scale=0.0),
                dict(softmax_scale=float("nan")), dict(norm_eps=-1.0), dict(dtype=moe.MOE_FP8_E4M3_B128)):
        with pytest.raises(moe.MoeError) as e:
            moe.Attention(moe.make_attn_config(**{**good, **bad}))
        assert e.value.status == moe.MOE_ERR_INVALID, bad
    s = Step([40], [2])
    gen = torch.Generator("cuda").manual_seed(1)
    kc, vc = s.cache(gen)
    q = torch.zeros(2, s.hq, s.dim, device="cuda", dtype=s.dtype)
    out = torch.empty_like(q)
    with pytest.raises(ValueError):
        s.handle.forward(q.float(), s.start, s.seq, 2, kc, vc, s.table, out)
    with pytest.raises(ValueError):
        s.handle.forward(q, s.start, s.seq.long(), 2, kc, vc, s.table, out)
    with pytest.raises(ValueError):
        s.handle.forward(q, s.start, s.seq, 2, kc, vc[:, :1], s.table, out)
    with pytest.raises(ValueError):
        s.handle.forward(q.transpose(1, 2).contiguous().transpose(1, 2), s.start, s.seq, 2, kc, vc, s.table, out)
    lib, h, st = moe._lib, s.handle.h, torch.cuda.current_stream().cuda_stream

    def raw(**kw):
        a = dict(q=q.data_ptr(), stride=s.hq * s.dim, rows=2, start=s.start.data_ptr(), seq=s.seq.data_ptr(), R=1, new=2,
                 k=kc.data_ptr(), v=vc.data_ptr(), pages=s.pages, table=s.table.data_ptr(), width=s.width, out=out.data_ptr())
        a.update(kw)
        return lib.moe_attn_forward(h, a["q"], a["stride"], a["rows"], a["start"], a["seq"], a["R"], a["new"], a["k"], a["v"],
                                    a["pages"], a["table"], a["width"], a["out"], st)
    assert raw() == moe.MOE_OK
    for kw in (dict(q=None), dict(q=q.data_ptr() + 2), dict(stride=8), dict(stride=s.hq * s.dim + 1), dict(rows=-1), dict(R=1025),
               dict(new=3), dict(new=-1), dict(k=None), dict(v=vc.data_ptr() + 4), dict(pages=0), dict(pages=1 << 30),
               dict(table=None), dict(width=0), dict(out=None), dict(out=out.data_ptr() + 8), dict(start=s.start.data_ptr() + 1)):
        assert raw(**kw) == moe.MOE_ERR_INVALID, kw
    assert raw(R=0) == moe.MOE_OK and raw(rows=0, new=0) == moe.MOE_OK
    # seq_len must not be the lengths it is computed from
    assert lib.moe_attn_tables(h, s.seq.data_ptr(), s.seq.data_ptr(), 1, s.table.data_ptr(), s.width, s.free_d.data_ptr(), 1,
                               s.head.data_ptr(), s.head.data_ptr(), 2, s.start.data_ptr(), s.seq.data_ptr(),
                               s.pos.data_ptr(), s.slot.data_ptr(), st) == moe.MOE_ERR_INVALID


@pytest.mark.parametrize("page", [16, 64])
def test_tables_that_are_complete_are_only_mapped(page):
    # growth over page ends, requests that rest or begin, and no free list: the pages come from the table itself
    ctx, new, rows = [16, 5, 0, 127, 200, 64, 0], [1, 30, 40, 2, 0, 64, 0], 140
    rng = np.random.default_rng(page)
    need = [-(-(c + n) // page) for c, n in zip(ctx, new)]
    table = np.full((len(ctx), max(need) + 1), 1 << 30)
    order = rng.permutation(sum(need))
    for r, n in enumerate(need):
        table[r, :n] = order[sum(need[:r]):sum(need[:r + 1])]
    handle = moe.Attention(moe.make_attn_config(8, 2, 128, page))
    given, none = ints(table), ints([])
    head, start, seq, pos, slot = ints([5]), ints(np.zeros(len(ctx) + 1)), ints(np.zeros(len(ctx))), ints(np.zeros(rows)), ints(np.zeros(rows))
    handle.tables(ints(ctx), ints(new), given, none, ints([7]), head, start, seq, pos, slot)
    assert handle.status() == moe.MOE_OK
    assert given.cpu().tolist() == table.tolist() and int(head) == 7         # nothing is taken or written
    where = [(r, p) for r, (c, n) in enumerate(zip(ctx, new)) for p in range(c, c + n)]
    pad = rows - len(where)
    assert pos.cpu().tolist() == [p for _, p in where] + [0] * pad
    assert slot.cpu().tolist() == [int(table[r, p // page]) * page + p % page for r, p in where] + [-1] * pad
    assert start.cpu().tolist() == [0, *np.cumsum(new).tolist()]
    assert seq.cpu().tolist() == [c + n for c, n in zip(ctx, new)]
    # a page that is missing all the same is reported, and its rows have no slot
    given[1, (5 + 30 - 1) // page] = -1
    handle.tables(ints(ctx), ints(new), given, none, ints([7]), head, start, seq, pos, slot)
    assert handle.status() == moe.MOE_ERR_BOUNDS and int(slot[30]) == -1 and int(slot[0]) >= 0


@pytest.mark.parametrize("dtype,hq,hkv,page,width,requests,new", [
    ("f32", 64, 1, 16, 1 << 20, 1, 2100), ("f32", 64, 1, 16, 1 << 20, 1, 4200),        # above 2^30 units, 2^31
    ("f32", 64, 1, 16, 1 << 20, 1, 8300), ("f32", 64, 1, 16, 1 << 20, 34, 70),         # and 2^32; many requests
    ("f32", 64, 64, 16, 1 << 20, 33, 1), ("f32", 64, 64, 16, 1 << 20, 32, 9),          # few rows
    ("bf16", 64, 64, 128, 1 << 20, 20, 1), ("bf16", 64, 64, 128, 1 << 19, 40, 1),
    ("bf16", 512, 8, 128, 1 << 20, 1, 1100), ("bf16", 512, 8, 128, 1 << 20, 40, 28)])  # chunks
def test_steps_of_more_units_than_are_counted_are_refused(dtype, hq, hkv, page, width, requests, new):
    # every table entry names the one page of the cache, so that the lengths are long but the memory is not
    dt = DT[dtype][0]
    handle = moe.Attention(moe.make_attn_config(hq, hkv, 64, page, DT[dtype][1]))
    rows = requests * new
    table = torch.zeros(requests, width, dtype=torch.int32, device="cuda")
    start, seq = ints(np.arange(requests + 1) * new), ints([width * page] * requests)
    kc, vc = torch.ones(1, hkv, page, 64, dtype=dt, device="cuda"), torch.full((1, hkv, page, 64), 3.0, dtype=dt, device="cuda")
    q = torch.zeros(rows, hq, 64, dtype=dt, device="cuda")
    out = torch.full_like(q, 7.0)
    handle.forward(q, start, seq, new, kc, vc, table, out)
    assert handle.status() == moe.MOE_ERR_CAPACITY and (out == 7.0).all()
    handle.clear_status()
    seq.fill_(new)                                         # the same rows over as many keys; 3 n * fl(1 / n), joined or not
    handle.forward(q, start, seq, new, kc, vc, table, out)
    assert handle.status() == moe.MOE_OK and ((out - 3.0).abs() <= 2.0 ** -20).all()


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("page", [16, 32, 64, 128])
@pytest.mark.parametrize("ctx,new,window", [([700, 1000], [1, 1], 20), ([1100, 5], [40, 1], 50), ([400, 3000], [3, 130], 129)])
def test_pages_behind_the_window_may_be_gone(dtype, page, ctx, new, window):
    # a server gives the pages that no token of the call sees to others and marks their entries
    s = Step(ctx, new, dtype, page=page, window=window)
    gen = torch.Generator("cuda").manual_seed(5)
    kc, vc = s.cache(gen)
    q = torch.randn(s.rows, s.hq, s.dim, generator=gen, device="cuda").to(s.dtype)
    ref, out = torch.full_like(q, 7.0), torch.full_like(q, 9.0)
    s.handle.forward(q, s.start, s.seq, max(new), kc, vc, s.table, ref)
    assert s.handle.status() == moe.MOE_OK
    for mark in (-1, s.pages, 1 << 30):
        table = s.table.clone()
        for r, c in enumerate(ctx):
            gone = max(0, c - window + 1) // page              # pages wholly before the first token's window
            table[r, :gone] = mark
        s.handle.forward(q, s.start, s.seq, max(new), kc, vc, table, out)
        assert s.handle.status() == moe.MOE_OK, mark
        assert torch.equal(out, ref)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("new,seq", [(1, 1), (6, 2), (60, 7), (9, 40)])
def test_a_window_of_any_size_sees_all_keys(dtype, new, seq):
    # rows before the first key have negative positions, from which a window near 2^31 is subtracted
    outs = []
    for window in (0, (1 << 31) - 1, (1 << 31) - 3, 1 << 30):
        s = Step([max(0, seq - new)], [new], dtype, window=window)
        gen = torch.Generator("cuda").manual_seed(1)
        kc, vc = s.cache(gen)
        q = torch.randn(new, s.hq, s.dim, generator=gen, device="cuda").to(s.dtype)
        outs.append(torch.full_like(q, 7.0))
        s.handle.forward(q, s.start, ints([seq]), new, kc, vc, s.table, outs[-1])
        assert s.handle.status() == moe.MOE_OK
        assert torch.equal(outs[-1], outs[0]), window
    assert (outs[0][:max(0, new - seq)] == 0).all() and (outs[0][new - 1] != 0).any()


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("new", [1, 40])
def test_lengths_near_31_bits(dtype, new):
    # every table entry names the one page, so keys repeat every 128; the window keeps the work small
    s = Step([0], [new], dtype, page=128, window=30)
    gen = torch.Generator("cuda").manual_seed(1)
    kc, vc = (torch.randn(1, s.hkv, 128, s.dim, generator=gen, device="cuda").to(s.dtype) for _ in range(2))
    q = torch.randn(new, s.hq, s.dim, generator=gen, device="cuda").to(s.dtype)
    table = torch.zeros(1, 1 << 24, dtype=torch.int32, device="cuda")
    ref, out = torch.full_like(q, 7.0), torch.full_like(q, 9.0)
    most = (1 << 31) - 1 - 2 * moe.MOE_ATTN_MAX_ROWS
    for seq in (most, most - 1, most - 60, 1 << 30):
        s.handle.forward(q, s.start, ints([256 + seq % 128]), new, kc, vc, table, ref)
        s.handle.forward(q, s.start, ints([seq]), new, kc, vc, table, out)
        assert s.handle.status() == moe.MOE_OK
        # two results over the same keys in other places of their units, each off by at most 2^-7 sum p|v| (about 1 here)
        assert ((out.float() - ref.float()).abs() <= 2.0 ** -6).all() and ref.float().abs().max() > 0.1
    for seq in (most + 1, (1 << 31) - 1):                  # longer ones are reported and cut there
        s.handle.forward(q, s.start, ints([seq]), new, kc, vc, table, out)
        assert s.handle.status() == moe.MOE_ERR_BOUNDS
        s.handle.clear_status()


@pytest.mark.parametrize("page", [16, 128])
@pytest.mark.parametrize("where", ["table", "free"])
def test_tables_report_pages_whose_slots_have_no_number(page, where):
    # page * page_size past 31 bits would come out as the slot of another page; so would a negative entry
    handle = moe.Attention(moe.make_attn_config(8, 2, 128, page))
    for bad in ((1 << 31) // page, (1 << 32) // page + 3, (1 << 31) - 1, -5):
        if bad >= 1 << 31:
            continue
        table, free = ints([[4, 9], [6, 8]]), ints([3, 2])
        if where == "table":
            table[0, 0] = bad                                  # request 0 goes on in its first page
            ctx = [1, 1]
        else:
            free[0] = bad                                      # or takes it anew
            ctx = [0, 1]
        start, seq, pos, slot = ints([0, 0, 0]), ints([0, 0]), ints([0] * 2), ints([99] * 2)
        handle.tables(ints(ctx), ints([1, 1]), table, free, ints([0]), ints([0]), start, seq, pos, slot)
        assert handle.status() == moe.MOE_ERR_BOUNDS and slot.tolist() == [-1, 6 * page + 1], bad
        handle.clear_status()
