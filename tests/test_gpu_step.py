"""The operators between attention, experts and token choice, run together as a step runs them.

A step's dense path: residual joins and norms, 4-bit projections, scores of the sampled tokens, on the buffers of one
stream, eagerly and in a captured graph.  The reference is the 64-bit oracle fed with the same inputs, operator by operator, so
that every tolerance is that of the operator's own test.
"""
import numpy as np
import pytest
import torch

import expert_offload_slot_gb300 as moe
from oracle import step as oracle

pytestmark = pytest.mark.gpu


def host(t):
    return t.double().cpu().numpy()


@pytest.mark.parametrize("dtype, rows", [(torch.float32, 1), (torch.float32, 7), (torch.bfloat16, 1), (torch.bfloat16, 12),
                                         (torch.bfloat16, 150)])
def test_a_step_of_the_dense_path(dtype, rows):
    hidden, inner, vocab, group = 512, 1024, 6000, 64
    rng = np.random.default_rng(rows)

    def weight(n, k):
        codes, scales = moe.moe_q4_pack(rng.standard_normal((n, k), np.float32) * k ** -0.5, group)
        return torch.from_numpy(codes).cuda(), torch.from_numpy(scales).cuda()
    w_in, w_out, w_head = weight(inner, hidden), weight(hidden, inner), weight(vocab, hidden)
    tensor = lambda *s: torch.from_numpy(rng.standard_normal(s).astype(np.float32)).cuda()  # noqa: E731
    stream = tensor(rows, hidden)                              # the residual stream in 32 bits
    norm = [(1 + 0.1 * tensor(hidden)).to(dtype) for _ in range(3)]
    new = lambda *s, t=dtype: torch.empty(*s, dtype=t, device="cuda")  # noqa: E731
    h, mid, out, after, last = new(rows, hidden), new(rows, inner), new(rows, hidden), new(rows, hidden, t=torch.float32), new(rows, hidden)
    logits, u = new(rows, vocab, t=torch.float32), torch.rand(rows, device="cuda")
    ids, logp, ent = new(rows, t=torch.int32), new(rows, t=torch.float32), new(rows, t=torch.float32)
    rank, top, toplp = new(rows, t=torch.int32), new(rows, 4, t=torch.int32), new(rows, 4, t=torch.float32)

    def step():
        moe.moe_residual_norm(None, stream, None, h, pre_weight=norm[0])
        moe.moe_linear_q4(h, *w_in, mid, group=group)
        moe.moe_linear_q4(mid, *w_out, out, group=group)
        moe.moe_residual_norm(out, stream, after, last, post_weight=norm[1], pre_weight=norm[2], gate=h[:, :1], gate_sigmoid=True,
                              residual_scale=0.5)
        moe.moe_linear_q4(last, *w_head, logits, group=group)
        moe.moe_sample(logits, u, ids)
        moe.moe_logprobs(logits, ids, logp, entropy=ent, rank=rank, top_ids=top, top_logp=toplp)

    def check():
        half, eps = torch.finfo(dtype).eps / 2, 2.0 ** -24
        ref = oracle.residual_norm(None, host(stream), pre=host(norm[0]))[1]
        assert (np.abs(host(h) - ref) <= (100 * eps + half) * np.abs(ref)).all()
        for x, w, y in ((h, w_in, mid), (mid, w_out, out), (last, w_head, logits)):
            ref, size = oracle.linear_q4(host(x), w[0].cpu().numpy(), host(w[1]), group)
            assert (np.abs(host(y) - ref) <= (52 + x.shape[1] / group) * 2 * eps * size + torch.finfo(y.dtype).eps / 2 * np.abs(ref)).all()
        ref, y, size = oracle.residual_norm(host(out), host(stream), host(norm[1]), host(norm[2]), host(h[:, :1]), True, 0.5)
        assert (np.abs(host(after) - ref) <= 100 * eps * size + 2.0 ** -24 * np.abs(ref)).all()
        per = np.abs(y / ref)
        assert (np.abs(host(last) - y) <= 100 * eps * (size * per + np.abs(y)) + half * np.abs(y)).all()
        tol = (52 + vocab / 256) * eps
        for r in range(rows):
            lp, e, rk, best, blp = oracle.logprobs(host(logits[r]), int(ids[r]), 4)
            assert 0 <= int(ids[r]) < vocab and int(rank[r]) == rk and top[r].tolist() == best
            assert abs(float(logp[r]) - lp) <= tol - 2.0 ** -22 * lp and abs(float(ent[r]) - e) <= 24 * tol + 2.0 ** -22 * e
            assert np.abs(host(toplp[r]) - blp).max() <= tol + 2.0 ** -22 * 40

    step()
    check()
    first = [t.clone() for t in (h, mid, out, after, last, logits, ids, logp, ent, rank, top, toplp)]
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=torch.cuda.Stream()):
        step()
    for _ in range(2):                                         # the same bits from a replay
        graph.replay()
        assert all(torch.equal(a, b) for a, b in zip(first, (h, mid, out, after, last, logits, ids, logp, ent, rank, top, toplp)))
    stream.mul_(0.5).add_(1)                                   # and new results on new inputs
    graph.replay()
    check()
    assert moe.moe_step_status() == moe.MOE_OK


def test_two_streams_at_once():
    """The operators keep nothing between calls: calls on two streams do not disturb each other."""
    rng = np.random.default_rng(0)
    streams = [torch.cuda.Stream() for _ in range(2)]
    codes = torch.from_numpy(rng.integers(0, 256, (20480, 512), dtype=np.uint8)).cuda()
    scales = torch.rand(20480, 8, device="cuda")
    xs = [torch.randn(40, 1024, device="cuda").bfloat16() for _ in range(2)]
    outs = [[torch.empty(40, 20480, device="cuda") for _ in range(2)] for _ in range(3)]
    lps = [[torch.empty(40, device="cuda") for _ in range(2)] for _ in range(3)]
    t = torch.arange(40, dtype=torch.int32, device="cuda")

    def work(i, k):
        moe.moe_linear_q4(xs[i], codes, scales, outs[k][i])
        moe.moe_logprobs(outs[k][i], t, lps[k][i])
    for i in range(2):
        work(i, 0)
    torch.cuda.synchronize()
    for k in (1, 2):
        for i, s in enumerate(streams):
            with torch.cuda.stream(s):
                work(i, k)
    torch.cuda.synchronize()
    for k in (1, 2):
        for i in range(2):
            assert torch.equal(outs[0][i], outs[k][i]) and torch.equal(lps[0][i], lps[k][i])
