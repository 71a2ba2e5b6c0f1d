"""moe_sample against the 64-bit oracle.

The token has to be the oracle's unless u lies within 1e-5 of a boundary between two kept tokens:
fp32 exponentials of arguments up to 27.7 are off by at most 27.7 2^-23 + 2^-23 = 3.5e-6 relative,
so is every partial sum over the total, twice that at worst.  Rows with a near cut (top-p, min-p)
are drawn so that the cut is far.  logp: 2e-5.
"""
import numpy as np
import pytest
import torch

import expert_offload_slot_gb300 as moe
from oracle import sampling as oracle

pytestmark = pytest.mark.gpu


def run(x, u, temperature=None, top_k=None, top_p=None, min_p=None):
    rows = x.shape[0]
    ids = torch.full((rows,), -9, dtype=torch.int32, device="cuda")
    logp = torch.full((rows,), 9.0, device="cuda")
    f = lambda v: None if v is None else torch.tensor(v, dtype=torch.float32, device="cuda")  # noqa: E731
    k = None if top_k is None else torch.tensor(top_k, dtype=torch.int32, device="cuda")
    moe.moe_sample(x, f(u), ids, logp, temperature=f(temperature), top_k=k, top_p=f(top_p), min_p=f(min_p))
    return ids.cpu().numpy(), logp.cpu().numpy()


def cut_is_far(x, t, k, p, m):
    """No kept mass within 1e-5 of the top-p cut, no weight within 1e-5 of min-p."""
    x = np.asarray(x, np.float64)
    w = np.exp((x - x.max()) / t)
    order = sorted(range(len(x)), key=lambda i: (-x[i], i))[:k if k > 0 else None]
    c = np.cumsum(w[order]) / w[order].sum()
    return (p >= 1 or np.abs(c - p).min() > 1e-5) and (m <= 0 or np.abs(w / m - 1).min() > 1e-5)


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("vocab", [1, 2, 31, 33, 1000, 4097, 8191, 32771, 100277, 327680])
def test_rows_against_the_oracle(dtype, vocab):
    rng = np.random.default_rng(vocab)
    gen = torch.Generator("cuda").manual_seed(vocab)
    rows = 12 if vocab < 50000 else 5
    wide = (3 * torch.randn(rows, vocab + 5, generator=gen, device="cuda")).to(dtype)
    x = wide[:, 3:3 + vocab]                                   # rows at odd offsets
    host = x.double().cpu().numpy()
    t, k, p, m, u = [], [], [], [], rng.random(rows).astype(np.float32)
    for r in range(rows):
        while True:
            one = (float(np.float32(rng.uniform(0.3, 1.5))), int(rng.choice([0, 1, 2, 7, 50, 700])),
                   float(np.float32(rng.choice([1.0, rng.uniform(0.05, 0.99)]))), float(np.float32(rng.choice([0.0, rng.uniform(0.01, 0.3)]))))
            if cut_is_far(host[r], *one):
                break
        for to, v in zip((t, k, p, m), one):
            to.append(v)
    t[0] = 0.0
    ids, logp = run(x, u, t, k, p, m)
    for r in range(rows):
        ref, lp, margin = oracle.sample(host[r], t[r], k[r], p[r], m[r], float(u[r]))
        if margin > 1e-5:
            assert ids[r] == ref, (r, t[r], k[r], p[r], m[r])
            assert abs(logp[r] - lp) <= 2e-5
        else:
            assert ids[r] >= 0


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_ties_go_to_the_lowest_index(dtype):
    x = torch.zeros(4, 20000, device="cuda", dtype=dtype)      # all equal
    x[1, 777] = 1.0
    ids, logp = run(x, [0.999999, 0.0, 0.5, 0.99], [1.0, 0.0, 1.0, 1.0], [3, 0, 0, 20000], [1.0, 1.0, 0.25, 1.0])
    assert ids.tolist() == [2, 777, 2500, 19800]               # 0.25 of the mass: indices 0 .. 4999
    assert abs(logp[0] + np.log(3)) < 1e-5 and abs(logp[2] + np.log(5000)) < 2e-5
    x = torch.tensor([[0.0, -0.0, 0.0, -1.0]], device="cuda", dtype=dtype)       # -0 is 0
    assert run(x, [0.99], None, [2])[0].tolist() == [1]


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("vocab", [1500, 20011, 150000])
def test_long_lists_with_a_mass_cut(dtype, vocab):
    rng = np.random.default_rng(vocab)
    gen = torch.Generator("cuda").manual_seed(vocab)
    ks = [129, 256, 257, 300, 512, 513, 900, 1000, 1024, 1025]
    x = (2 * torch.randn(len(ks), vocab, generator=gen, device="cuda")).to(dtype)
    host, u = x.double().cpu().numpy(), rng.random(len(ks)).astype(np.float32)
    t, p = [], []
    for r, k in enumerate(ks):                                 # hot rows keep hundreds of tokens, cold ones few
        while True:
            one = float(np.float32(rng.uniform(0.3, 4.0))), float(np.float32(rng.uniform(0.2, 0.999)))
            if cut_is_far(host[r], one[0], k, one[1], 0.0):
                break
        t.append(one[0])
        p.append(one[1])
    ids, logp = run(x, u, t, ks, p)
    for r, k in enumerate(ks):
        ref, lp, margin = oracle.sample(host[r], t[r], k, p[r], 0.0, float(u[r]))
        assert ids[r] >= 0
        if margin > 1e-5:
            assert ids[r] == ref, (k, t[r], p[r])
            assert abs(logp[r] - lp) <= 2e-5


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_infinities_and_nan(dtype):
    inf, nan, low = float("inf"), float("nan"), torch.finfo(dtype).min
    x = torch.full((6, 5000), -inf, device="cuda", dtype=dtype)
    x[1, 4321] = -3.0                                          # a single token
    x[2, [7, 4999]] = inf                                      # +inf takes all mass, the others none
    x[2, 8] = 100.0
    x[3] = nan
    x[3, 11] = 0.0
    x[4] = low                                                 # a mask of the type's lowest value
    x[4, 3000] = 5.0
    x[5] = low
    ids, logp = run(x, [0.5, 0.999, 0.75, 0.3, 0.9999, 0.5], [1.0, 0.7, 1.0, 1.0, 0.5, 1.0])
    assert ids.tolist() == [-1, 4321, 4999, 11, 3000, 2500]
    assert logp[0] == -np.inf and logp[1] == 0 and abs(logp[2] + np.log(2)) < 1e-6 and logp[3] == 0 and logp[4] == 0
    assert run(x, [0.5] * 6, [0.0] * 6)[0].tolist() == [-1, 4321, 7, 11, 3000, 0]
    for kw in (dict(top_k=[2] * 6), dict(top_p=[0.5] * 6), dict(min_p=[0.5] * 6)):
        assert run(x, [0.1] * 6, **kw)[0].tolist()[:5] == [-1, 4321, 7, 11, 3000]


def test_uniform_numbers_at_the_ends_and_odd_parameters():
    x = torch.tensor([[1.0, 2.0, 0.5, 2.0]] * 8, device="cuda")
    ids, _ = run(x, [0.0, 0.99999994, 1.0, 2.0, -1.0, float("nan"), 0.5, 0.5], None, None, None, None)
    assert ids.tolist()[:6] == [0, 3, 3, 3, 0, 0]
    ids, _ = run(x, [0.0] * 8, [float("inf"), float("nan"), -1.0, 1e-30, 1.0, 1.0, 1.0, 1.0], [0, 0, 0, 0, -3, 9, 1, 0],
                 [1.0, 1.0, 1.0, 1.0, 1.0, 1.0, 1.0, float("nan")], [0.0, 0.0, 0.0, 0.0, 0.0, 0.0, 2.0, float("nan")])
    assert ids.tolist() == [0, 1, 1, 1, 0, 0, 1, 0]
    assert run(x, [0.6] * 8, None, None, [0.0] * 8)[0].tolist() == [1] * 8          # top_p 0 keeps the first


def test_frequencies_of_a_thousand_draws():
    w = torch.tensor([0.1, 0.4, 0.1, 0.3, 0.1], device="cuda")
    x = w.log().expand(1000, 5).contiguous()
    ids, _ = run(x, [(i + 0.5) / 1000 for i in range(1000)])
    assert np.bincount(ids).tolist() == [100, 400, 100, 300, 100]


def test_refusals():
    x = torch.zeros(2, 8, device="cuda")
    ids, u = torch.zeros(2, dtype=torch.int32, device="cuda"), torch.zeros(2, device="cuda")
    with pytest.raises(ValueError):
        moe.moe_sample(x.half(), u, ids)
    with pytest.raises(ValueError):
        moe.moe_sample(x, u[:1], ids)
    with pytest.raises(ValueError):
        moe.moe_sample(x.t(), u, ids)
    with pytest.raises(ValueError):
        moe.moe_sample(x, u, ids.long())
    f = moe._lib.moe_sample
    st = torch.cuda.current_stream().cuda_stream

    def raw(logits=x.data_ptr(), dtype=moe.MOE_F32, rows=2, vocab=8, stride=8, u_=u.data_ptr(), ids_=ids.data_ptr()):
        return f(logits, dtype, rows, vocab, stride, None, None, None, None, u_, ids_, None, st)
    assert raw() == moe.MOE_OK and raw(rows=0) == moe.MOE_OK
    for kw in (dict(logits=None), dict(logits=x.data_ptr() + 2), dict(dtype=moe.MOE_FP8_E4M3_B128), dict(rows=-1), dict(vocab=0),
               dict(vocab=327681, stride=327681), dict(stride=7), dict(u_=None), dict(ids_=None), dict(ids_=ids.data_ptr() + 1)):
        assert raw(**kw) == moe.MOE_ERR_INVALID, kw
