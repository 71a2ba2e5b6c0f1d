"""moe_logprobs against the 64-bit oracle.

Ranks and tokens are exact.  An exponential's argument is off by 2^-24 of itself, where it counts (down to about -24:
e below 2^-24 is lost anyway); the exponential by 2^-22; a thread adds up vocab / 256 of them one after another, the
rest is a tree: (24 + 4 + vocab / 256 + 24) 2^-24 relative.  The logarithm, the difference of two numbers of opposite
signs and the product round three times: 2^-22 of |logp| or the entropy.
"""
import numpy as np
import pytest
import torch

import expert_offload_slot_gb300 as moe
from oracle import step as oracle

pytestmark = pytest.mark.gpu


def run(x, target, top=5):
    rows = x.shape[0]
    dev = dict(device="cuda")
    out = {"logp": torch.full((rows,), 9.0, **dev), "entropy": torch.full((rows,), 9.0, **dev),
           "rank": torch.full((rows,), -9, dtype=torch.int32, **dev),
           "top_ids": torch.full((rows, top), -9, dtype=torch.int32, **dev), "top_logp": torch.full((rows, top), 9.0, **dev)}
    moe.moe_logprobs(x, torch.as_tensor(target, dtype=torch.int32, **dev), **out)
    return {k: v.cpu().numpy() for k, v in out.items()}


def close(got, want, tol):
    got, want = np.asarray(got, np.float64), np.asarray(want, np.float64)
    same = got == want
    with np.errstate(invalid="ignore"):
        assert (same | (np.abs(got - want) <= tol + 2.0 ** -22 * np.abs(want))).all(), (got, want)


def check(x, target, top=5):
    got = run(x, target, top)
    host = x.double().cpu().numpy()
    for r in range(x.shape[0]):
        tol = (52 + x.shape[1] / 256) * 2.0 ** -24
        lp, h, rank, ids, lps = oracle.logprobs(host[r], int(target[r]), top)
        assert got["rank"][r] == rank and got["top_ids"][r].tolist() == ids, r
        close(got["logp"][r], lp, tol)
        close(got["entropy"][r], h, 24 * tol)                  # its terms are the logs, up to 24, times p
        close(got["top_logp"][r], lps, tol)
    return got


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("vocab", [1, 2, 7, 33, 100, 257, 1000, 4097, 8191, 32771, 100277, 327680])
def test_rows_against_the_oracle(dtype, vocab):
    gen = torch.Generator("cuda").manual_seed(vocab)
    rows = 12 if vocab < 50000 else 4
    wide = torch.randn(rows, vocab + 5, generator=gen, device="cuda")
    wide *= torch.linspace(0.1, 6, rows, device="cuda")[:, None]
    rng = np.random.default_rng(vocab)
    for shift in (0, 3):
        x = wide.to(dtype)[:, shift:shift + vocab]             # rows at odd offsets
        target = rng.integers(0, vocab, rows)
        target[0], target[-1] = 0, vocab - 1
        target[1] = int(x[1].float().argmax())
        for top in (0, 5, 32):
            check(x, target, top)


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("rows, vocab", [(1, 131072), (3, 50257), (20, 9000), (40, 8192), (77, 4100), (160, 2000), (333, 9000), (700, 600)])
def test_numbers_of_rows(dtype, rows, vocab):
    gen = torch.Generator("cuda").manual_seed(rows)
    x = (3 * torch.randn(rows, vocab, generator=gen, device="cuda")).to(dtype)
    check(x, np.random.default_rng(rows).integers(-1, vocab, rows), 20)


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("vocab", [40, 5000, 60000])
def test_ties(dtype, vocab):
    gen = torch.Generator("cuda").manual_seed(vocab)
    x = torch.zeros(6, vocab, device="cuda")
    x[1] = torch.randint(0, 3, (vocab,), generator=gen, device="cuda").float()
    x[2] = torch.arange(vocab, device="cuda").float() / vocab
    x[3] = -x[2]
    x[4, ::7] = 1.0
    x[5, vocab // 2:] = -0.0
    for where in (0, vocab // 3, vocab - 1):
        check(x.to(dtype), [where] * 6, 32)


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("vocab", [50, 5000, 50001])
def test_infinities_nan_and_masks(dtype, vocab):
    inf, nan, low = float("inf"), float("nan"), torch.finfo(dtype).min
    x = torch.full((9, vocab), -inf, device="cuda", dtype=dtype)
    x[1, 43] = -3.0                                            # a single token
    x[2, [7, 49]] = inf                                        # +inf takes all mass
    x[2, 8] = 100.0
    x[3] = nan
    x[3, [11, 12]] = 0.5
    x[4] = low                                                 # a mask of the type's lowest value
    x[4, 30] = 5.0
    x[5] = low
    x[6] = torch.randn(vocab, device="cuda", generator=torch.Generator("cuda").manual_seed(2)).to(dtype)
    x[6, ::3], x[6, 1::9] = -inf, nan
    x[7] = 1e30                                                # far from zero
    x[7, 5] = 1.01e30
    x[8, :20] = torch.linspace(3e5, 3.001e5, 20, device="cuda").to(dtype)
    for target in ([0] * 9, [43, 43, 7, 11, 30, 49, 2, 5, 3], [8, 42, 8, 12, 31, 0, 1, 6, 30], [-1, -100, vocab, 2 ** 31 - 1] + [45] * 5):
        check(x, target, 5)
        check(x, target, 32)


def test_peaked_rows():
    x = torch.zeros(3, 30000, device="cuda")
    x[0, 9], x[1, 9], x[2, 9] = 12.0, 25.0, 60.0
    got = check(x, [9, 9, 9])
    # the maximum's own exponential is 2^r, r the rounding of 60 log2(e) to 24 bits, at most 2^-18.  With s = 2^r (1 + a),
    # |a| <= 2^-22 of the exponential, log2 s = r + 1.45 a, rounded by 2^-42 (r is that small) and by the logarithm's
    # 2^-22 where s is within 2^-17 of 1: logp = r - log2 s is off by 1.45 2^-22 + 2^-22, times log(2): below 2^-21
    assert (got["logp"] <= 0).all() and (got["entropy"] >= 0).all() and got["logp"][2] >= -2.0 ** -21


def test_optional_outputs_and_a_captured_call():
    x = torch.randn(4, 20000, device="cuda")
    t = torch.tensor([1, 2, 3, -1], dtype=torch.int32, device="cuda")
    full = run(x, t.cpu(), 3)
    logp, ids, lps = torch.empty(4, device="cuda"), torch.empty(4, 3, dtype=torch.int32, device="cuda"), torch.empty(4, 3, device="cuda")
    moe.moe_logprobs(x, t, logp)
    assert np.array_equal(logp.cpu().numpy(), full["logp"])
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=torch.cuda.Stream()):
        moe.moe_logprobs(x, t, logp, top_ids=ids, top_logp=lps)
    for seed in (1, 2):
        x.copy_(torch.randn(4, 20000, generator=torch.Generator().manual_seed(seed)))
        graph.replay()
        full = run(x, t.cpu(), 3)
        assert np.array_equal(logp.cpu().numpy(), full["logp"]) and np.array_equal(ids.cpu().numpy(), full["top_ids"])
        assert np.array_equal(lps.cpu().numpy(), full["top_logp"])
