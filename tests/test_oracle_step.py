"""The 64-bit oracles of the residual norms, 4-bit projections and token scores, against closed forms and torch."""
import numpy as np
import pytest
import torch

import expert_offload_slot_gb300 as moe
from oracle import step as oracle


def test_residual_norm_by_hand():
    # mean squares 12.5 and, after 0.5 * 2 * (3, 4) / sqrt(12.5) * (1 + w), read off directly
    r, y, size = oracle.residual_norm([[3.0, 4.0]], [[1.0, -1.0]], post=np.array([0.0, 1.0]), pre=None,
                                      gate=np.array([[2.0]]), scale=0.5, eps=0.0, offset=1.0)
    n = np.array([3.0, 8.0]) / np.sqrt(12.5)
    assert np.allclose(r, [1.0 + n[0], -1.0 + n[1]], rtol=1e-15) and np.allclose(size, [[1.0 + n[0], 1.0 + n[1]]])
    assert np.allclose((y * y).mean(), 1.0)
    assert np.array_equal(oracle.residual_norm(None, [[2.0, 2.0]], eps=0.0)[1], [[1.0, 1.0]])
    half = oracle.residual_norm([[4.0, 8.0]], [[0.0, 0.0]], gate=np.zeros((1, 2)), sigmoid=True)[0]
    assert np.array_equal(half, [[2.0, 4.0]])


@pytest.mark.parametrize("k, group", [(32, 32), (96, 64), (128, 128), (160, 128), (416, 32)])
def test_packing_is_within_half_a_step_and_follows_the_records_codec(k, group):
    rng = np.random.default_rng(k + group)
    w = rng.standard_normal((5, k)).astype(np.float32)
    w[2] = 0
    w[3, :32] = 0
    codes, scales = moe.moe_q4_pack(w, group)
    assert codes.shape == (5, k // 2) and scales.shape == (5, -(-k // group))
    back = oracle.unpacked(codes, scales, group)
    for g in range(scales.shape[1]):
        cols = slice(g * group, min((g + 1) * group, k))
        amax = np.abs(w[:, cols]).max(1)
        assert np.array_equal(scales[:, g], np.where(amax > 0, amax / np.float32(7), np.float32(1)))
        # half a step, and the fp32 rounding of w / scale (up to 7: 7 2^-24)
        assert (np.abs(back[:, cols] - w[:, cols]) <= scales[:, g:g + 1] * (0.5 + 7 * 2.0 ** -24)).all()
    assert not back[2].any() and np.abs(back).max() > 0


def test_packing_refusals():
    w = np.zeros((2, 64), np.float32)
    for bad, group in ((w[:, :48], 32), (w, 16), (w, 0), (np.zeros((0, 64), np.float32), 32), (w[0], 32)):
        with pytest.raises((moe.MoeError, ValueError)):
            moe.moe_q4_pack(bad, group)
    for v in (np.nan, np.inf):
        w[1, 5] = v
        with pytest.raises(moe.MoeError, match="not finite"):
            moe.moe_q4_pack(w, 32)


def test_every_code_is_read_in_its_place():
    codes = np.arange(256, dtype=np.uint8).reshape(2, 128)
    w = oracle.unpacked(codes, np.ones((2, 2)), 128)
    signed = [c - 16 if c > 7 else c for c in range(16)]
    for b in range(256):
        assert w[b // 128, 2 * (b % 128)] == signed[b % 16] and w[b // 128, 2 * (b % 128) + 1] == signed[b // 16]
    x = np.random.default_rng(0).standard_normal((3, 256))
    out, size = oracle.linear_q4(x, codes, np.ones((2, 2)), 128, np.array([1.0, -2.0]))
    assert np.allclose(out, x @ w.T + [1.0, -2.0]) and (size >= np.abs(out)).all()


def test_scores_against_torch_and_at_the_edges():
    x = torch.randn(50, dtype=torch.float64, generator=torch.Generator().manual_seed(3))
    x[7] = x[31]
    logs = torch.log_softmax(x, 0)
    lp, h, rank, ids, lps = oracle.logprobs(x.numpy(), 31, 4)
    assert abs(lp - logs[31]) < 1e-14 and abs(h + (logs.exp() * logs).sum()) < 1e-13
    assert rank == int((x > x[31]).sum()) + 1 and ids[0] == int(x.argmax()) and np.allclose(lps, logs[ids])
    inf, nan = np.inf, np.nan
    assert oracle.logprobs([-inf, nan], 1, 2) == (-inf, 0.0, 1, [-1, -1], [-inf, -inf])
    lp, h, rank, ids, lps = oracle.logprobs([inf, 3.0, inf], 2, 3)
    assert np.isclose(lp, -np.log(2)) and np.isclose(h, np.log(2)) and rank == 1 and ids == [0, 2, 1] and lps[2] == -inf
    assert oracle.logprobs([0.0, 1.0], -1, 0)[::2] == (0.0, -1, [])
