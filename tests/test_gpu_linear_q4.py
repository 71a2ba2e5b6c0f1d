"""moe_linear_q4 against the 64-bit oracle.

Codes are exact in bf16 and so are the products with bf16 inputs (an fp32 input is three of them), so
the error is that of the fp32 sums.  A tensor core adds 16 or more products to its accumulator at a time and may
cut off what lies below the largest one's last bit: 4 2^-23 of the sum of absolute products each time,
8 times at most in a group; the groups' sums are added one after another (rounded at most 1 + K / group
times, the scaling included) and up to 16 parts joined: (32 + K / group + 16 + 4) 2^-23 of the
products' absolute sum.  Outputs in bf16 are off by half a step more.
"""
import numpy as np
import pytest
import torch

import expert_offload_slot_gb300 as moe
from oracle import step as oracle

pytestmark = pytest.mark.gpu
F32, BF16 = torch.float32, torch.bfloat16


def host(t):
    return None if t is None else t.double().cpu().numpy()


def weights(rng, n, k, group, scale_type):
    codes = torch.from_numpy(rng.integers(0, 256, (n, k // 2), dtype=np.uint8)).cuda()
    scales = torch.from_numpy(rng.uniform(0.5, 1.5, (n, -(-k // group))).astype(np.float32)).cuda().to(scale_type)
    return codes, scales


def inputs(rng, rows, k, dtype, pad=0):
    return torch.from_numpy(rng.standard_normal((rows, k + pad)).astype(np.float32)).cuda().to(dtype)[:, :k]


def check(x, codes, scales, group, bias=None, out_type=None, pad=0):
    rows, n, k = x.shape[0], codes.shape[0], x.shape[1]
    wide = torch.full((rows, n + pad), 77.0, dtype=out_type or x.dtype, device="cuda")
    out = wide[:, :n]
    moe.moe_linear_q4(x, codes, scales, out, group=group, bias=bias)
    ref, size = oracle.linear_q4(host(x), codes.cpu().numpy(), host(scales), group, host(bias))
    tol = (52 + k / group) * 2.0 ** -23 * size + torch.finfo(out.dtype).eps / 2 * np.abs(ref)
    worst = (np.abs(host(out) - ref) - tol).max()
    assert worst <= 0, (worst, rows, n, k)
    assert (wide[:, n:] == 77).all()
    return out


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("group", [32, 64, 128])
@pytest.mark.parametrize("rows, n, k", [(1, 1, 32), (1, 16, 128), (1, 17, 160), (2, 100, 96), (3, 333, 1120), (5, 64, 2048), (8, 15, 416),
                                        (9, 129, 512), (10, 31, 4096), (16, 200, 2016), (17, 2000, 256), (31, 48, 64), (33, 260, 544),
                                        (64, 130, 1056), (100, 257, 800), (129, 384, 1152), (40, 1, 256),
                                        (300, 77, 608), (90, 120, 2048)])
def test_sizes(dtype, group, rows, n, k):
    rng = np.random.default_rng(rows * n + k)
    for scale_type, out_type, pad in ((F32, None, 0), (BF16, F32, 3)):
        codes, scales = weights(rng, n, k, group, scale_type)
        x = inputs(rng, rows, k, dtype, pad)
        bias = inputs(rng, 1, n, dtype)[0].contiguous() if pad else None
        check(x, codes, scales, group, bias, out_type, pad)


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("rows, n, k", [(1, 40, 16384), (3, 24, 65536), (12, 33, 16416), (40, 20, 30016), (1, 20011, 512), (2, 5000, 2048)])
def test_long_inputs_and_many_outputs(dtype, rows, n, k):
    rng = np.random.default_rng(k + n)
    codes, scales = weights(rng, n, k, 128, F32)
    check(inputs(rng, rows, k, dtype), codes, scales, 128)


@pytest.mark.parametrize("dtype, rows, n, k, pad", [(BF16, 24, 40000, 512, 0), (BF16, 3, 39000, 1184, 0), (BF16, 300, 12100, 640, 0),
                                                    (BF16, 70, 24000, 928, 8), (F32, 100, 20100, 384, 0), (F32, 12, 39937, 256, 1),
                                                    (BF16, 40, 23000, 352, 1), (BF16, 100, 40001, 384, 0), (BF16, 128, 60000, 1664, 0),
                                                    (BF16, 50, 60000, 640, 0), (BF16, 18, 80000, 288, 0), (BF16, 600, 20000, 896, 0),
                                                    (F32, 84, 19300, 384, 0), (F32, 170, 20000, 288, 0), (BF16, 200, 19300, 352, 1)])
def test_several_tiles_for_each_pair_of_ctas(dtype, rows, n, k, pad):
    rng = np.random.default_rng(n)
    for group in (128, 32):
        codes, scales = weights(rng, n, k, group, F32)
        check(inputs(rng, rows, k, dtype, pad), codes, scales, group, pad=5)


@pytest.mark.parametrize("rows", [1, 40, 200])
def test_every_code_and_input_is_in_its_place(rows):
    """One input at a time is 1: the outputs are its weights, exactly."""
    n, k, group = 130, 320, 64
    rng = np.random.default_rng(rows)
    codes, scales = weights(rng, n, k, group, BF16)
    w = oracle.unpacked(codes.cpu().numpy(), host(scales), group)
    for dtype in (F32, BF16):
        for k0 in range(0, k, rows):
            x = torch.zeros(rows, k, device="cuda", dtype=dtype)
            m = min(rows, k - k0)
            x[torch.arange(m), torch.arange(k0, k0 + m)] = 1
            out = torch.empty(rows, n, device="cuda")
            moe.moe_linear_q4(x, codes, scales, out, group=group)
            assert np.array_equal(host(out)[:m], w[:, k0:k0 + m].T) and not out[m:].any()
            if rows == 1 and k0 > 140:
                break


def test_fp32_inputs_keep_their_bits():
    """fp32 inputs over a wide range of magnitudes, one product an output: exact up to one rounding."""
    k, n = 64, 64
    rng = np.random.default_rng(1)
    x = torch.from_numpy((rng.standard_normal(n) * 10.0 ** rng.uniform(-28, 30, n)).astype(np.float32)).cuda()
    codes = torch.full((n, k // 2), 0x77, dtype=torch.uint8, device="cuda")
    out = torch.empty(n, n, device="cuda")
    moe.moe_linear_q4(torch.diag(x).contiguous(), codes, torch.ones(n, 1, device="cuda"), out, group=64)
    want = 7 * host(x)
    assert (np.abs(host(out) - want[:, None]) <= 2.0 ** -23 * np.abs(want)[:, None]).all()


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("rows", [1, 6, 70])
def test_infinities_and_nan_stay_in_their_rows(dtype, rows):
    n, k = 50, 256
    rng = np.random.default_rng(9)
    codes, scales = weights(rng, n, k, 128, F32)
    codes.fill_(0x11)                                          # weights of one sign
    x = inputs(rng, rows, k, dtype).contiguous()
    clean = torch.empty(rows, n, device="cuda")
    moe.moe_linear_q4(x, codes, scales, clean)
    for v in (float("inf"), float("-inf"), float("nan")):
        bad = x.clone()
        bad[rows // 2, 77] = v
        out = torch.empty(rows, n, device="cuda")
        moe.moe_linear_q4(bad, codes, scales, out)
        keep = torch.arange(rows, device="cuda") != rows // 2
        assert torch.equal(out[keep], clean[keep])
        assert out[rows // 2].isnan().all() if v != v else (out[rows // 2] == v).all()


def test_the_same_call_gives_the_same_bits_also_in_a_graph():
    rng = np.random.default_rng(4)
    for rows in (1, 20, 150):
        codes, scales = weights(rng, 700, 1056, 32, F32)
        x = inputs(rng, rows, 1056, BF16)
        out = check(x, codes, scales, 32)
        again = torch.empty_like(out)
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=torch.cuda.Stream()):
            moe.moe_linear_q4(x, codes, scales, again, group=32)
        for _ in range(3):
            again.fill_(0)
            graph.replay()
            assert torch.equal(again, out)
