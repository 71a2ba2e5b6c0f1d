"""moe_residual_norm against the 64-bit oracle.

In fp32 a sum of squares of up to 16384 numbers goes through at most 16 + 10 + 32 additions, 58 2^-24
relative, half of it after the root; the root, the division and the products round up to eight
times more: 40 2^-24 of what an element adds up (|r| + |scale gate n|), which the second norm scales
as it scales the element.  The first norm's error (40 2^-24 again) is in the sum.  A sigmoid: exp
2 2^-24, sum, division.  Together 100 2^-24 of the size.  Outputs in bf16 are off by half a step more.
"""
import numpy as np
import pytest
import torch

import expert_offload_slot_gb300 as moe
from oracle import step as oracle

pytestmark = pytest.mark.gpu
F32, BF16 = torch.float32, torch.bfloat16
TOL = 100 * 2.0 ** -24


def host(t):
    return None if t is None else t.double().cpu().numpy()


def rows_of(gen, rows, hidden, dtype, pad, scale):
    return (scale * torch.randn(rows, hidden + pad, generator=gen, device="cuda")).to(dtype)[:, :hidden]


def check(x, residual, post, pre, gate, sigmoid=False, scale=1.0, eps=1e-6, offset=0.0, pad=0, inplace=False):
    dtype, (rows, hidden) = (residual if x is None else x).dtype, residual.shape
    ref, ref_y, size = oracle.residual_norm(host(x), host(residual), host(post), host(pre), host(gate), sigmoid, scale, eps, offset)
    wide = torch.full((rows, hidden + pad), 7.0, dtype=residual.dtype, device="cuda")
    wide_y = torch.full((rows, hidden + pad), 7.0, dtype=dtype, device="cuda")
    out, y = wide[:, :hidden], wide_y[:, :hidden]
    if inplace:
        out, y = residual, x
    moe.moe_residual_norm(x, residual, None if x is None else out, y, post, pre, gate, sigmoid, scale, eps, offset)
    half = lambda t: torch.finfo(t).eps / 2  # noqa: E731
    if x is not None:
        assert (np.abs(host(out) - ref) <= TOL * size + half(out.dtype) * np.abs(ref)).all()
    per = np.abs(ref_y) / np.where(ref == 0, 1, np.abs(ref))
    per = np.where(ref == 0, per.max(1, keepdims=True), per)
    assert (np.abs(host(y) - ref_y) <= TOL * size * per + half(dtype) * np.abs(ref_y) + TOL * np.abs(ref_y)).all()
    if pad and not inplace:
        assert (wide_y[:, hidden:] == 7).all() and (wide[:, hidden:] == 7).all()


@pytest.mark.parametrize("types", [(F32, F32), (BF16, BF16), (BF16, F32)])
@pytest.mark.parametrize("hidden", [1, 2, 7, 8, 31, 128, 130, 256, 264, 511, 1537, 2048, 2056, 4095, 4104, 7168, 8192, 8200, 9001, 16383, 16384])
def test_widths(types, hidden):
    gen = torch.Generator("cuda").manual_seed(hidden)
    dtype, stream = types
    rows = 5 if hidden < 9000 else 2
    weight = lambda: (1 + 0.2 * torch.randn(hidden, generator=gen, device="cuda")).to(dtype)  # noqa: E731
    for pad in (0, 3, 8):
        x, r = rows_of(gen, rows, hidden, dtype, pad, 1.5), rows_of(gen, rows, hidden, stream, pad, 5.0)
        gate = torch.randn(hidden, generator=gen, device="cuda").to(dtype)
        check(x, r, weight(), weight(), gate, pad == 3, 0.37, 1e-6, float(pad == 8), pad)
        check(x, r, None, weight(), None, pad=pad)


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("gate", ["none", "row", "channel", "element"])
@pytest.mark.parametrize("hidden", [200, 77])
def test_gates_weights_and_missing_parts(dtype, gate, hidden):
    gen = torch.Generator("cuda").manual_seed(5)
    rows = 9
    x, r = rows_of(gen, rows, hidden, dtype, 0, 2.0), rows_of(gen, rows, hidden, dtype, 0, 3.0)
    g = {"none": None, "row": rows_of(gen, rows, 1, dtype, 4, 1.0), "channel": rows_of(gen, 1, hidden, dtype, 0, 1.0)[0],
         "element": rows_of(gen, rows, hidden, dtype, 8, 1.0)}[gate]
    w = rows_of(gen, 2, hidden, dtype, 0, 1.0)
    for post in (None, w[0]):
        for pre in (None, w[1].contiguous()):
            for sigmoid in (False, True):
                check(x, r, post, pre, g, sigmoid, 0.5, 1e-5, 1.0)
    check(None, r, None, w[0], None)                           # a step's first norm
    out = torch.full_like(r, 7.0)                              # no next norm
    moe.moe_residual_norm(x, r, out, None, gate=g, residual_scale=-2.0)
    ref, _, size = oracle.residual_norm(host(x), host(r), gate=host(g), scale=-2.0)
    assert (np.abs(host(out) - ref) <= TOL * size + torch.finfo(dtype).eps / 2 * np.abs(ref)).all()


@pytest.mark.parametrize("types", [(F32, F32), (BF16, BF16), (BF16, F32)])
@pytest.mark.parametrize("rows, hidden", [(1, 4096), (700, 2048), (5000, 256), (3001, 100), (2500, 1024), (900, 4100)])
def test_in_place_and_many_rows(types, rows, hidden):
    gen = torch.Generator("cuda").manual_seed(rows)
    x, r = rows_of(gen, rows, hidden, types[0], 0, 1.0), rows_of(gen, rows, hidden, types[1], 0, 4.0)
    w = (1 + 0.1 * torch.randn(hidden, generator=gen, device="cuda")).to(types[0])
    copies = x.clone(), r.clone()
    out, y = torch.empty_like(r), torch.empty_like(x)
    moe.moe_residual_norm(x, r, out, y, w, w)
    check(x, r, w, w, None, inplace=True)
    assert torch.equal(x, y) and torch.equal(r, out)           # the same bits in place
    moe.moe_residual_norm(None, copies[0], None, copies[0], pre_weight=w)        # the norm alone, in place
    assert torch.isfinite(copies[0].float()).all()


def test_zeros_infinities_and_nan_stay_in_their_rows():
    inf, nan = float("inf"), float("nan")
    for dtype in (F32, BF16):
        x, r = torch.ones(5, 64, device="cuda", dtype=dtype), torch.ones(5, 64, device="cuda", dtype=dtype)
        x[1, 3], r[2, 5], x[3, 0] = nan, inf, -inf
        x[4], r[4] = 0, 0
        out, y = torch.empty_like(r), torch.empty_like(x)
        moe.moe_residual_norm(x, r, out, y)
        assert torch.allclose(y[0].float(), torch.ones(64, device="cuda"), atol=1e-2) and (out[0] == 2).all()
        assert y[1].isnan().all() and out[1].isnan().sum() == 1
        assert y[2, 5].isnan() and (y[2, :5] == 0).all() and out[2, 5] == inf and out[3, 0] == -inf
        assert (y[4] == 0).all() and (out[4] == 0).all()


def test_captured_calls_replay_on_new_inputs():
    x, r = torch.randn(3, 512, device="cuda"), torch.randn(3, 512, device="cuda")
    out, y = torch.empty_like(r), torch.empty_like(x)
    side = torch.cuda.Stream()
    moe.moe_residual_norm(x, r, out, y, gate=x[:, :1])
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        moe.moe_residual_norm(x, r, out, y, gate=x[:, :1])
        moe.moe_residual_norm(y, out, out, y, pre_weight=r[0])
    for seed in (1, 2):
        x.copy_(torch.randn(3, 512, generator=torch.Generator().manual_seed(seed)))
        graph.replay()
        first, f_y = torch.empty_like(r), torch.empty_like(x)
        moe.moe_residual_norm(x, r, first, f_y, gate=x[:, :1])
        moe.moe_residual_norm(f_y, first, first, f_y, pre_weight=r[0])
        assert torch.equal(first, out) and torch.equal(f_y, y)
