"""moe_residual_norm of the residual alone, in place: the same bits as into another tensor."""
import numpy as np
import pytest
import torch

import expert_offload_slot_gb300 as moe
from oracle import step as oracle

pytestmark = pytest.mark.gpu
TOL = 100 * 2.0 ** -24                         # of the size, as in test_gpu_residual_norm.py


def host(t):
    return t.double().cpu().numpy()


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("rows, hidden, pad", [(1, 4096, 0), (700, 2048, 0), (5000, 256, 8), (3001, 100, 0), (2500, 1024, 0), (900, 4100, 3),
                                               (400, 16384, 0), (1200, 777, 1), (3, 16383, 1)])
def test_the_norm_alone_in_place(dtype, rows, hidden, pad):
    gen = torch.Generator("cuda").manual_seed(rows)
    wide = (3 * torch.randn(rows, hidden + pad, generator=gen, device="cuda")).to(dtype)
    r = wide[:, :hidden]
    w = (1 + 0.1 * torch.randn(hidden, generator=gen, device="cuda")).to(dtype)
    for weight in (w, None):
        before = wide.clone()
        y = torch.full((rows, hidden), 7.0, dtype=dtype, device="cuda")
        moe.moe_residual_norm(None, r, None, y, pre_weight=weight)
        ref = oracle.residual_norm(None, host(r), pre=None if weight is None else host(weight))[1]
        assert (np.abs(host(y) - ref) <= (2 * TOL + torch.finfo(dtype).eps / 2) * np.abs(ref)).all()
        assert torch.equal(wide, before)
        moe.moe_residual_norm(None, r, None, r, pre_weight=weight)
        assert torch.equal(r, y) and torch.equal(wide[:, hidden:], before[:, hidden:])
