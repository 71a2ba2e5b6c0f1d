"""moe_linear_q4 where the converter warpgroups' turns go on over several tiles of an odd number of steps.

Tolerances are those of test_gpu_linear_q4.py: (52 + K / group) 2^-23 of the products' absolute sum, and half a step of
a bf16 output.
"""
import numpy as np
import pytest
import torch

import expert_offload_slot_gb300 as moe
from oracle import step as oracle

pytestmark = pytest.mark.gpu
F32, BF16 = torch.float32, torch.bfloat16


def host(t):
    return t.double().cpu().numpy()


# outputs are tiles of 256, pairs of CTAs 76; steps are of 128 inputs.  pad: rows of x off 16-byte boundaries
@pytest.mark.parametrize("dtype, rows, n, k, pad", [
    (BF16, 24, 117000, 288, 0), (BF16, 32, 60000, 384, 0), (BF16, 1, 140001, 384, 0), (BF16, 20, 60001, 896, 0), (BF16, 9, 45000, 2880, 0),
    (BF16, 40, 120001, 384, 0), (BF16, 64, 60000, 896, 0), (BF16, 110, 60000, 384, 0), (F32, 12, 117001, 288, 0),
    (BF16, 36, 117000, 384, 1)])
def test_odd_numbers_of_steps_over_several_tiles(dtype, rows, n, k, pad):
    rng = np.random.default_rng(n + k)
    group = 128
    codes = torch.from_numpy(rng.integers(0, 256, (n, k // 2), dtype=np.uint8)).cuda()
    scales = torch.from_numpy(rng.uniform(0.5, 1.5, (n, -(-k // group))).astype(np.float32)).cuda()
    x = torch.from_numpy(rng.standard_normal((rows, k + pad)).astype(np.float32)).cuda().to(dtype)[:, :k]
    out = torch.empty(rows, n, dtype=dtype, device="cuda")
    moe.moe_linear_q4(x, codes, scales, out, group=group)
    for at in range(0, n, 16384):
        ref, size = oracle.linear_q4(host(x), codes[at:at + 16384].cpu().numpy(), host(scales[at:at + 16384]), group)
        tol = (52 + k / group) * 2.0 ** -23 * size + torch.finfo(dtype).eps / 2 * np.abs(ref)
        assert (np.abs(host(out[:, at:at + 16384]) - ref) <= tol).all(), at
    again = torch.empty_like(out)
    for _ in range(5):                                         # the same sums, however the loads land
        again.fill_(7)
        moe.moe_linear_q4(x, codes, scales, again, group=group)
        assert torch.equal(again, out)
    assert moe.moe_step_status() == moe.MOE_OK
