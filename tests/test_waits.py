"""Bounded waits of a warp on a barrier: one answer in all lanes.

A warp whose lanes disagree about a wait that ran out would part where the code goes on as one (shuffles and votes
over all lanes), so the kernels that go different ways after it take the warp's common answer.
"""
import ctypes
import os
import re
import subprocess

import pytest

HERE = os.path.dirname(os.path.abspath(__file__))


def waits(name):
    """The statements of a source file that use a wait's answer, comments removed."""
    import __graft_entry__
    b = __graft_entry__._build_module()
    code = re.sub(r"//[^\n]*", "", open(os.path.join(b.CSRC, name)).read())
    return re.findall(r"(?:if|while|=|\(|!|&&|\|\|)\s*\(?!?\s*(?:\w+\s*=\s*)?(?:sm103::)?(bar_wait(?:_warp)?)\(([^,]*),", code)


def test_warps_that_part_after_a_wait_take_one_answer():
    assert waits("k_attn_rows.cu") == [("bar_wait_warp", "bar + st")]
    # of the norm + rotation kernel, the loading warp has left but for its one lane
    assert waits("k_attn_step.cu") == [("bar_wait", "empty + st"), ("bar_wait_warp", "full + st")]


@pytest.mark.gpu
def test_a_warp_has_one_answer_at_the_limit(tmp_path):
    import torch

    import __graft_entry__
    b = __graft_entry__._build_module()
    so = str(tmp_path / "wait_probe.so")
    r = subprocess.run([b._nvcc(), *b.ARCH, "-O3", "-std=c++17", "-Xcompiler", "-fPIC", "-shared", "-o", so,
                        os.path.join(HERE, "wait_probe.cu")], capture_output=True, text=True)
    assert r.returncode == 0, r.stderr
    limit = 1_000_000_000
    delays = [0, 1000, limit // 2, -1, -1] + [limit + 200 * k for k in range(-100, 100)]       # the last ones about at the limit
    delay = torch.tensor(delays, dtype=torch.int64, device="cuda")
    answer = torch.full((len(delays), 32), 7, dtype=torch.int32, device="cuda")
    torch.cuda.synchronize()
    f = ctypes.CDLL(so).wait_probe
    f.argtypes = [ctypes.c_void_p, ctypes.c_void_p, ctypes.c_int]
    assert f(delay.data_ptr(), answer.data_ptr(), len(delays)) == 0
    got = answer.cpu()
    assert (got == got[:, :1]).all() and set(got.flatten().tolist()) <= {0, 1}
    assert got[:5, 0].tolist() == [1, 1, 1, 0, 0]
