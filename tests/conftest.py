import os
import sys

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
if ROOT not in sys.path:
    sys.path.insert(0, ROOT)


def pytest_configure(config):
    config.addinivalue_line("markers", "gpu: needs a CUDA GPU (GB300, sm_103a) and the built libmoeslot.so")


def pytest_collection_modifyitems(config, items):
    try:
        import torch
        have_gpu = torch.cuda.is_available()
    except Exception:  # pragma: no cover
        have_gpu = False
    if have_gpu:
        return
    skip = pytest.mark.skip(reason="no CUDA device in this process")
    for item in items:
        if "gpu" in item.keywords:
            item.add_marker(skip)


@pytest.fixture(autouse=True)
def projections_end(request):
    """4-bit projections report a wait that ran out in a status of the device alone: read after each test that makes them."""
    yield
    if "gpu" in request.node.keywords and request.module.__name__.split(".")[-1] in (
            "test_gpu_linear_q4", "test_gpu_linear_q4_turns", "test_gpu_generate_q4", "test_gpu_step"):
        import expert_offload_slot_gb300 as moe
        assert moe.moe_step_status() == moe.MOE_OK
