"""The host side of the attention calls, without a GPU: argument checks and the device each call selects.

csrc/attn_api.cu is linked with stand-ins for the CUDA runtime (two devices) and for the kernels' launchers
(tests/attn_host_stub.cpp, .cu), which log what was called and which device was current.
"""
import ctypes
import os
import subprocess

import pytest

import expert_offload_slot_gb300 as moe

HERE = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(HERE)


@pytest.fixture(scope="module")
def lib(tmp_path_factory):
    import __graft_entry__
    b = __graft_entry__._build_module()
    out = tmp_path_factory.mktemp("attn_host")
    so = str(out / "libattn_host.so")
    cmd = [b._nvcc(), *b.ARCH, "-O1", "-std=c++17", "-Xcompiler", "-fPIC,-fvisibility=hidden", f"-I{b.INCLUDE}", "-shared",
           "-cudart", "none", "-Xlinker", "-Bsymbolic", "-o", so, os.path.join(b.CSRC, "attn_api.cu"),
           os.path.join(HERE, "attn_host_stub.cu"), os.path.join(HERE, "attn_host_stub.cpp")]
    r = subprocess.run(cmd, capture_output=True, text=True)
    assert r.returncode == 0, r.stderr
    so = ctypes.CDLL(so)
    for name in moe.EXPORTED:
        if hasattr(so, name):
            f = getattr(so, name)
            f.restype, f.argtypes = moe._sig[name]
    so.stub_log.restype = so.stub_error.restype = ctypes.c_char_p
    return so


def create(lib, device, dtype=moe.MOE_BF16):
    h = ctypes.c_void_p()
    cfg = moe.make_attn_config(8, 2, 128, 16, dtype)
    assert lib.moe_attn_create(ctypes.byref(cfg), device, ctypes.byref(h)) == moe.MOE_OK, lib.stub_error()
    return h


def called(lib, f, *args):
    lib.stub_clear()
    assert f(*args) == moe.MOE_OK, lib.stub_error()
    return lib.stub_log().decode().split()


P, Q = 1 << 12, 1 << 13                    # addresses: aligned, never read


def forward(lib, h, max_new, stream=None):
    return called(lib, lib.moe_attn_forward, h, P, 1024, 64, P, P, 1, max_new, P, P, 9, P, 4, P, stream)


@pytest.mark.parametrize("other", [0, 1])
def test_calls_run_on_their_handles_device_and_leave_the_threads(lib, other):
    for device in (0, 1):
        lib.stub_set_device(other)
        lib.stub_clear()
        h, h32 = create(lib, device), create(lib, device, moe.MOE_F32)
        log = lib.stub_log().decode().split()
        assert log and all(f"@{device}/" in e for e in log) and lib.stub_device() == other
        for stream in (None, 64):          # the default stream belongs to the current device
            at = f"@{device}/{stream or 0}"
            assert called(lib, lib.moe_attn_tables, h, P, P, 1, P, 4, P, 3, P, P, 8, Q, Q, P, P, stream) == ["tables" + at]
            assert called(lib, lib.moe_attn_qkv, h, P, 1536, 8, P, P, P, 9, P, P, P, P, P, 9, stream) == ["qkv" + at]
            assert forward(lib, h, 1, stream) == ["rows" + at]
            assert forward(lib, h, 64, stream) == ["tiles" + at]
            assert forward(lib, h32, 1, stream) == ["f32" + at]
            assert lib.stub_device() == other
        for f in (lib.moe_attn_get_status, lib.moe_attn_clear_status, lib.moe_attn_destroy):
            log = called(lib, f, h)
            assert log and all(f"@{device}/" in e for e in log) and lib.stub_device() == other
        lib.moe_attn_destroy(h32)
    lib.stub_set_device(0)


def test_a_device_that_is_not_there_is_refused(lib):
    h, cfg = ctypes.c_void_p(), moe.make_attn_config(8, 2, 128, 16)
    for device in (-1, 2):
        assert lib.moe_attn_create(ctypes.byref(cfg), device, ctypes.byref(h)) == moe.MOE_ERR_INVALID and not h
    assert lib.stub_device() == 0
