"""moe_residual_norm, moe_linear_q4 and moe_logprobs without a GPU: refusals of the library and the binding's checks.

The library refuses before anything is launched; addresses are never read.  The binding is called with tensors that
only say where they are, and with a stand-in for the library.
"""
import ctypes
import types

import pytest
import torch

import expert_offload_slot_gb300 as moe
from tests.test_attn_binding import On, calls  # noqa: F401

P = 1 << 20
F32, BF16, I32, U8 = torch.float32, torch.bfloat16, torch.int32, torch.uint8


def norm(cfg=(), **kw):
    c = dict(hidden=64, dtype=moe.MOE_BF16, residual_dtype=moe.MOE_F32, gate=0, gate_sigmoid=0, residual_scale=1.0, norm_eps=1e-6,
             weight_offset=0.0)
    c.update(cfg)
    c = moe.moe_norm_config(*c.values())
    a = dict(x=P, x_stride=64, gate=None, gate_stride=0, post=None, residual=P, residual_stride=64, out=P, out_stride=64, pre=None,
             y=P, y_stride=64, rows=2, stream=None)
    a.update(kw)
    return moe._lib.moe_residual_norm(ctypes.byref(c), *a.values())


def linear(**kw):
    a = dict(x=P, dtype=moe.MOE_BF16, x_stride=64, rows=2, k=64, codes=P, scales=P, scale_dtype=moe.MOE_F32, group=32, bias=None, n=10,
             out=P, out_dtype=moe.MOE_BF16, out_stride=10, stream=None)
    a.update(kw)
    return moe._lib.moe_linear_q4(*a.values())


def logprobs(**kw):
    a = dict(logits=P, dtype=moe.MOE_BF16, rows=2, vocab=50, stride=50, targets=P, top=3, logp=P, entropy=P, rank=P, ids=P, lps=P,
             stream=None)
    a.update(kw)
    return moe._lib.moe_logprobs(*a.values())


@pytest.mark.parametrize("cfg, kw", [
    ({}, dict(rows=-1)), ({}, dict(rows=moe.MOE_ATTN_MAX_ROWS + 1)), (dict(hidden=0), {}), (dict(hidden=16385), {}), (dict(dtype=2), {}),
    (dict(dtype=0, residual_dtype=1), {}), (dict(residual_dtype=3), {}), (dict(gate=4), dict(gate=P)), (dict(gate=-1), {}),
    (dict(gate=1), {}), (dict(gate=1), dict(gate=P)), (dict(gate=3), dict(gate=P, gate_stride=63)), (dict(gate_sigmoid=2), {}),
    (dict(norm_eps=-1.0), {}), (dict(norm_eps=float("nan")), {}), (dict(residual_scale=float("inf")), {}),
    (dict(weight_offset=float("nan")), {}), ({}, dict(x_stride=63)), ({}, dict(residual_stride=0)), ({}, dict(out_stride=63)),
    ({}, dict(y_stride=-64)), ({}, dict(residual=None)), ({}, dict(out=None)), ({}, dict(x=None)), ({}, dict(x=None, out=None, y=None)),
    ({}, dict(x=None, out=None, post=P)), (dict(gate=2), dict(x=None, out=None, gate=P)), ({}, dict(x=P + 1)), ({}, dict(residual=P + 2)),
    ({}, dict(out=P + 2)), ({}, dict(y=P + 1)), ({}, dict(pre=P + 1)), ({}, dict(post=P + 1)), (dict(gate=2), dict(gate=P + 1))])
def test_norm_refusals(cfg, kw):
    assert norm(cfg, **kw) == moe.MOE_ERR_INVALID and moe._lib.moe_last_error()


@pytest.mark.parametrize("kw", [
    dict(rows=-1), dict(rows=moe.MOE_ATTN_MAX_ROWS + 1), dict(dtype=2), dict(scale_dtype=3), dict(out_dtype=2),
    dict(dtype=0, out_dtype=1, x_stride=64), dict(group=16), dict(group=0), dict(group=256), dict(k=0), dict(k=48), dict(k=-32),
    dict(k=65568, x_stride=65568), dict(n=0), dict(n=moe.MOE_LINEAR_MAX_OUT + 1, out_stride=1 << 21), dict(x_stride=63), dict(out_stride=9),
    dict(x=None), dict(codes=None), dict(scales=None), dict(out=None), dict(codes=P + 8), dict(x=P + 1), dict(scales=P + 2),
    dict(bias=P + 1), dict(out=P + 1), dict(out_dtype=0, out=P + 2)])
def test_linear_refusals(kw):
    assert linear(**kw) == moe.MOE_ERR_INVALID and moe._lib.moe_last_error()


@pytest.mark.parametrize("kw", [
    dict(rows=-1), dict(rows=moe.MOE_ATTN_MAX_ROWS + 1), dict(dtype=2), dict(vocab=0), dict(vocab=327681, stride=327681), dict(stride=49),
    dict(top=-1), dict(top=33), dict(logits=None), dict(targets=None), dict(logp=None), dict(ids=None), dict(lps=None),
    dict(logits=P + 1), dict(dtype=0, logits=P + 2), dict(targets=P + 2), dict(logp=P + 1), dict(entropy=P + 2), dict(rank=P + 3),
    dict(ids=P + 2), dict(lps=P + 2)])
def test_score_refusals(kw):
    assert logprobs(**kw) == moe.MOE_ERR_INVALID and moe._lib.moe_last_error()


def test_calls_without_rows_do_nothing():
    assert norm(rows=0) == linear(rows=0) == logprobs(rows=0) == moe.MOE_OK
    assert moe._lib.moe_residual_norm(None, *[0] * 14) == moe.MOE_ERR_INVALID


def arguments(place, odd=None, odd_place=0):
    """Keyword tensors of the three calls on `place`, the one called `odd` elsewhere."""
    t = lambda name, shape, dtype: On(shape, dtype, odd_place if name == odd else place)  # noqa: E731
    return {
        "moe_residual_norm": {**{n: t(n, s, BF16) for n, s in dict(x=(7, 64), y=(7, 64), post_weight=(64,), pre_weight=(64,), gate=(64,)).items()},
                              **{n: t(n, (7, 64), F32) for n in ("residual", "residual_out")}},
        "moe_linear_q4": {"x": t("x", (7, 256), BF16), "codes": t("codes", (50, 128), U8), "scales": t("scales", (50, 2), F32),
                          "out": t("out", (7, 50), F32), "bias": t("bias", (50,), BF16)},
        "moe_logprobs": {"logits": t("logits", (7, 50), BF16), **{n: t(n, (7,), I32) for n in ("targets", "rank")},
                         **{n: t(n, (7,), F32) for n in ("logp", "entropy")}, "top_ids": t("top_ids", (7, 4), I32),
                         "top_logp": t("top_logp", (7, 4), F32)},
    }


On.dim = lambda self: len(self.shape)
LEAD = {"moe_residual_norm": "residual", "moe_linear_q4": "x", "moe_logprobs": "logits"}


@pytest.mark.parametrize("device", [0, 1])
@pytest.mark.parametrize("what", list(LEAD))
def test_calls_run_on_their_tensors_device_and_its_stream(calls, what, device):  # noqa: F811
    for current in (0, 1):
        calls.state["device"] = current
        getattr(moe, what)(**arguments(device)[what])
        assert calls.seen[-1] == (what, device, 100 + device) and calls.state["device"] == current
        getattr(moe, what)(**arguments(device)[what], stream=64)
        assert calls.seen[-1] == (what, device, 64)


@pytest.mark.parametrize("device", [0, 1])
@pytest.mark.parametrize("elsewhere", ["host", "gpu"])
@pytest.mark.parametrize("what", list(LEAD))
def test_tensors_elsewhere_are_refused(calls, what, device, elsewhere):  # noqa: F811
    place = -1 if elsewhere == "host" else 1 - device
    for name in arguments(device)[what]:
        with pytest.raises(ValueError, match="must" if name == LEAD[what] else f"^{name} must"):
            getattr(moe, what)(**arguments(device, name, place)[what])
    assert not calls.seen


def test_wrong_types_and_sizes_are_refused(calls):  # noqa: F811
    def changed(what, **kw):
        a = arguments(0)[what]
        a.update(kw)
        with pytest.raises(ValueError):
            getattr(moe, what)(**a)
    for kw in (dict(x=On((7, 64), torch.float16, 0)), dict(y=On((7, 64), F32, 0)), dict(residual=On((7, 64), torch.float16, 0)),
               dict(residual_out=On((7, 64), BF16, 0)), dict(gate=On((63,), BF16, 0)), dict(gate=On((6, 1), BF16, 0)),
               dict(gate=On((7, 2), BF16, 0)), dict(pre_weight=On((65,), BF16, 0)), dict(post_weight=On((64,), F32, 0)),
               dict(x=On((8, 64), BF16, 0)), dict(x=None, y=None)):
        changed("moe_residual_norm", **kw)
    for kw in (dict(codes=On((50, 127), U8, 0)), dict(codes=On((50, 128), torch.int8, 0)), dict(scales=On((50, 4), F32, 0)),
               dict(scales=On((50, 2), torch.float16, 0)), dict(out=On((7, 49), F32, 0)), dict(out=On((7, 50), torch.float16, 0)),
               dict(bias=On((50,), F32, 0)), dict(group=48), dict(group=64)):
        changed("moe_linear_q4", **kw)
    for kw in (dict(logits=On((7, 50), torch.float16, 0)), dict(targets=On((7,), torch.int64, 0)), dict(targets=On((6,), I32, 0)),
               dict(top_ids=None), dict(top_logp=None), dict(top_logp=On((7, 5), F32, 0)), dict(top_ids=On((7, 4), torch.int64, 0)),
               dict(logp=On((7,), BF16, 0)), dict(rank=On((7,), F32, 0))):
        changed("moe_logprobs", **kw)
    assert not calls.seen


def test_strides_of_rows_are_passed_on(monkeypatch):
    seen = []
    monkeypatch.setattr(moe, "_lib", types.SimpleNamespace(moe_logprobs=lambda *a: seen.append(a) or moe.MOE_OK))
    kinds = dict(moe._torch_kinds())
    kinds.update(stream=lambda d: 5, device=lambda: 0)
    monkeypatch.setattr(moe, "_kinds", kinds)

    class Wide(On):
        def is_contiguous(self):
            return False

        def stride(self, i=None):
            return (61, 1) if i is None else (61, 1)[i]
    a = arguments(0)["moe_logprobs"]
    a["logits"] = Wide((7, 50), F32, 0)
    moe.moe_logprobs(**a)
    assert seen[0][1:5] == (moe.MOE_F32, 7, 50, 61) and seen[0][6] == 4
