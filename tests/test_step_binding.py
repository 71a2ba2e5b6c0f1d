"""Shapes that the binding of moe_residual_norm, moe_linear_q4 and moe_logprobs looks at, without a GPU."""
import ctypes
import types

import pytest
import torch

import expert_offload_slot_gb300 as moe
from tests.test_attn_binding import On, calls  # noqa: F401

F32, BF16, I32, U8 = torch.float32, torch.bfloat16, torch.int32, torch.uint8


def linear(**kw):
    a = dict(x=On((7, 256), BF16, 0), codes=On((50, 128), U8, 0), scales=On((50, 2), F32, 0), out=On((7, 50), F32, 0))
    moe.moe_linear_q4(**{**a, **kw})


def norm(**kw):
    a = {n: On((7, 64), BF16, 0) for n in ("x", "residual", "residual_out", "y")}
    moe.moe_residual_norm(**{**a, **kw})


def scores(**kw):
    a = dict(logits=On((7, 50), F32, 0), targets=On((7,), I32, 0), logp=On((7,), F32, 0), top_ids=On((7, 4), I32, 0),
             top_logp=On((7, 4), F32, 0))
    moe.moe_logprobs(**{**a, **kw})


@pytest.mark.parametrize("dtype", [F32, BF16])
def test_scales_of_another_order_are_refused(calls, dtype):  # noqa: F811
    """[groups, out], as several 4-bit formats store them, has the right count of elements."""
    with pytest.raises(ValueError, match="^scales must"):
        linear(scales=On((2, 50), dtype, 0))
    with pytest.raises(ValueError, match="^scales must"):
        linear(scales=On((2, 5, 10), dtype, 0))
    assert not calls.seen
    linear(scales=On((50, 2), dtype, 0))
    linear(scales=On((50, 2, 1), dtype, 0))
    linear(scales=On((100,), dtype, 0))
    assert len(calls.seen) == 3


def test_outputs_and_inputs_of_another_order_are_refused(calls):  # noqa: F811
    for call, name, shape, dtype in [(linear, "out", (50, 7), F32), (norm, "x", (64, 7), BF16), (norm, "residual_out", (64, 7), BF16),
                                     (norm, "y", (64, 7), BF16), (norm, "y", (8, 7, 8), BF16), (scores, "top_logp", (4, 7), F32)]:
        with pytest.raises(ValueError, match=f"^{name} must"):
            call(**{name: On(shape, dtype, 0)})
    assert not calls.seen


def test_rows_in_several_dimensions_are_taken(calls):  # noqa: F811
    linear(out=On((7, 5, 10), F32, 0))
    linear(out=On((7, 50, 1), F32, 0))
    linear(x=On((8, 256), BF16, 0), out=On((2, 4, 50), F32, 0))
    linear(x=On((1, 256), BF16, 0), out=On((50,), F32, 0))
    norm(y=On((7, 4, 16), BF16, 0), x=On((7, 1, 64), BF16, 0))
    norm(residual=On((0, 64), BF16, 0), x=On((0, 64), BF16, 0), y=On((0, 64), BF16, 0), residual_out=On((0, 64), BF16, 0))
    scores(top_logp=On((28,), F32, 0))
    scores(logits=On((1, 50), F32, 0), targets=On((1,), I32, 0), logp=On((1,), F32, 0), top_ids=On((1, 4), I32, 0),
           top_logp=On((4,), F32, 0))
    assert len(calls.seen) == 8


def test_norm_numbers_are_taken_anew_in_every_call(monkeypatch):
    """Numbers held in tensors that change between calls, as a learned scale does: none is kept by its identity."""
    seen = []

    def call(cfg, *args):
        c = ctypes.cast(cfg, ctypes.POINTER(moe.moe_norm_config)).contents
        seen.append((c.gate_sigmoid, c.residual_scale, c.norm_eps, c.weight_offset))
        return moe.MOE_OK
    monkeypatch.setattr(moe, "_lib", types.SimpleNamespace(moe_residual_norm=call))
    monkeypatch.setattr(moe, "_kinds", {**moe._torch_kinds(), "stream": lambda d: 5, "device": lambda: 0})
    sigmoid, scale, eps, offset = torch.tensor(False), torch.tensor(2.0), torch.tensor(0.5), torch.tensor(1.0)
    for k in range(3):
        norm(gate_sigmoid=sigmoid, residual_scale=scale, eps=eps, weight_offset=offset)
        norm(gate_sigmoid=k % 2, residual_scale=2 + k, eps=0.5 + k, weight_offset=True)
        assert seen[-2] == (k % 2, 2.0 + k, 0.5 + k, 1.0 + k) and seen[-1] == (k % 2, 2.0 + k, 0.5 + k, 1.0)
        for t in (scale, eps, offset):
            t += 1
        sigmoid.logical_not_()


def test_strides_of_padded_rows(monkeypatch):
    """The address and row stride that each form of rows gives; a column that is not contiguous is refused."""
    kind = torch.float32
    monkeypatch.setattr(torch.Tensor, "get_device", lambda self: 0)
    wide = torch.zeros(6, 20)
    for t, want in [(wide, 20), (wide[:, :7], 20), (wide[::2, :7], 40), (wide[:1, :7], 7), (wide[:, 3:4], 20), (wide.T[:4].T, 20),
                    (wide[:, :8].unflatten(1, (2, 4)), 20), (wide[:0, :7], 7)]:
        rows, width = t.shape[0], t[0].numel() if t.shape[0] else 7
        assert moe._matrix("t", t, kind, rows, width, 0) == (t.data_ptr(), want) == moe._rows("t", t, kind, rows, width, 0)
    for t in (wide.T[:4], wide[:, ::2], wide[:1, ::2], wide[:, :8].unflatten(1, (2, 4)).transpose(1, 2)):
        for f in (moe._matrix, moe._rows):
            with pytest.raises(ValueError, match="^t must"):
                f("t", t, kind, t.shape[0], t[0].numel(), 0)
    assert moe._matrix("t", wide[:, 3:4].expand(6, 1), kind, 6, 1, 0)[1] == 20
