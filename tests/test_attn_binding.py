"""The attention binding's checks of its tensors' devices, without a GPU: tensors that only say where they are."""
import contextlib
import math
import types

import pytest
import torch

import expert_offload_slot_gb300 as moe


class On:
    """What the binding asks of a contiguous tensor; `place` -1 is the host."""

    def __init__(self, shape, dtype, place):
        self.shape, self.dtype, self.place = tuple(shape), dtype, place
        self.device = torch.device("cpu") if place < 0 else torch.device("cuda", place)
        self.is_cuda = place >= 0

    def get_device(self):
        return self.place

    def numel(self):
        return math.prod(self.shape)

    def size(self, i):
        return self.shape[i]

    def is_contiguous(self):
        return True

    def stride(self, i=None):
        st = [math.prod(self.shape[k + 1:]) for k in range(len(self.shape))]
        return st if i is None else st[i]

    def data_ptr(self):
        return 4096


@pytest.fixture
def calls(monkeypatch):
    """The library's calls as (name, current device, stream); stream 100 + d is the current one of device d."""
    seen, state = [], {"device": 0}

    class Lib:
        def __getattr__(self, name):
            def call(*args):
                seen.append((name, state["device"], args[-1]))
                return moe.MOE_OK
            return call

    @contextlib.contextmanager
    def on(device):
        before, state["device"] = state["device"], device
        yield
        state["device"] = before
    kinds = dict(moe._torch_kinds())
    kinds.update(stream=lambda d: 100 + d, device=lambda: state["device"], on=on)
    monkeypatch.setattr(moe, "_kinds", kinds)
    monkeypatch.setattr(moe, "_lib", Lib())
    return types.SimpleNamespace(seen=seen, state=state)


def arguments(place, odd=None, odd_place=0):
    """Keyword tensors of the four calls on `place`, the one called `odd` elsewhere."""
    f, b, i = torch.float32, torch.bfloat16, torch.int32

    def t(name, shape, dtype):
        return On(shape, dtype, odd_place if name == odd else place)
    cache = (9, 2, 16, 128)
    return {
        "tables": {n: t(n, s, i) for n, s in dict(ctx_len=(3,), new_len=(3,), block_table=(3, 4), free_pages=(5,), free_head=(1,),
                                                   free_head_out=(1,), row_start=(4,), seq_len=(3,), positions=(7,),
                                                   slot_map=(7,)).items()},
        "qkv": {**{n: t(n, s, b) for n, s in dict(qkv=(7, 12 * 128), q_norm=(128,), k_norm=(128,), q=(7, 8, 128), k_cache=cache,
                                                  v_cache=cache).items()},
                "rope": t("rope", (50, 128), f), "positions": t("positions", (7,), i), "slot_map": t("slot_map", (7,), i)},
        "forward": {**{n: t(n, s, b) for n, s in dict(q=(7, 8, 128), k_cache=cache, v_cache=cache, out=(7, 8, 128)).items()},
                    **{n: t(n, s, i) for n, s in dict(row_start=(4,), seq_len=(3,), block_table=(3, 4)).items()}, "max_new": 3},
        "sample": {**{n: t(n, (7,), f) for n in ("u", "logp", "temperature", "top_p", "min_p")},
                   **{n: t(n, (7,), i) for n in ("ids", "top_k")}, "logits": t("logits", (7, 50), b)},
    }


def call(device, what, args):
    if what == "sample":
        return moe.moe_sample(**args)
    return getattr(moe.Attention(moe.make_attn_config(8, 2, 128, 16), device), what)(**args)


@pytest.mark.parametrize("device", [0, 1])
@pytest.mark.parametrize("what", ["tables", "qkv", "forward", "sample"])
def test_calls_take_the_devices_stream(calls, what, device):
    for current in (0, 1):
        calls.state["device"] = current
        call(device, what, arguments(device)[what])
        name, at, stream = [c for c in calls.seen if c[0] in ("moe_sample", f"moe_attn_{what}")][-1]
        assert stream == 100 + device and calls.state["device"] == current
        if what == "sample":               # it has no handle: the library runs it on the current device
            assert at == device


@pytest.mark.parametrize("device", [0, 1])
@pytest.mark.parametrize("elsewhere", ["host", "gpu"])
@pytest.mark.parametrize("what", ["tables", "qkv", "forward", "sample"])
def test_tensors_elsewhere_are_refused(calls, what, device, elsewhere):
    place = -1 if elsewhere == "host" else 1 - device
    for name in arguments(device)[what]:
        if name == "max_new" or (what, name, elsewhere) == ("sample", "logits", "gpu"):
            continue
        with pytest.raises(ValueError, match="logits|u must" if name == "logits" else f"^{name} must"):
            call(device, what, arguments(device, name, place)[what])
    assert not [c for c in calls.seen if c[0] in ("moe_sample", f"moe_attn_{what}")]
