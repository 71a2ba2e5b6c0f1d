"""Python binding of libmoeslot, the GB300 slot-pool MoE layer.

Argument marshalling only: every step of the layer runs in the CUDA kernels of
libmoeslot.so, reached through ctypes with the C names of include/moeslot.h.
Tensors are passed as raw device pointers (``tensor.data_ptr()``) and streams
as ``torch.cuda.Stream.cuda_stream``.  There is no fallback: if the library has
not been built, importing this package raises.
"""
import ctypes
import numbers
import os

import numpy as np

from ._build import LIB, build  # noqa: F401

if not os.path.exists(LIB):
    raise ImportError(f"{LIB} is missing: build it with `python -c 'import __graft_entry__ as g; g.build()'`")

_lib = ctypes.CDLL(LIB)

MOE_OK, MOE_ERR_INVALID, MOE_ERR_OOM, MOE_ERR_CUDA, MOE_ERR_CAPACITY = 0, 1, 2, 3, 4
MOE_ERR_TIMEOUT, MOE_ERR_TAG, MOE_ERR_BOUNDS = 5, 6, 7
MOE_F32, MOE_BF16, MOE_FP8_E4M3_B128, MOE_RESPLIT_Q4R4 = 0, 1, 2, 3
MOE_GATE_SOFTMAX_RENORM, MOE_GATE_SIGMOID_RENORM = 0, 1
MOE_EVICT_CORE, MOE_EVICT_MRS, MOE_EVICT_LRU = 0, 1, 2
MOE_MODE_AUTO, MOE_MODE_DECODE, MOE_MODE_PREFILL_STAGED = 0, 1, 2
MOE_ROTARY_HALF, MOE_ROTARY_PAIRS = 0, 1
MOE_RESIDUAL_GATE_NONE, MOE_RESIDUAL_GATE_ROW, MOE_RESIDUAL_GATE_CHANNEL, MOE_RESIDUAL_GATE_ELEMENT = 0, 1, 2, 3
MOE_NORM_MAX_HIDDEN, MOE_LINEAR_MAX_IN, MOE_LINEAR_MAX_OUT, MOE_LOGPROBS_MAX_TOP = 16384, 65536, 1 << 20, 32
MOE_ATTN_MAX_REQUESTS, MOE_ATTN_MAX_ROWS, MOE_SAMPLE_MAX_VOCAB = 1024, 1 << 20, 327680
STAGES = ("route", "plan", "copy", "ffn")
MOE_NUM_STAGES = len(STAGES)

STATUS_NAMES = {0: "MOE_OK", 1: "MOE_ERR_INVALID", 2: "MOE_ERR_OOM", 3: "MOE_ERR_CUDA", 4: "MOE_ERR_CAPACITY",
                5: "MOE_ERR_TIMEOUT", 6: "MOE_ERR_TAG", 7: "MOE_ERR_BOUNDS"}


class moe_config(ctypes.Structure):
    _fields_ = [("num_layers", ctypes.c_int32), ("num_experts", ctypes.c_int32), ("top_k", ctypes.c_int32),
                ("hidden", ctypes.c_int32), ("inter", ctypes.c_int32), ("num_slots", ctypes.c_int32),
                ("weight_dtype", ctypes.c_int32), ("act_dtype", ctypes.c_int32), ("gating", ctypes.c_int32),
                ("has_shared_expert", ctypes.c_int32), ("evict_policy", ctypes.c_int32),
                ("window", ctypes.c_int32), ("ema_decay", ctypes.c_float), ("core_w", ctypes.c_float * 4),
                ("staging_regions", ctypes.c_int32), ("max_tokens", ctypes.c_int32)]


class moe_stats(ctypes.Structure):
    _fields_ = [(n, ctypes.c_uint64) for n in ("steps", "hits", "misses", "bypass", "evictions",
                                               "bytes_copied", "near_ties", "staged_layers", "prefetch_issued",
                                               "prefetch_committed", "prefetch_demanded", "prefetch_bytes",
                                               "aes_substitutions", "critical_entries")]


class moe_attn_config(ctypes.Structure):
    _fields_ = [(n, ctypes.c_int32) for n in ("num_q_heads", "num_kv_heads", "head_dim", "page_size", "dtype",
                                              "rotary_dim", "rotary_style", "window")] + \
               [("softmax_scale", ctypes.c_float), ("norm_eps", ctypes.c_float)]


class moe_norm_config(ctypes.Structure):
    _fields_ = [(n, ctypes.c_int32) for n in ("hidden", "dtype", "residual_dtype", "gate", "gate_sigmoid")] + \
               [(n, ctypes.c_float) for n in ("residual_scale", "norm_eps", "weight_offset")]


_vp, _i32, _sz = ctypes.c_void_p, ctypes.c_int32, ctypes.c_size_t
_P, _i64 = ctypes.POINTER, ctypes.c_int64
_sig = {
    "moe_expert_layout": (_i32, [_P(moe_config), _P(_sz), _P(_sz), _P(_sz), _P(_sz), _P(_sz)]),
    "moe_pack_expert_record": (_i32, [_P(moe_config), _vp, _vp, _vp, _vp, _vp, _vp, _vp, _sz]),
    "moe_plan_quotas": (_i32, [_P(moe_config), _vp, _vp, _i32, _i32, _i32, _i32, ctypes.c_double, _vp, _vp]),
    "moe_profile_lut": (_i32, [_P(moe_config), _vp, _i32, _i32, _vp, _vp]),
    "moe_host_alloc": (_i32, [_sz, _P(_vp)]),
    "moe_host_free": (_i32, [_vp]),
    "moe_pool_create": (_i32, [_P(moe_config), _vp, _sz, _vp, _vp, _vp, ctypes.c_int, _P(_vp)]),
    "moe_pool_destroy": (_i32, [_vp]),
    "moe_set_lut": (_i32, [_vp, _vp, _vp]),
    "moe_load_slot": (_i32, [_vp, _i32, _i32, _i32, _vp]),
    "moe_forward": (_i32, [_vp, _i32, _vp, _i32, _vp, _i32, _vp]),
    "moe_forward_routed": (_i32, [_vp, _i32, _vp, _i32, _vp, _vp, _vp, _vp, _vp]),
    "moe_update_scores": (_i32, [_vp, _i32, _vp, _vp, _i32, _vp]),
    "moe_set_wait_limit": (_i32, [_vp, ctypes.c_uint64]),
    "moe_prefetch_enable": (_i32, [_vp, _i32]),
    "moe_set_aes": (_i32, [_vp, _i32, ctypes.c_float]),
    "moe_set_umia": (_i32, [_vp, ctypes.c_float, _vp, ctypes.c_float, ctypes.c_float]),
    "moe_prefetch_drain": (_i32, [_vp]),
    "moe_prefetch_inject_wrong_tags": (_i32, [_vp, ctypes.c_uint32]),
    "moe_get_status": (_i32, [_vp]),
    "moe_clear_status": (_i32, [_vp]),
    "moe_get_routing": (_i32, [_vp, _vp, _vp, _vp, _vp, _vp, _vp, _vp, _i32, _P(_i32)]),
    "moe_get_state": (_i32, [_vp, _vp, _vp, _vp, _vp]),
    "moe_read_slot": (_i32, [_vp, _i32, _vp, _sz]),
    "moe_get_stats": (_i32, [_vp, _P(moe_stats)]),
    "moe_launch_count": (ctypes.c_uint64, [_vp]),
    "moe_profile_enable": (_i32, [_vp, _i32]),
    "moe_profile_read": (_i32, [_vp, _i32, _P(ctypes.c_float)]),
    "moe_attn_create": (_i32, [_P(moe_attn_config), ctypes.c_int, _P(_vp)]),
    "moe_attn_destroy": (_i32, [_vp]),
    "moe_attn_get_status": (_i32, [_vp]),
    "moe_attn_clear_status": (_i32, [_vp]),
    "moe_attn_tables": (_i32, [_vp, _vp, _vp, _i32, _vp, _i32, _vp, _i32, _vp, _vp, _i32, _vp, _vp, _vp, _vp, _vp]),
    "moe_attn_qkv": (_i32, [_vp, _vp, ctypes.c_int64, _i32, _vp, _vp, _vp, _i32, _vp, _vp, _vp, _vp, _vp, _i32, _vp]),
    "moe_attn_forward": (_i32, [_vp, _vp, ctypes.c_int64, _i32, _vp, _vp, _i32, _i32, _vp, _vp, _i32, _vp, _i32, _vp,
                                _vp]),
    "moe_sample": (_i32, [_vp, _i32, _i32, _i32, ctypes.c_int64, _vp, _vp, _vp, _vp, _vp, _vp, _vp, _vp]),
    "moe_residual_norm": (_i32, [_P(moe_norm_config), _vp, _i64, _vp, _i64, _vp, _vp, _i64, _vp, _i64, _vp, _vp, _i64, _i32, _vp]),
    "moe_q4_pack": (_i32, [_vp, _i32, _i32, _i32, _vp, _vp]),
    "moe_linear_q4": (_i32, [_vp, _i32, _i64, _i32, _i32, _vp, _vp, _i32, _i32, _vp, _i32, _vp, _i32, _i64, _vp]),
    "moe_logprobs": (_i32, [_vp, _i32, _i32, _i32, _i64, _vp, _i32, _vp, _vp, _vp, _vp, _vp, _vp]),
    "moe_step_status": (_i32, []),
    "moe_last_error": (ctypes.c_char_p, []),
    "moe_route_topk_noalloc": (_i32, [_i32, _i32, _i32, _i32, _i32, _vp, _i32, _vp, _vp, _vp, _vp, _vp, _vp, _vp]),
}
for _name, (_res, _args) in _sig.items():
    _f = getattr(_lib, _name)
    _f.restype = _res
    _f.argtypes = _args

EXPORTED = tuple(_sig)


class MoeError(RuntimeError):
    def __init__(self, status, where):
        msg = _lib.moe_last_error().decode(errors="replace")
        super().__init__(f"{where}: {STATUS_NAMES.get(status, status)}: {msg}")
        self.status = status


def _check(status, where):
    if status != MOE_OK:
        raise MoeError(status, where)


def _ptr(t):
    """Device/host address of a tensor, numpy array or int; None -> NULL."""
    if t is None:
        return None
    if isinstance(t, int):
        return t
    if isinstance(t, np.ndarray):
        return t.ctypes.data
    return t.data_ptr()


def _stream(stream):
    if stream is None:
        import torch
        return torch.cuda.current_stream().cuda_stream
    if isinstance(stream, int):
        return stream
    return stream.cuda_stream


def make_config(L, E, k, H, I, S, weight_dtype, act_dtype, gating=MOE_GATE_SOFTMAX_RENORM, shared=False,
                evict=MOE_EVICT_CORE, window=16, ema_decay=0.9, core_w=(0.25, 0.25, 0.25, 0.25),
                staging_regions=0, max_tokens=64):
    c = moe_config()
    c.num_layers, c.num_experts, c.top_k, c.hidden, c.inter, c.num_slots = L, E, k, H, I, S
    c.weight_dtype, c.act_dtype, c.gating, c.has_shared_expert = weight_dtype, act_dtype, gating, int(shared)
    c.evict_policy, c.window, c.ema_decay = evict, window, ema_decay
    c.core_w = (ctypes.c_float * 4)(*core_w)
    c.staging_regions, c.max_tokens = staging_regions, max_tokens
    return c


def moe_expert_layout(cfg):
    v = [_sz() for _ in range(5)]
    _check(_lib.moe_expert_layout(ctypes.byref(cfg), *[ctypes.byref(x) for x in v]), "moe_expert_layout")
    return tuple(x.value for x in v)   # (w13_off, w2_off, s13_off, s2_off, record_bytes)


def moe_pack_expert_record(cfg, w_gate, w_up, w_down, s_gate=None, s_up=None, s_down=None):
    """One record (uint8 numpy array) from row-major numpy matrices in the weight dtype's storage."""
    rec = moe_expert_layout(cfg)[4]
    out = np.zeros(rec, np.uint8)
    mats = [np.ascontiguousarray(m) for m in (w_gate, w_up, w_down)]
    scales = [None if v is None else np.ascontiguousarray(v, np.float32) for v in (s_gate, s_up, s_down)]
    _check(_lib.moe_pack_expert_record(ctypes.byref(cfg), *(m.ctypes.data for m in mats),
                                       *(None if v is None else v.ctypes.data for v in scales),
                                       out.ctypes.data, rec), "moe_pack_expert_record")
    return out


def moe_plan_quotas(cfg, ids, probs, budget, delta_k, tau_low):
    """Per-layer slot quotas from a profiling trace (ids int32 [steps,L,T,k], probs float32
    [steps,L,T,E], host numpy).  Returns (quota int32 [L], hit rate float64 [L])."""
    ids = np.ascontiguousarray(ids, np.int32)
    probs = np.ascontiguousarray(probs, np.float32)
    steps, L, T = ids.shape[:3]
    quota = np.zeros(L, np.int32)
    hit = np.zeros(L, np.float64)
    _check(_lib.moe_plan_quotas(ctypes.byref(cfg), ids.ctypes.data, probs.ctypes.data, steps, T, budget, delta_k,
                                float(tau_low), quota.ctypes.data, hit.ctypes.data), "moe_plan_quotas")
    return quota, hit


def moe_profile_lut(cfg, probs, quota):
    """Initial table [L, E] from a profiling trace's probabilities (host numpy) and per-layer quotas."""
    probs = np.ascontiguousarray(probs, np.float32)
    steps, L, T, E = probs.shape
    q = np.ascontiguousarray(quota, np.int32)
    lut = np.zeros((L, E), np.int32)
    _check(_lib.moe_profile_lut(ctypes.byref(cfg), probs.ctypes.data, steps, T, q.ctypes.data, lut.ctypes.data),
           "moe_profile_lut")
    return lut


MOE_NOALLOC_MAX_LOGITS = 65536


def moe_route_topk_noalloc(E, k, H, act_dtype, gating, x, router_w, router_b, ids, w, probs, gap, stream=None):
    """Router + top-k without any device allocation (scratch in a static device array).

    For callers that cannot allocate device memory where they route tokens; see
    include/moeslot.h.  All outputs are caller-owned device tensors.
    """
    _check(_lib.moe_route_topk_noalloc(E, k, H, act_dtype, gating, _ptr(x), x.shape[0], _ptr(router_w),
                                       _ptr(router_b), _ptr(ids), _ptr(w), _ptr(probs), _ptr(gap),
                                       _stream(stream)), "moe_route_topk_noalloc")


class HostPool:
    """Pinned, mapped host memory from moe_host_alloc, viewable as a uint8 numpy array."""

    def __init__(self, nbytes):
        p = _vp()
        _check(_lib.moe_host_alloc(nbytes, ctypes.byref(p)), "moe_host_alloc")
        self.ptr, self.nbytes = p.value, nbytes

    def numpy(self):
        return np.ctypeslib.as_array((ctypes.c_uint8 * self.nbytes).from_address(self.ptr))

    def torch(self):
        import torch
        return torch.frombuffer((ctypes.c_uint8 * self.nbytes).from_address(self.ptr), dtype=torch.uint8)

    def free(self):
        if self.ptr:
            _lib.moe_host_free(self.ptr)
            self.ptr = 0

    def __del__(self):
        try:
            self.free()
        except Exception:
            pass


class Pool:
    """One slot pool (moe_pool_create ... moe_pool_destroy)."""

    def __init__(self, cfg, host_pool_ptr, host_pool_bytes, router_w, router_b, shared_w=None, device=0):
        self.cfg = cfg
        self._keep = (router_w, router_b, shared_w)
        h = _vp()
        _check(_lib.moe_pool_create(ctypes.byref(cfg), host_pool_ptr, host_pool_bytes, _ptr(router_w),
                                    _ptr(router_b), _ptr(shared_w), device, ctypes.byref(h)), "moe_pool_create")
        self.h = h.value
        self.record_bytes = moe_expert_layout(cfg)[4]

    def close(self):
        if self.h:
            _lib.moe_pool_destroy(self.h)
            self.h = None

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass

    def set_lut(self, lut, stream=None):
        a = np.ascontiguousarray(lut, dtype=np.int32).reshape(-1)
        _check(_lib.moe_set_lut(self.h, a.ctypes.data, _stream(stream)), "moe_set_lut")

    def load_slot(self, layer, expert, slot, stream=None):
        _check(_lib.moe_load_slot(self.h, layer, expert, slot, _stream(stream)), "moe_load_slot")

    def forward(self, layer, x, out, mode=MOE_MODE_DECODE, stream=None, T=None):
        T = x.shape[0] if T is None else T
        _check(_lib.moe_forward(self.h, layer, _ptr(x), T, _ptr(out), mode, _stream(stream)), "moe_forward")

    def forward_routed(self, layer, x, ids, w, probs, out, stream=None):
        _check(_lib.moe_forward_routed(self.h, layer, _ptr(x), x.shape[0], _ptr(ids), _ptr(w), _ptr(probs),
                                       _ptr(out), _stream(stream)), "moe_forward_routed")

    def update_scores(self, layer, ids, probs, stream=None):
        _check(_lib.moe_update_scores(self.h, layer, _ptr(ids), _ptr(probs), ids.shape[0], _stream(stream)),
               "moe_update_scores")

    def set_umia(self, theta, beta=None, gamma_decode=1.0, gamma_prefill=1.0):
        b = None if beta is None else np.ascontiguousarray(beta, np.float32)
        _check(_lib.moe_set_umia(self.h, float(theta), None if b is None else b.ctypes.data, float(gamma_decode),
                                 float(gamma_prefill)), "moe_set_umia")

    def set_aes(self, on, alpha=0.0):
        _check(_lib.moe_set_aes(self.h, int(on), float(alpha)), "moe_set_aes")

    def prefetch_enable(self, per_step):
        _check(_lib.moe_prefetch_enable(self.h, int(per_step)), "moe_prefetch_enable")

    def prefetch_drain(self):
        _check(_lib.moe_prefetch_drain(self.h), "moe_prefetch_drain")

    def prefetch_inject_wrong_tags(self, n):
        _check(_lib.moe_prefetch_inject_wrong_tags(self.h, int(n)), "moe_prefetch_inject_wrong_tags")

    def set_wait_limit(self, ns):
        _check(_lib.moe_set_wait_limit(self.h, int(ns)), "moe_set_wait_limit")

    def status(self):
        return _lib.moe_get_status(self.h)

    def clear_status(self):
        _check(_lib.moe_clear_status(self.h), "moe_clear_status")

    def routing(self, cap_T):
        c = self.cfg
        k, E = c.top_k, c.num_experts
        out = {"ids": np.zeros((cap_T, k), np.int32), "w": np.zeros((cap_T, k), np.float32),
               "probs": np.zeros((cap_T, E), np.float32), "gap": np.zeros(cap_T, np.float32),
               "slots": np.zeros((cap_T, k), np.int32), "perm": np.zeros(cap_T * k, np.int32),
               "offs": np.zeros(E + 1, np.int32)}
        T = _i32()
        _check(_lib.moe_get_routing(self.h, *(out[n].ctypes.data for n in ("ids", "w", "probs", "gap", "slots",
                                                                           "perm", "offs")),
                                    cap_T, ctypes.byref(T)), "moe_get_routing")
        T = T.value
        for n in ("ids", "w", "probs", "gap", "slots"):
            out[n] = out[n][:T]
        out["perm"] = out["perm"][:T * k]
        out["T"] = T
        return out

    def state(self):
        c = self.cfg
        LE, S = c.num_layers * c.num_experts, c.num_slots
        lut, owner = np.zeros(LE, np.int32), np.zeros(S, np.int32)
        tag, score = np.zeros(S, np.uint32), np.zeros(LE, np.float32)
        _check(_lib.moe_get_state(self.h, lut.ctypes.data, owner.ctypes.data, tag.ctypes.data, score.ctypes.data),
               "moe_get_state")
        return {"lut": lut.reshape(c.num_layers, c.num_experts), "owner": owner, "tag": tag,
                "score": score.reshape(c.num_layers, c.num_experts)}

    def read_slot(self, slot):
        """The record bytes slot `slot` holds (host copy, blocking)."""
        rec = moe_expert_layout(self.cfg)[4]
        buf = np.zeros(rec, np.uint8)
        _check(_lib.moe_read_slot(self.h, int(slot), buf.ctypes.data, rec), "moe_read_slot")
        return buf

    def stats(self):
        s = moe_stats()
        _check(_lib.moe_get_stats(self.h, ctypes.byref(s)), "moe_get_stats")
        return {n: getattr(s, n) for n, _ in moe_stats._fields_}

    def profile_enable(self, on=True):
        _check(_lib.moe_profile_enable(self.h, int(on)), "moe_profile_enable")

    def profile_read(self, layer):
        v = (ctypes.c_float * MOE_NUM_STAGES)()
        _check(_lib.moe_profile_read(self.h, layer, v), "moe_profile_read")
        return list(v)

    def launch_count(self):
        return int(_lib.moe_launch_count(self.h))


def make_attn_config(num_q_heads, num_kv_heads, head_dim, page_size, dtype=MOE_BF16, rotary_dim=None,
                     rotary_style=MOE_ROTARY_HALF, window=0, softmax_scale=None, norm_eps=1e-6):
    c = moe_attn_config()
    c.num_q_heads, c.num_kv_heads, c.head_dim, c.page_size, c.dtype = num_q_heads, num_kv_heads, head_dim, page_size, dtype
    c.rotary_dim = head_dim if rotary_dim is None else rotary_dim
    c.rotary_style, c.window, c.norm_eps = rotary_style, window, norm_eps
    c.softmax_scale = head_dim ** -0.5 if softmax_scale is None else softmax_scale
    return c


# The calls below run once per layer and step, beside kernels of a few microseconds, so their checks
# are written flat: type, device, element count and contiguity of each tensor, since the library sees
# addresses only.  (numel() takes a third of size(0)'s time, and len(tensor) is a Python function of torch's.)
_kinds = {}


def _torch_kinds():
    """(float32, bfloat16, int32), the raw-stream getter and the current device, looked up once."""
    if not _kinds:
        import torch
        raw = getattr(torch._C, "_cuda_getCurrentRawStream", None)
        _kinds["stream"] = raw or (lambda device: torch.cuda.current_stream(device).cuda_stream)
        _kinds["device"], _kinds["on"] = getattr(torch._C, "_cuda_getDevice", torch.cuda.current_device), torch.cuda.device
        _kinds[MOE_F32], _kinds[MOE_BF16], _kinds["i32"] = torch.float32, torch.bfloat16, torch.int32
        _kinds["u8"] = torch.uint8
    return _kinds


def _flat(name, t, kind, count, device):
    """Address of a contiguous tensor of this type with `count` elements on GPU `device` (a host tensor's is -1)."""
    if t.dtype is kind and t.numel() == count and t.get_device() == device and t.is_contiguous():
        return t.data_ptr()
    raise ValueError(f"{name} must be a contiguous tensor of {kind} with {count} elements on cuda:{device}, "
                     f"got {t.dtype}, {tuple(t.shape)}, strides {t.stride()}, on {t.device}")


def _rows(name, t, kind, rows, width, device):
    """Address and row stride in elements of a tensor [rows, ...] on GPU `device` whose rows hold `width` contiguous elements."""
    if t.dtype is kind and t.numel() == rows * width and t.get_device() == device:
        if t.is_contiguous():
            return t.data_ptr(), width
        inner = 1
        for n, st in zip(reversed(t.shape[1:]), reversed(t.stride())):
            if n != 1 and st != inner:
                break
            inner *= n
        else:
            return t.data_ptr(), (t.stride(0) if rows > 1 else width)
    raise ValueError(f"{name} must be a tensor of {kind} with {rows} rows of {width} contiguous elements on cuda:{device}, "
                     f"got {t.dtype}, {tuple(t.shape)}, strides {t.stride()}, on {t.device}")


def _splits(shape, width):
    """Whether the trailing dimensions make up rows of `width` (a flat tensor's layout is the caller's word)."""
    inner = 1
    for n in reversed(shape):
        if inner == width:
            return True
        inner *= n
    return inner == width or len(shape) == 1


def _not_rows(name, t, rows, width):
    return ValueError(f"{name} must hold [{rows}, {width}], got {tuple(t.shape)}")


def _matrix(name, t, kind, rows, width, device):
    """_rows() of a tensor [rows, width], the same count in another order ([width, rows]) refused."""
    if t.dtype is kind and t.shape == (rows, width) and t.get_device() == device:
        if t.is_contiguous():
            return t.data_ptr(), width
        step, inner = t.stride()
        if inner == 1 or width == 1:
            return t.data_ptr(), (step if rows > 1 else width)
    at = _rows(name, t, kind, rows, width, device)
    if not _splits(t.shape, width):
        raise _not_rows(name, t, rows, width)
    return at


def _table(name, t, kind, rows, width, device):
    """_flat() of a tensor [rows, width], the same count in another order refused."""
    if t.dtype is kind and t.shape == (rows, width) and t.get_device() == device and t.is_contiguous():
        return t.data_ptr()
    at = _flat(name, t, kind, rows * width, device)
    if not _splits(t.shape, width):
        raise _not_rows(name, t, rows, width)
    return at


class Attention:
    """The attention of a step over a paged cache (moe_attn_create ... moe_attn_destroy).

    The handle keeps the workspace that every layer and step shares; its calls must be ordered.
    Cache tensors are [num_pages, num_kv_heads, page_size, head_dim], one pair per layer.
    """

    def __init__(self, cfg, device=0):
        self.cfg = cfg
        self.h = None
        h = _vp()
        _check(_lib.moe_attn_create(ctypes.byref(cfg), device, ctypes.byref(h)), "moe_attn_create")
        self.h = h.value
        kinds = _torch_kinds()
        self._kind, self._i32, self._f32 = kinds[cfg.dtype], kinds["i32"], kinds[MOE_F32]
        self._current, self._device = kinds["stream"], device
        self._q_width = cfg.num_q_heads * cfg.head_dim
        self._qkv_width = self._q_width + 2 * cfg.num_kv_heads * cfg.head_dim
        self._page = cfg.num_kv_heads * cfg.page_size * cfg.head_dim
        self._dim, self._rotary = cfg.head_dim, cfg.rotary_dim

    def close(self):
        if self.h:
            _lib.moe_attn_destroy(self.h)
            self.h = None

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass

    def tables(self, ctx_len, new_len, block_table, free_pages, free_head, free_head_out, row_start, seq_len, positions,
               slot_map, stream=None):
        """Fill block_table, free_head_out, row_start, seq_len, positions and slot_map for the step."""
        i32, n, rows, free, dev = self._i32, ctx_len.numel(), positions.numel(), free_pages.numel(), self._device
        width = block_table.size(1)
        st = _lib.moe_attn_tables(
            self.h, _flat("ctx_len", ctx_len, i32, n, dev), _flat("new_len", new_len, i32, n, dev), n,
            _flat("block_table", block_table, i32, n * width, dev), width,
            _flat("free_pages", free_pages, i32, free, dev), free, _flat("free_head", free_head, i32, 1, dev),
            _flat("free_head_out", free_head_out, i32, 1, dev), rows, _flat("row_start", row_start, i32, n + 1, dev),
            _flat("seq_len", seq_len, i32, n, dev), _flat("positions", positions, i32, rows, dev),
            _flat("slot_map", slot_map, i32, rows, dev), self._current(dev) if stream is None else _stream(stream))
        if st:
            _check(st, "moe_attn_tables")

    def qkv(self, qkv, q_norm, k_norm, rope, positions, slot_map, q, k_cache, v_cache, stream=None):
        """Norm, rotation and cache write of qkv [rows, (Hq + 2 Hkv) * D]; queries go to q [rows, Hq, D]."""
        kind, i32, rows, pages, dim, dev = self._kind, self._i32, qkv.size(0), k_cache.size(0), self._dim, self._device
        length = 0 if rope is None else rope.size(0)
        at, stride = _rows("qkv", qkv, kind, rows, self._qkv_width, dev)
        st = _lib.moe_attn_qkv(
            self.h, at, stride, rows, None if q_norm is None else _flat("q_norm", q_norm, kind, dim, dev),
            None if k_norm is None else _flat("k_norm", k_norm, kind, dim, dev),
            None if rope is None else _flat("rope", rope, self._f32, length * self._rotary, dev), length,
            _flat("positions", positions, i32, rows, dev), _flat("slot_map", slot_map, i32, rows, dev),
            _flat("q", q, kind, rows * self._q_width, dev), _flat("k_cache", k_cache, kind, pages * self._page, dev),
            _flat("v_cache", v_cache, kind, pages * self._page, dev), pages,
            self._current(dev) if stream is None else _stream(stream))
        if st:
            _check(st, "moe_attn_qkv")

    def forward(self, q, row_start, seq_len, max_new, k_cache, v_cache, block_table, out, stream=None):
        """Attention of q [rows, Hq, D] over the cache, into out [rows, Hq, D]."""
        kind, i32, rows, n, pages, dev = self._kind, self._i32, q.size(0), seq_len.numel(), k_cache.size(0), self._device
        width = block_table.size(1)
        at, stride = _rows("q", q, kind, rows, self._q_width, dev)
        st = _lib.moe_attn_forward(
            self.h, at, stride, rows, _flat("row_start", row_start, i32, n + 1, dev), _flat("seq_len", seq_len, i32, n, dev), n,
            max_new, _flat("k_cache", k_cache, kind, pages * self._page, dev),
            _flat("v_cache", v_cache, kind, pages * self._page, dev), pages,
            _flat("block_table", block_table, i32, n * width, dev), width,
            _flat("out", out, kind, rows * self._q_width, dev),
            self._current(dev) if stream is None else _stream(stream))
        if st:
            _check(st, "moe_attn_forward")

    def status(self):
        return _lib.moe_attn_get_status(self.h)

    def clear_status(self):
        _check(_lib.moe_attn_clear_status(self.h), "moe_attn_clear_status")


def moe_sample(logits, u, ids, logp=None, temperature=None, top_k=None, top_p=None, min_p=None, stream=None):
    """Next token of each row of logits [rows, vocab] into ids (and its log probability into logp)."""
    kinds = _torch_kinds()
    f32, i32 = kinds[MOE_F32], kinds["i32"]
    rows, vocab = logits.shape
    dtype = MOE_F32 if logits.dtype is f32 else MOE_BF16
    dev = max(logits.get_device(), 0)          # a host tensor (-1) is refused below
    at, stride = _rows("logits", logits, f32 if dtype == MOE_F32 else kinds[MOE_BF16], rows, vocab, dev)
    args = (
        at, dtype, rows, vocab, stride, None if temperature is None else _flat("temperature", temperature, f32, rows, dev),
        None if top_k is None else _flat("top_k", top_k, i32, rows, dev),
        None if top_p is None else _flat("top_p", top_p, f32, rows, dev),
        None if min_p is None else _flat("min_p", min_p, f32, rows, dev), _flat("u", u, f32, rows, dev),
        _flat("ids", ids, i32, rows, dev), None if logp is None else _flat("logp", logp, f32, rows, dev),
        kinds["stream"](dev) if stream is None else _stream(stream))
    if kinds["device"]() == dev:               # the library's call runs on the current device
        st = _lib.moe_sample(*args)
    else:
        with kinds["on"](dev):
            st = _lib.moe_sample(*args)
    if st:
        _check(st, "moe_sample")


def _launch(name, dev, stream, *args):
    """A call of the library that has no handle and so runs on the current device: on `dev` and its stream."""
    kinds = _kinds
    args += (kinds["stream"](dev) if stream is None else _stream(stream),)
    if kinds["device"]() == dev:
        st = getattr(_lib, name)(*args)
    else:
        with kinds["on"](dev):
            st = getattr(_lib, name)(*args)
    if st:
        _check(st, name)


_norm_configs = {}


def moe_residual_norm(x, residual, residual_out, y, post_weight=None, pre_weight=None, gate=None, gate_sigmoid=False,
                      residual_scale=1.0, eps=1e-6, weight_offset=0.0, stream=None):
    """residual_out = residual + residual_scale gate norm(x, post_weight), y = norm(residual_out, pre_weight).

    x, residual, residual_out and y are [rows, hidden] with contiguous rows; x (then residual_out, too) or y may be
    None.  The block's output is normed only where post_weight [hidden] is given.  gate is [rows, 1], [hidden] or
    [rows, hidden].  residual_out may be residual, and y may be x or, without x, residual.
    """
    kinds = _torch_kinds()
    f32, bf16 = kinds[MOE_F32], kinds[MOE_BF16]
    rows, hidden = residual.shape
    dev = residual.get_device()
    if dev < 0:                                # a host tensor is refused below
        dev = 0
    first = y if x is None else x
    if first is None:
        raise ValueError("x and y must not both be None")
    dtype = f32 if first.dtype is f32 else bf16
    stream_type = f32 if residual.dtype is f32 else dtype
    kind = MOE_RESIDUAL_GATE_NONE
    gate_at, gate_step = None, 0
    if gate is not None:
        if gate.dim() == 1:
            kind, gate_at = MOE_RESIDUAL_GATE_CHANNEL, _flat("gate", gate, dtype, hidden, dev)
        elif gate.shape[-1] == 1:
            kind = MOE_RESIDUAL_GATE_ROW
            gate_at, gate_step = _matrix("gate", gate, dtype, rows, 1, dev)
        else:
            kind = MOE_RESIDUAL_GATE_ELEMENT
            gate_at, gate_step = _matrix("gate", gate, dtype, rows, hidden, dev)
    key = (hidden, dtype, stream_type, kind, gate_sigmoid, residual_scale, eps, weight_offset)
    cfg = _norm_configs.get(key)
    if cfg is None:
        cfg = moe_norm_config(hidden, MOE_F32 if dtype is f32 else MOE_BF16, MOE_F32 if stream_type is f32 else MOE_BF16, kind,
                              int(bool(gate_sigmoid)), residual_scale, eps, weight_offset)
        # plain numbers alone are kept: a tensor's number may change, and its hash is the tensor's identity
        if all(isinstance(v, numbers.Real) for v in key[4:]):
            if len(_norm_configs) > 256:
                _norm_configs.clear()
            _norm_configs[key] = cfg
    x_at, x_step = (None, 0) if x is None else _matrix("x", x, dtype, rows, hidden, dev)
    r_at, r_step = _rows("residual", residual, stream_type, rows, hidden, dev)
    s_at, s_step = (None, 0) if residual_out is None else _matrix("residual_out", residual_out, stream_type, rows, hidden, dev)
    y_at, y_step = (None, 0) if y is None else _matrix("y", y, dtype, rows, hidden, dev)
    _launch("moe_residual_norm", dev, stream, ctypes.byref(cfg), x_at, x_step, gate_at, gate_step,
            None if post_weight is None else _flat("post_weight", post_weight, dtype, hidden, dev), r_at, r_step, s_at, s_step,
            None if pre_weight is None else _flat("pre_weight", pre_weight, dtype, hidden, dev), y_at, y_step, rows)


def moe_q4_pack(w, group=128):
    """4-bit codes (uint8 [out, in / 2]) and scales (float32 [out, ceil(in / group)]) of weights [out, in], host numpy."""
    w = np.ascontiguousarray(w, np.float32)
    if w.ndim != 2:
        raise ValueError(f"weights must be [out, in], got {w.shape}")
    if group not in (32, 64, 128):
        raise ValueError("group must be 32, 64 or 128")
    n, k = w.shape
    codes, scales = np.zeros((n, k // 2), np.uint8), np.zeros((n, -(-k // group)), np.float32)
    _check(_lib.moe_q4_pack(w.ctypes.data, n, k, group, codes.ctypes.data, scales.ctypes.data), "moe_q4_pack")
    return codes, scales


def moe_linear_q4(x, codes, scales, out, group=128, bias=None, stream=None):
    """out [rows, out] = x [rows, in] times the 4-bit weights (codes [out, in / 2], scales [out, ceil(in / group)]) + bias [out]."""
    kinds = _torch_kinds()
    f32, bf16 = kinds[MOE_F32], kinds[MOE_BF16]
    rows, k = x.shape
    n = codes.shape[0]
    dev = x.get_device()
    if dev < 0:                                # a host tensor is refused below
        dev = 0
    dtype = f32 if x.dtype is f32 else bf16
    out_type = f32 if out.dtype is f32 else dtype
    scale_type = f32 if scales.dtype is f32 else bf16
    if group not in (32, 64, 128):
        raise ValueError("group must be 32, 64 or 128")
    x_at, x_step = _rows("x", x, dtype, rows, k, dev)
    out_at, out_step = _matrix("out", out, out_type, rows, n, dev)
    _launch("moe_linear_q4", dev, stream, x_at, MOE_F32 if dtype is f32 else MOE_BF16, x_step, rows, k,
            _flat("codes", codes, kinds["u8"], n * (k // 2), dev),
            _table("scales", scales, scale_type, n, -(-k // group), dev), MOE_F32 if scale_type is f32 else MOE_BF16, group,
            None if bias is None else _flat("bias", bias, dtype, n, dev), n, out_at, MOE_F32 if out_type is f32 else MOE_BF16,
            out_step)


def moe_logprobs(logits, targets, logp, entropy=None, rank=None, top_ids=None, top_logp=None, stream=None):
    """Log probability (logp) and rank of a token of each row of logits [rows, vocab], the rows' entropy and their best
    tokens (top_ids and top_logp, [rows, top])."""
    kinds = _torch_kinds()
    f32, i32 = kinds[MOE_F32], kinds["i32"]
    rows, vocab = logits.shape
    dtype = MOE_F32 if logits.dtype is f32 else MOE_BF16
    dev = logits.get_device()
    if dev < 0:                                # a host tensor is refused below
        dev = 0
    at, step = _rows("logits", logits, f32 if dtype == MOE_F32 else kinds[MOE_BF16], rows, vocab, dev)
    if (top_ids is None) != (top_logp is None):
        raise ValueError("top_ids and top_logp go together")
    top = 0 if top_ids is None else top_ids.shape[1]
    _launch("moe_logprobs", dev, stream, at, dtype, rows, vocab, step, _flat("targets", targets, i32, rows, dev), top,
            _flat("logp", logp, f32, rows, dev), None if entropy is None else _flat("entropy", entropy, f32, rows, dev),
            None if rank is None else _flat("rank", rank, i32, rows, dev),
            None if top_ids is None else _flat("top_ids", top_ids, i32, rows * top, dev),
            None if top_logp is None else _table("top_logp", top_logp, f32, rows, top, dev))


def moe_step_status():
    """MOE_OK, or MOE_ERR_TIMEOUT where a moe_linear_q4 on the current device gave up; blocking, resets it."""
    return _lib.moe_step_status()
