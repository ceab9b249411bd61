"""Python binding of libtpmlp: the t-sharded Megatron tensor-parallel MLP block
on one GB300.

The functions named ``tpmlp_*`` mirror the C ABI of ``include/tpmlp.h`` one to
one: they only marshal arguments (torch CUDA tensors or raw device pointers,
lists of per-shard tensors) and raise :class:`TpmlpError` on a non-OK status.
Every step of the computation runs in the library's CUDA kernels; there is no
CPU or PyTorch fallback, and :func:`load` raises if the library is missing.

``ShardedMLP`` is a small convenience layer that allocates the outputs with
PyTorch (device memory and streams are all PyTorch provides here) and
``TPMLPFunction`` wraps forward/backward as a ``torch.autograd.Function``.
``ShardedAttentionProj`` does the same for the attention block's QKV and
output projections (``tpmlp_attn_*``).
"""
from __future__ import annotations

import contextlib
import ctypes
import os
import threading
from typing import List, Optional, Sequence

from . import _build

__all__ = [
    "TpmlpError", "load", "Plan", "tpmlp_plan_create", "tpmlp_plan_destroy", "tpmlp_workspace_size",
    "tpmlp_plan_set_timeout", "tpmlp_plan_set_stall_injection", "tpmlp_plan_set_stream_k",
    "STREAM_K_OFF", "STREAM_K_AUTO", "STREAM_K_ALWAYS", "STREAM_K_BALANCE",
    "tpmlp_forward", "tpmlp_backward", "tpmlp_backward_recompute", "tpmlp_forward_column", "tpmlp_forward_row", "tpmlp_forward_row_noalloc", "tpmlp_backward_dgrad",
    "tpmlp_backward_fsum", "tpmlp_check", "tpmlp_status_string", "tpmlp_last_cuda_error", "tpmlp_version",
    "tpmlp_last_launch_count", "tpmlp_last_error", "ShardedMLP", "TPMLPFunction", "EXPORTED_SYMBOLS",
    "AttnPlan", "tpmlp_attn_plan_create", "tpmlp_attn_qkv_forward", "tpmlp_attn_out_forward",
    "tpmlp_attn_out_backward", "tpmlp_attn_qkv_backward", "ShardedAttentionProj",
    "tpmlp_plan_set_sequence_stripes", "tpmlp_forward_sp", "tpmlp_backward_sp", "tpmlp_last_split_tiles",
    "LAUNCH_FWD_COLUMN", "LAUNCH_FWD_ROW", "LAUNCH_BWD_DGRAD", "LAUNCH_BWD_FSUM", "tpmlp_eval_activation",
    "ACT_EVAL", "tpmlp_attn_plan_set_qk_norm_rope", "tpmlp_attn_qk_norm_rope_forward",
    "tpmlp_attn_qk_norm_rope_backward", "tpmlp_ckpt8_size", "tpmlp_ckpt8_pack", "tpmlp_ckpt8_unpack",
    "tpmlp_forward_ckpt8", "tpmlp_backward_ckpt8", "ckpt8_pack", "ckpt8_unpack", "TPMLPCheckpointFunction",
    "ROPE_LAYOUT",
]

ACT = {"gelu": 0, "swiglu": 1}
DTYPE = {"bf16": 0, "fp32": 1}
ROPE_LAYOUT = {"halves": 0, "pairs": 1}
STATUS = {0: "TPMLP_OK", 1: "TPMLP_ERR_INVALID_ARG", 2: "TPMLP_ERR_SHAPE", 3: "TPMLP_ERR_ALIGNMENT",
          4: "TPMLP_ERR_UNSUPPORTED", 5: "TPMLP_ERR_CUDA", 6: "TPMLP_ERR_DEVICE_TIMEOUT",
          7: "TPMLP_ERR_NOT_IMPLEMENTED"}
MAX_SHARDS = 16

EXPORTED_SYMBOLS = (
    "tpmlp_plan_create", "tpmlp_plan_destroy", "tpmlp_workspace_size", "tpmlp_forward", "tpmlp_backward",
    "tpmlp_forward_column", "tpmlp_forward_row", "tpmlp_forward_row_noalloc", "tpmlp_backward_dgrad",
    "tpmlp_backward_fsum", "tpmlp_check", "tpmlp_status_string", "tpmlp_last_cuda_error", "tpmlp_version",
    "tpmlp_last_launch_count", "tpmlp_last_error", "tpmlp_plan_set_timeout", "tpmlp_plan_set_stall_injection",
    "tpmlp_backward_recompute", "tpmlp_attn_plan_create", "tpmlp_attn_qkv_forward", "tpmlp_attn_out_forward",
    "tpmlp_attn_out_backward", "tpmlp_attn_qkv_backward", "tpmlp_plan_set_sequence_stripes", "tpmlp_forward_sp",
    "tpmlp_backward_sp", "tpmlp_plan_set_stream_k", "tpmlp_last_split_tiles", "tpmlp_eval_activation",
    "tpmlp_attn_plan_set_qk_norm_rope", "tpmlp_attn_qk_norm_rope_forward", "tpmlp_attn_qk_norm_rope_backward",
    "tpmlp_ckpt8_size", "tpmlp_ckpt8_pack", "tpmlp_ckpt8_unpack", "tpmlp_forward_ckpt8", "tpmlp_backward_ckpt8",
)

# forms of tpmlp_eval_activation
ACT_EVAL = {"gelu": 0, "gelu_bwd": 1, "gelu_bwd_h": 2, "swiglu": 3, "swiglu_bwd": 4, "swiglu_bwd_h": 5,
            "fp32_gelu": 6, "fp32_swiglu": 7}

# launch kinds of tpmlp_last_split_tiles
LAUNCH_FWD_COLUMN, LAUNCH_FWD_ROW, LAUNCH_BWD_DGRAD, LAUNCH_BWD_FSUM = 0, 1, 2, 3


class TpmlpError(RuntimeError):
    def __init__(self, status: int, where: str):
        self.status = int(status)
        name = STATUS.get(self.status, f"status {status}")
        extra = ""
        if _lib is not None:
            msg = _lib.tpmlp_last_error()
            if msg:
                extra = f": {msg.decode(errors='replace')}"
        super().__init__(f"{where}: {name}{extra}")


class _Desc(ctypes.Structure):
    _fields_ = [("T", ctypes.c_int64), ("d", ctypes.c_int64), ("t", ctypes.c_int32),
                ("d_i", ctypes.POINTER(ctypes.c_int64)), ("act", ctypes.c_int), ("dtype", ctypes.c_int)]


class _AttnDesc(ctypes.Structure):
    _fields_ = [("T", ctypes.c_int64), ("d", ctypes.c_int64), ("t", ctypes.c_int32),
                ("dq_i", ctypes.POINTER(ctypes.c_int64)), ("dkv_i", ctypes.POINTER(ctypes.c_int64)),
                ("dtype", ctypes.c_int)]


class _QkDesc(ctypes.Structure):
    _fields_ = [("head_dim", ctypes.c_int32), ("rotary_dim", ctypes.c_int32), ("layout", ctypes.c_int),
                ("norm", ctypes.c_int32), ("eps", ctypes.c_float), ("base", ctypes.c_double),
                ("inv_freq", ctypes.POINTER(ctypes.c_double))]


_lib = None
_lock = threading.Lock()


def library_path() -> str:
    return _build.LIB


def load():
    """Load libtpmlp.so (built by ``__graft_entry__.build()`` / ``_build.build()``)."""
    global _lib
    with _lock:
        if _lib is not None:
            return _lib
        path = _build.LIB
        if not os.path.exists(path):
            raise RuntimeError(f"CUDA library not built: {path} is missing (run __graft_entry__.build())")
        lib = ctypes.CDLL(path)
        vp, pp, i32, st = ctypes.c_void_p, ctypes.POINTER(ctypes.c_void_p), ctypes.c_int, ctypes.c_int
        lib.tpmlp_plan_create.argtypes = [ctypes.POINTER(_Desc), ctypes.POINTER(vp)]
        lib.tpmlp_plan_create.restype = st
        lib.tpmlp_plan_destroy.argtypes = [vp]
        lib.tpmlp_plan_destroy.restype = None
        lib.tpmlp_plan_set_timeout.argtypes = [vp, ctypes.c_uint32]
        lib.tpmlp_plan_set_timeout.restype = st
        lib.tpmlp_plan_set_stall_injection.argtypes = [vp, ctypes.c_int]
        lib.tpmlp_plan_set_stall_injection.restype = st
        lib.tpmlp_plan_set_stream_k.argtypes = [vp, ctypes.c_int]
        lib.tpmlp_plan_set_stream_k.restype = st
        lib.tpmlp_workspace_size.argtypes = [vp]
        lib.tpmlp_workspace_size.restype = ctypes.c_size_t
        lib.tpmlp_forward.argtypes = [vp, vp, pp, pp, pp, pp, pp, vp, vp, pp, pp, vp, vp]
        lib.tpmlp_forward.restype = st
        lib.tpmlp_backward.argtypes = [vp, vp, pp, pp, pp, pp, pp, vp, pp, vp, pp, pp, pp, pp, pp, vp, vp, vp]
        lib.tpmlp_backward.restype = st
        lib.tpmlp_backward_recompute.argtypes = [vp, vp, pp, pp, pp, pp, pp, vp, pp, vp, pp, pp, pp, pp, pp, vp, vp,
                                                 vp]
        lib.tpmlp_backward_recompute.restype = st
        lib.tpmlp_forward_column.argtypes = [vp, vp, pp, pp, pp, pp, pp, pp, vp, vp]
        lib.tpmlp_forward_column.restype = st
        lib.tpmlp_forward_row.argtypes = [vp, pp, vp, pp, vp, vp, vp]
        lib.tpmlp_forward_row.restype = st
        lib.tpmlp_forward_row_noalloc.argtypes = [vp, pp, pp, vp, vp]
        lib.tpmlp_forward_row_noalloc.restype = st
        lib.tpmlp_backward_dgrad.argtypes = [vp, pp, pp, pp, vp, pp, pp, vp, vp, vp]
        lib.tpmlp_backward_dgrad.restype = st
        lib.tpmlp_backward_fsum.argtypes = [vp, vp, pp, pp, pp, vp, pp, pp, pp, pp, vp, vp]
        lib.tpmlp_backward_fsum.restype = st
        lib.tpmlp_attn_plan_create.argtypes = [ctypes.POINTER(_AttnDesc), ctypes.POINTER(vp)]
        lib.tpmlp_attn_plan_create.restype = st
        lib.tpmlp_attn_qkv_forward.argtypes = [vp, vp, pp, pp, vp, vp]
        lib.tpmlp_attn_qkv_forward.restype = st
        lib.tpmlp_attn_out_forward.argtypes = [vp, pp, pp, vp, vp, vp]
        lib.tpmlp_attn_out_forward.restype = st
        lib.tpmlp_attn_out_backward.argtypes = [vp, pp, pp, vp, pp, pp, vp, vp]
        lib.tpmlp_attn_out_backward.restype = st
        lib.tpmlp_attn_qkv_backward.argtypes = [vp, vp, pp, pp, vp, pp, vp, vp]
        lib.tpmlp_attn_qkv_backward.restype = st
        lib.tpmlp_plan_set_sequence_stripes.argtypes = [vp, ctypes.c_int32, ctypes.POINTER(ctypes.c_int64)]
        lib.tpmlp_plan_set_sequence_stripes.restype = st
        lib.tpmlp_forward_sp.argtypes = [vp, pp, pp, pp, pp, pp, pp, vp, pp, pp, pp, vp, vp]
        lib.tpmlp_forward_sp.restype = st
        lib.tpmlp_backward_sp.argtypes = [vp, pp, pp, pp, pp, pp, pp, pp, pp, pp, pp, pp, pp, pp, pp, vp, vp, vp]
        lib.tpmlp_backward_sp.restype = st
        lib.tpmlp_check.argtypes = [vp, vp, vp]
        lib.tpmlp_check.restype = st
        lib.tpmlp_status_string.argtypes = [i32]
        lib.tpmlp_status_string.restype = ctypes.c_char_p
        lib.tpmlp_last_error.argtypes = []
        lib.tpmlp_last_error.restype = ctypes.c_char_p
        lib.tpmlp_last_cuda_error.argtypes = []
        lib.tpmlp_last_cuda_error.restype = i32
        lib.tpmlp_version.argtypes = []
        lib.tpmlp_version.restype = i32
        lib.tpmlp_last_launch_count.argtypes = []
        lib.tpmlp_last_launch_count.restype = i32
        lib.tpmlp_last_split_tiles.argtypes = [i32, ctypes.POINTER(ctypes.c_int64), i32]
        lib.tpmlp_last_split_tiles.restype = i32
        lib.tpmlp_eval_activation.argtypes = [i32, vp, vp, vp, vp, vp, vp, ctypes.c_int64, vp]
        lib.tpmlp_eval_activation.restype = st
        i64 = ctypes.c_int64
        lib.tpmlp_attn_plan_set_qk_norm_rope.argtypes = [vp, ctypes.POINTER(_QkDesc)]
        lib.tpmlp_attn_plan_set_qk_norm_rope.restype = st
        lib.tpmlp_attn_qk_norm_rope_forward.argtypes = [vp, pp, vp, vp, vp, pp, vp]
        lib.tpmlp_attn_qk_norm_rope_forward.restype = st
        lib.tpmlp_attn_qk_norm_rope_backward.argtypes = [vp, pp, vp, vp, vp, pp, pp, pp, vp, vp, vp, vp]
        lib.tpmlp_attn_qk_norm_rope_backward.restype = st
        lib.tpmlp_ckpt8_size.argtypes = [i64, i64]
        lib.tpmlp_ckpt8_size.restype = ctypes.c_size_t
        lib.tpmlp_ckpt8_pack.argtypes = [i32, i64, i64, vp, i64, vp, vp]
        lib.tpmlp_ckpt8_pack.restype = st
        lib.tpmlp_ckpt8_unpack.argtypes = [i32, i64, i64, vp, vp, i64, vp]
        lib.tpmlp_ckpt8_unpack.restype = st
        lib.tpmlp_forward_ckpt8.argtypes = lib.tpmlp_forward.argtypes
        lib.tpmlp_forward_ckpt8.restype = st
        lib.tpmlp_backward_ckpt8.argtypes = lib.tpmlp_backward_recompute.argtypes
        lib.tpmlp_backward_ckpt8.restype = st
        _lib = lib
        return lib


# ---------------------------------------------------------------- marshalling

def _addr(x) -> Optional[int]:
    if x is None:
        return None
    if isinstance(x, int):
        return x
    if hasattr(x, "data_ptr"):
        if x.numel() and not x.is_cuda:
            raise ValueError("tensor must live on a CUDA device")
        if x.numel() and not x.is_contiguous():
            raise ValueError("tensor must be contiguous (row-major)")
        return x.data_ptr() or None
    raise TypeError(f"expected a tensor or an int device pointer, got {type(x)}")


def _arr(xs, n=0) -> Optional[ctypes.Array]:
    """A host array of addresses; n: how many of them the call reads."""
    if xs is not None and len(xs) < n:
        raise ValueError(f"expected {n} tensors or addresses, got {len(xs)}")
    if xs is None or (isinstance(xs, ctypes.Array) and xs._type_ is ctypes.c_void_p):
        return xs
    return (ctypes.c_void_p * len(xs))(*[_addr(x) for x in xs])


def _positions(plan, x) -> Optional[int]:
    if hasattr(x, "data_ptr"):
        if str(x.dtype) != "torch.int64" or x.numel() != plan.T:
            raise ValueError(f"positions must be {plan.T} int64 numbers, got {x.numel()} of {x.dtype}")
    return _addr(x)


def _stream(stream) -> Optional[int]:
    if stream is None:
        try:
            import torch
            return torch.cuda.current_stream().cuda_stream or None
        except Exception:  # no torch CUDA: legacy default stream
            return None
    if isinstance(stream, int):
        return stream or None
    return stream.cuda_stream or None


def _ok(status: int, where: str):
    if status != 0:
        raise TpmlpError(status, where)


class Plan:
    """Owns a ``tpmlp_plan*`` (host memory only)."""

    def __init__(self, T: int, d: int, d_i: Sequence[int], act: str = "gelu", dtype: str = "bf16"):
        lib = load()
        self.T, self.d, self.d_i = int(T), int(d), tuple(int(v) for v in d_i)
        self.t = len(self.d_i)
        self.act, self.dtype = act, dtype
        self._d_i = (ctypes.c_int64 * max(1, self.t))(*self.d_i)
        desc = _Desc(self.T, self.d, self.t, ctypes.cast(self._d_i, ctypes.POINTER(ctypes.c_int64)),
                     ACT[act] if isinstance(act, str) else int(act),
                     DTYPE[dtype] if isinstance(dtype, str) else int(dtype))
        h = ctypes.c_void_p()
        _ok(lib.tpmlp_plan_create(ctypes.byref(desc), ctypes.byref(h)), "tpmlp_plan_create")
        self.handle = h
        self.stripe_rows = ()  # sequence-parallel token stripes (tpmlp_plan_set_sequence_stripes)

    @property
    def dff(self) -> int:
        return sum(self.d_i)

    def __del__(self):
        h = getattr(self, "handle", None)
        if h is not None and h.value and _lib is not None:
            _lib.tpmlp_plan_destroy(h)
            self.handle = None


def tpmlp_plan_create(T, d, d_i, act="gelu", dtype="bf16") -> Plan:
    return Plan(T, d, d_i, act, dtype)


def tpmlp_plan_destroy(plan: Plan):
    if plan.handle is not None and plan.handle.value:
        load().tpmlp_plan_destroy(plan.handle)
        plan.handle = None


class AttnPlan(Plan):
    """Owns an attention ``tpmlp_plan*``: per-shard query widths dq_i and
    key/value widths dkv_i (fused QKV width n_i = dq_i + 2 dkv_i)."""

    def __init__(self, T: int, d: int, dq_i: Sequence[int], dkv_i: Sequence[int], dtype: str = "bf16"):
        lib = load()
        self.T, self.d = int(T), int(d)
        self.dq_i, self.dkv_i = tuple(int(v) for v in dq_i), tuple(int(v) for v in dkv_i)
        if len(self.dq_i) != len(self.dkv_i):
            raise ValueError("dq_i and dkv_i must have one entry per shard")
        self.t = len(self.dq_i)
        self.d_i = tuple(q + 2 * kv for q, kv in zip(self.dq_i, self.dkv_i))
        self.act, self.dtype = None, dtype
        self._dq = (ctypes.c_int64 * max(1, self.t))(*self.dq_i)
        self._dkv = (ctypes.c_int64 * max(1, self.t))(*self.dkv_i)
        desc = _AttnDesc(self.T, self.d, self.t, ctypes.cast(self._dq, ctypes.POINTER(ctypes.c_int64)),
                         ctypes.cast(self._dkv, ctypes.POINTER(ctypes.c_int64)),
                         DTYPE[dtype] if isinstance(dtype, str) else int(dtype))
        h = ctypes.c_void_p()
        _ok(lib.tpmlp_attn_plan_create(ctypes.byref(desc), ctypes.byref(h)), "tpmlp_attn_plan_create")
        self.handle = h


def tpmlp_attn_plan_create(T, d, dq_i, dkv_i, dtype="bf16") -> AttnPlan:
    return AttnPlan(T, d, dq_i, dkv_i, dtype)


def tpmlp_attn_qkv_forward(plan, X, Wqkv, QKV, workspace, stream=None):
    _ok(load().tpmlp_attn_qkv_forward(plan.handle, _addr(X), _arr(Wqkv), _arr(QKV), _addr(workspace),
                                      _stream(stream)), "tpmlp_attn_qkv_forward")


def tpmlp_attn_out_forward(plan, WO, O, Z, workspace, stream=None):
    _ok(load().tpmlp_attn_out_forward(plan.handle, _arr(WO), _arr(O), _addr(Z), _addr(workspace), _stream(stream)),
        "tpmlp_attn_out_forward")


def tpmlp_attn_out_backward(plan, WO, O, dZ, dO, dWO, workspace, stream=None):
    _ok(load().tpmlp_attn_out_backward(plan.handle, _arr(WO), _arr(O), _addr(dZ), _arr(dO), _arr(dWO),
                                       _addr(workspace), _stream(stream)), "tpmlp_attn_out_backward")


def tpmlp_attn_qkv_backward(plan, X, Wqkv, dQKV, dX, dWqkv, workspace, stream=None):
    _ok(load().tpmlp_attn_qkv_backward(plan.handle, _addr(X), _arr(Wqkv), _arr(dQKV), _addr(dX), _arr(dWqkv),
                                       _addr(workspace), _stream(stream)), "tpmlp_attn_qkv_backward")


def tpmlp_attn_plan_set_qk_norm_rope(plan, head_dim, rotary_dim=None, layout="halves", norm=True, eps=1e-6,
                                     base=10000.0, inv_freq=None):
    """Describe the plan's heads for tpmlp_attn_qk_norm_rope_*: head_dim elements, the first rotary_dim (None: all)
    of them rotated; inv_freq: rotary_dim / 2 radians per position (None: base ** (-2 j / rotary_dim))."""
    rotary_dim = head_dim if rotary_dim is None else rotary_dim
    freq = None
    if inv_freq is not None:
        if len(inv_freq) != int(rotary_dim) // 2:
            raise ValueError(f"inv_freq must have rotary_dim / 2 = {int(rotary_dim) // 2} entries, got {len(inv_freq)}")
        freq = (ctypes.c_double * max(1, len(inv_freq)))(*[float(f) for f in inv_freq])
    desc = _QkDesc(int(head_dim), int(rotary_dim), ROPE_LAYOUT[layout] if isinstance(layout, str) else int(layout),
                   int(norm), float(eps), float(base),
                   ctypes.cast(freq, ctypes.POINTER(ctypes.c_double)) if freq is not None else None)
    _ok(load().tpmlp_attn_plan_set_qk_norm_rope(plan.handle, ctypes.byref(desc)), "tpmlp_attn_plan_set_qk_norm_rope")
    plan.head_dim, plan.qk_norm = int(head_dim), bool(norm)


def tpmlp_attn_qk_norm_rope_forward(plan, QKV, positions, gq, gk, QK, stream=None):
    t = plan.t
    _ok(load().tpmlp_attn_qk_norm_rope_forward(plan.handle, _arr(QKV, t), _positions(plan, positions), _addr(gq),
                                               _addr(gk), _arr(QK, t), _stream(stream)),
        "tpmlp_attn_qk_norm_rope_forward")


def tpmlp_attn_qk_norm_rope_backward(plan, QKV, positions, gq, gk, dQK, dV, dQKV, dgq, dgk, workspace, stream=None):
    if hasattr(workspace, "numel") and workspace.numel() * workspace.element_size() < tpmlp_workspace_size(plan):
        raise ValueError("workspace is smaller than tpmlp_workspace_size(plan)")
    t = plan.t
    _ok(load().tpmlp_attn_qk_norm_rope_backward(plan.handle, _arr(QKV, t), _positions(plan, positions), _addr(gq),
                                                _addr(gk), _arr(dQK, t), _arr(dV, t), _arr(dQKV, t), _addr(dgq),
                                                _addr(dgk), _addr(workspace), _stream(stream)),
        "tpmlp_attn_qk_norm_rope_backward")


def tpmlp_ckpt8_size(rows: int, cols: int) -> int:
    """Bytes of the 8-bit checkpoint of a [rows x cols] tensor."""
    return int(load().tpmlp_ckpt8_size(int(rows), int(cols)))


def tpmlp_ckpt8_pack(dtype, rows, cols, src, ld, ckpt, stream=None):
    _ok(load().tpmlp_ckpt8_pack(DTYPE[dtype] if isinstance(dtype, str) else int(dtype), int(rows), int(cols),
                                _addr(src), int(ld), _addr(ckpt), _stream(stream)), "tpmlp_ckpt8_pack")


def tpmlp_ckpt8_unpack(dtype, rows, cols, ckpt, dst, ld, stream=None):
    _ok(load().tpmlp_ckpt8_unpack(DTYPE[dtype] if isinstance(dtype, str) else int(dtype), int(rows), int(cols),
                                  _addr(ckpt), _addr(dst), int(ld), _stream(stream)), "tpmlp_ckpt8_unpack")


def _shards(plan):
    """Shards, those that have a W3, and activation tensors of an MLP plan."""
    t3 = plan.t if getattr(plan, "act", None) in ("swiglu", ACT["swiglu"]) else 0
    return plan.t, t3, plan.t + t3


def tpmlp_forward_ckpt8(plan, X, W1, W3, W2, b1, b3, b2, Y, ckpt, H, workspace, stream=None):
    t, t3, n = _shards(plan)
    _ok(load().tpmlp_forward_ckpt8(plan.handle, _addr(X), _arr(W1, t), _arr(W3, t3), _arr(W2, t), _arr(b1, t),
                                   _arr(b3, t3), _addr(b2), _addr(Y), _arr(ckpt, n), _arr(H, t), _addr(workspace),
                                   _stream(stream)),
        "tpmlp_forward_ckpt8")


def tpmlp_backward_ckpt8(plan, X, W1, W3, W2, ckpt, H, dY, dact, dX, dW1, dW3, dW2, db1, db3, db2, workspace,
                         stream=None):
    t, t3, n = _shards(plan)
    _ok(load().tpmlp_backward_ckpt8(plan.handle, _addr(X), _arr(W1, t), _arr(W3, t3), _arr(W2, t), _arr(ckpt, n),
                                    _arr(H, t), _addr(dY), _arr(dact, n), _addr(dX), _arr(dW1, t), _arr(dW3, t3),
                                    _arr(dW2, t), _arr(db1, t), _arr(db3, t3), _addr(db2), _addr(workspace),
                                    _stream(stream)),
        "tpmlp_backward_ckpt8")


def tpmlp_plan_set_sequence_stripes(plan: Plan, stripe_rows: Sequence[int]):
    rows = (ctypes.c_int64 * max(1, len(stripe_rows)))(*[int(r) for r in stripe_rows])
    _ok(load().tpmlp_plan_set_sequence_stripes(plan.handle, len(stripe_rows), rows),
        "tpmlp_plan_set_sequence_stripes")
    plan.stripe_rows = tuple(int(r) for r in stripe_rows)


def tpmlp_forward_sp(plan, X_stripes, W1, W3, W2, b1, b3, b2, Y_stripes, saved, H, workspace, stream=None):
    _ok(load().tpmlp_forward_sp(plan.handle, _arr(X_stripes), _arr(W1), _arr(W3), _arr(W2), _arr(b1), _arr(b3),
                                _addr(b2), _arr(Y_stripes), _arr(saved), _arr(H), _addr(workspace), _stream(stream)),
        "tpmlp_forward_sp")


def tpmlp_backward_sp(plan, X_stripes, W1, W3, W2, saved, H, dY_stripes, dact, dX_stripes, dW1, dW3, dW2, db1, db3,
                      db2, workspace, stream=None):
    _ok(load().tpmlp_backward_sp(plan.handle, _arr(X_stripes), _arr(W1), _arr(W3), _arr(W2), _arr(saved), _arr(H),
                                 _arr(dY_stripes), _arr(dact), _arr(dX_stripes), _arr(dW1), _arr(dW3), _arr(dW2),
                                 _arr(db1), _arr(db3), _addr(db2), _addr(workspace), _stream(stream)),
        "tpmlp_backward_sp")


def tpmlp_plan_set_timeout(plan: Plan, timeout_ms: int):
    _ok(load().tpmlp_plan_set_timeout(plan.handle, int(timeout_ms)), "tpmlp_plan_set_timeout")


def tpmlp_plan_set_stall_injection(plan: Plan, enable):
    """False / True (1): producers load nothing; 2: stream-K parts are never published."""
    mode = 2 if enable == 2 else (1 if enable else 0)
    _ok(load().tpmlp_plan_set_stall_injection(plan.handle, mode), "tpmlp_plan_set_stall_injection")


STREAM_K_OFF, STREAM_K_AUTO, STREAM_K_ALWAYS, STREAM_K_BALANCE = 0, 1, 2, 3


def tpmlp_plan_set_stream_k(plan: Plan, mode: int):
    """Stream-K tail of the bf16 launches: STREAM_K_AUTO (default), _ALWAYS or _OFF."""
    _ok(load().tpmlp_plan_set_stream_k(plan.handle, int(mode)), "tpmlp_plan_set_stream_k")


def tpmlp_workspace_size(plan: Plan) -> int:
    return int(load().tpmlp_workspace_size(plan.handle))


def tpmlp_forward(plan, X, W1, W3, W2, b1, b3, b2, Y, saved, H, workspace, stream=None):
    _ok(load().tpmlp_forward(plan.handle, _addr(X), _arr(W1), _arr(W3), _arr(W2), _arr(b1), _arr(b3), _addr(b2),
                             _addr(Y), _arr(saved), _arr(H), _addr(workspace), _stream(stream)), "tpmlp_forward")


def tpmlp_backward(plan, X, W1, W3, W2, saved, H, dY, dact, dX, dW1, dW3, dW2, db1, db3, db2, workspace,
                   stream=None):
    _ok(load().tpmlp_backward(plan.handle, _addr(X), _arr(W1), _arr(W3), _arr(W2), _arr(saved), _arr(H),
                              _addr(dY), _arr(dact), _addr(dX), _arr(dW1), _arr(dW3), _arr(dW2), _arr(db1),
                              _arr(db3), _addr(db2), _addr(workspace), _stream(stream)), "tpmlp_backward")


def tpmlp_backward_recompute(plan, X, W1, W3, W2, saved, H, dY, dact, dX, dW1, dW3, dW2, db1, db3, db2, workspace,
                             stream=None):
    _ok(load().tpmlp_backward_recompute(plan.handle, _addr(X), _arr(W1), _arr(W3), _arr(W2), _arr(saved), _arr(H),
                                        _addr(dY), _arr(dact), _addr(dX), _arr(dW1), _arr(dW3), _arr(dW2), _arr(db1),
                                        _arr(db3), _addr(db2), _addr(workspace), _stream(stream)),
        "tpmlp_backward_recompute")


def tpmlp_forward_column(plan, X, W1, W3, b1, b3, saved, H, workspace, stream=None):
    _ok(load().tpmlp_forward_column(plan.handle, _addr(X), _arr(W1), _arr(W3), _arr(b1), _arr(b3), _arr(saved),
                                    _arr(H), _addr(workspace), _stream(stream)), "tpmlp_forward_column")


def tpmlp_forward_row(plan, W2, b2, H, Y, workspace, stream=None):
    _ok(load().tpmlp_forward_row(plan.handle, _arr(W2), _addr(b2), _arr(H), _addr(Y), _addr(workspace),
                                 _stream(stream)), "tpmlp_forward_row")


def tpmlp_forward_row_noalloc(plan, W2, H, Y, stream=None):
    """Row-parallel GEMM (g-sum) without a workspace: the scratch status word
    is a library-owned static device array, for callers that cannot allocate
    device memory.  Blocks until its kernel has finished."""
    _ok(load().tpmlp_forward_row_noalloc(plan.handle, _arr(W2), _arr(H), _addr(Y), _stream(stream)),
        "tpmlp_forward_row_noalloc")


def tpmlp_backward_dgrad(plan, W2, saved, H, dY, dact, dW2, db2, workspace, stream=None):
    _ok(load().tpmlp_backward_dgrad(plan.handle, _arr(W2), _arr(saved), _arr(H), _addr(dY), _arr(dact), _arr(dW2),
                                    _addr(db2), _addr(workspace), _stream(stream)), "tpmlp_backward_dgrad")


def tpmlp_backward_fsum(plan, X, W1, W3, dact, dX, dW1, dW3, db1, db3, workspace, stream=None):
    _ok(load().tpmlp_backward_fsum(plan.handle, _addr(X), _arr(W1), _arr(W3), _arr(dact), _addr(dX), _arr(dW1),
                                   _arr(dW3), _arr(db1), _arr(db3), _addr(workspace), _stream(stream)),
        "tpmlp_backward_fsum")


def tpmlp_check(plan, workspace, stream=None):
    _ok(load().tpmlp_check(plan.handle, _addr(workspace), _stream(stream)), "tpmlp_check")


def tpmlp_status_string(status: int) -> str:
    return load().tpmlp_status_string(int(status)).decode()


def tpmlp_last_cuda_error() -> int:
    return int(load().tpmlp_last_cuda_error())


def tpmlp_last_error() -> str:
    return load().tpmlp_last_error().decode(errors="replace")


def tpmlp_version() -> int:
    return int(load().tpmlp_version())


def tpmlp_last_launch_count() -> int:
    return int(load().tpmlp_last_launch_count())


def tpmlp_eval_activation(form: str, x, y=None, dh=None, out0=None, out1=None, out2=None, stream=None):
    """The epilogues' activation forms on fp32 device tensors of n elements
    (form: a key of ACT_EVAL); outputs are caller tensors like x."""
    n = x.numel()
    _ok(load().tpmlp_eval_activation(ACT_EVAL[form], _addr(x), _addr(y), _addr(dh), _addr(out0), _addr(out1),
                                     _addr(out2), n, _stream(stream)), "tpmlp_eval_activation")


def tpmlp_last_split_tiles(launch_kind: int) -> List[tuple]:
    """(problem, first row, first column, address of the problem's first output)
    of every tile the stream-K schedule split in the last launch of this kind on
    the calling thread."""
    lib = load()
    n = int(lib.tpmlp_last_split_tiles(int(launch_kind), None, 0))
    if n < 0:
        raise ValueError(f"unknown launch kind {launch_kind}")
    buf = (ctypes.c_int64 * max(1, 4 * n))()
    lib.tpmlp_last_split_tiles(int(launch_kind), buf, n)
    return [tuple(int(buf[4 * i + k]) for k in range(4)) for i in range(n)]


# ---------------------------------------------------------------- convenience layer

def _tdtype(dtype: str):
    import torch
    return {"bf16": torch.bfloat16, "fp32": torch.float32}[dtype]


def _ptr(name: str, x, shape, dtype, device) -> int:
    """The address of a tensor argument of the classes below, which has to be a dense tensor of this shape, type
    and device."""
    if x.shape != shape or x.dtype != dtype or x.device != device or not x.is_contiguous():
        raise ValueError(f"{name}: expected a contiguous {tuple(shape)} tensor of {dtype} on {device}, got "
                         f"{tuple(x.shape)} of {x.dtype} on {x.device}, strides {x.stride()}")
    return x.data_ptr()


def _ptrs(name: str, xs, shapes, dtype, device):
    if xs is None or len(xs) != len(shapes):
        raise ValueError(f"{name}: expected {len(shapes)} tensors, got {0 if xs is None else len(xs)}")
    return (ctypes.c_void_p * len(shapes))(*[_ptr(name, x, s, dtype, device) for x, s in zip(xs, shapes)])


def _new_list(like, shapes):
    """New tensors of like's type and device, and their addresses."""
    xs = [like.new_empty(s) for s in shapes]
    return xs, (ctypes.c_void_p * len(xs))(*[x.data_ptr() for x in xs])


def _current(device) -> int:
    """The handle of the device's current stream."""
    import torch
    return torch._C._cuda_getCurrentRawStream(device.index)


def _on(device, stream):
    """A context with the call's device and stream as the current ones, so that what the call allocates belongs to
    that stream.  stream: None (the device's current one), a torch stream or a raw handle (0: the default stream)."""
    import torch
    if stream is None:
        if torch.cuda.current_device() == device.index:
            return contextlib.nullcontext()
        return torch.cuda.device(device)
    if not hasattr(stream, "cuda_stream"):
        handle = int(stream)
        stream = torch.cuda.ExternalStream(handle, device) if handle else torch.cuda.default_stream(device)
    if stream.device != device:
        raise ValueError(f"the stream is on {stream.device}, the tensors are on {device}")
    return torch.cuda.stream(stream)


def _pieces(nbytes, device):
    """One uninitialised buffer cut into pieces of these sizes (multiples of 256 bytes apart): (buffer, addresses)."""
    import torch
    at, total = [], 0
    for n in nbytes:
        at.append(total)
        total += (n + 255) // 256 * 256
    buf = torch.empty(total, dtype=torch.uint8, device=device)
    base = buf.data_ptr()
    return buf, [base + a for a in at]


def _rows_apart(name, x):
    """(address, row stride) of a 2-D tensor whose rows are contiguous but may lie apart."""
    if not x.numel():
        return None, x.shape[1]
    if x.shape[1] > 1 and x.stride(1) != 1:
        raise ValueError(f"{name}: the rows must be contiguous, got strides {x.stride()}")
    return x.data_ptr(), x.stride(0) if x.shape[0] > 1 else x.shape[1]


def ckpt8_pack(x, out=None, stream=None):
    """The 8-bit checkpoint (a uint8 tensor of tpmlp_ckpt8_size bytes) of a 2-D bf16 or fp32 CUDA tensor, whose rows
    may be further apart than they are long (a column slice)."""
    import torch
    if x.dim() != 2 or x.dtype not in (torch.bfloat16, torch.float32) or not x.is_cuda:
        raise ValueError("expected a 2-D bf16 or fp32 CUDA tensor")
    rows, cols = x.shape
    src, ld = _rows_apart("x", x)
    n = tpmlp_ckpt8_size(rows, cols)
    with _on(x.device, stream):
        if out is None:
            out = torch.empty(n, dtype=torch.uint8, device=x.device)
        tpmlp_ckpt8_pack("bf16" if x.dtype == torch.bfloat16 else "fp32", rows, cols, src, ld,
                         _ptr("out", out, (n,), torch.uint8, x.device), _current(x.device))
    return out


def ckpt8_unpack(ckpt, rows: int, cols: int, dtype: str = "bf16", out=None, stream=None):
    """The [rows x cols] tensor that a checkpoint stands for; out: a tensor to write it to (rows may lie apart)."""
    import torch
    td = _tdtype(dtype)
    if not ckpt.is_cuda:
        raise ValueError("tensor must live on a CUDA device")
    src = _ptr("ckpt", ckpt, (tpmlp_ckpt8_size(rows, cols),), torch.uint8, ckpt.device)
    with _on(ckpt.device, stream):
        if out is None:
            out = torch.empty(rows, cols, dtype=td, device=ckpt.device)
        elif out.shape != (rows, cols) or out.dtype != td or out.device != ckpt.device:
            raise ValueError(f"out: expected {(rows, cols)} of {td} on {ckpt.device}, got {tuple(out.shape)} of "
                             f"{out.dtype} on {out.device}")
        dst, ld = _rows_apart("out", out)
        tpmlp_ckpt8_unpack(dtype, rows, cols, src, dst, ld, _current(ckpt.device))
    return out


class ShardedMLP:
    """Plan + workspace + output allocation for one problem shape.

    Tensors follow the C ABI: X [T, d]; W1_i, W3_i [d, d_i]; W2_i [d_i, d];
    every tensor contiguous on the current CUDA device, in the plan's dtype.
    """

    def __init__(self, T: int, d: int, d_i: Sequence[int], act: str = "gelu", dtype: str = "bf16", device=None):
        import torch
        self.plan = Plan(T, d, d_i, act, dtype)
        self.device = torch.device(device or "cuda")
        self.tdtype = {"bf16": torch.bfloat16, "fp32": torch.float32}[dtype]
        self.workspace = torch.zeros(tpmlp_workspace_size(self.plan), dtype=torch.uint8, device=self.device)
        # What the 8-bit calls check and make, worked out once: shapes of W1_i / W3_i, W2_i, biases, checkpoints; bytes
        # of one [T, d_i] array per shard.
        p = self.plan
        self._col, self._row = [(p.d, w) for w in p.d_i], [(w, p.d) for w in p.d_i]
        self._wide = [(w,) for w in p.d_i]
        self._ckpt8 = [(tpmlp_ckpt8_size(p.T, w),) for w in p.d_i] * (2 if self.swiglu else 1)
        self._act_bytes = [p.T * w * (2 if dtype == "bf16" else 4) for w in p.d_i]

    @property
    def swiglu(self) -> bool:
        return self.plan.act == "swiglu"

    def _empty(self, *shape):
        import torch
        return torch.empty(*shape, dtype=self.tdtype, device=self.device)

    def check_inputs(self, X, W1_i, W2_i, W3_i=None):
        p = self.plan
        assert tuple(X.shape) == (p.T, p.d), f"X shape {tuple(X.shape)} != {(p.T, p.d)}"
        assert len(W1_i) == p.t and len(W2_i) == p.t
        for i, w in enumerate(p.d_i):
            assert tuple(W1_i[i].shape) == (p.d, w) and tuple(W2_i[i].shape) == (w, p.d)
            if self.swiglu:
                assert tuple(W3_i[i].shape) == (p.d, w)
        for x in [X, *W1_i, *W2_i, *(W3_i or [])]:
            assert x.dtype == self.tdtype and x.is_cuda

    def alloc_forward(self):
        p = self.plan
        Y = self._empty(p.T, p.d)
        H = [self._empty(p.T, w) for w in p.d_i]
        saved = [self._empty(p.T, w) for w in p.d_i * (2 if self.swiglu else 1)]
        return Y, saved, H

    def alloc_backward(self):
        p = self.plan
        dX = self._empty(p.T, p.d)
        dact = [self._empty(p.T, w) for w in p.d_i * (2 if self.swiglu else 1)]
        dW1 = [self._empty(p.d, w) for w in p.d_i]
        dW3 = [self._empty(p.d, w) for w in p.d_i] if self.swiglu else None
        dW2 = [self._empty(w, p.d) for w in p.d_i]
        return dact, dX, dW1, dW3, dW2

    def forward(self, X, W1_i, W2_i, W3_i=None, out=None, stream=None, b1_i=None, b3_i=None, b2=None):
        """Y = sum_i act(X W1_i + b1_i) W2_i + b2 (biases optional).  Returns (Y, saved, H)."""
        self.check_inputs(X, W1_i, W2_i, W3_i)
        Y, saved, H = out if out is not None else self.alloc_forward()
        tpmlp_forward(self.plan, X, W1_i, W3_i, W2_i, b1_i, b3_i, b2, Y, saved, H, self.workspace, stream)
        return Y, saved, H

    def alloc_bias_grads(self):
        p = self.plan
        db1 = [self._empty(w) for w in p.d_i]
        db3 = [self._empty(w) for w in p.d_i] if self.swiglu else None
        return db1, db3, self._empty(p.d)

    def backward(self, X, W1_i, W2_i, saved, H, dY, W3_i=None, out=None, stream=None, bias_grads=False,
                 recompute=False):
        """Gradients of X, the weights and, with bias_grads, the biases.  With
        recompute, H is scratch (its contents are not read) and is rewritten."""
        dact, dX, dW1, dW3, dW2 = out if out is not None else self.alloc_backward()
        db1, db3, db2 = self.alloc_bias_grads() if bias_grads else (None, None, None)
        fn = tpmlp_backward_recompute if recompute else tpmlp_backward
        fn(self.plan, X, W1_i, W3_i, W2_i, saved, H, dY, dact, dX, dW1, dW3, dW2, db1, db3, db2, self.workspace,
           stream)
        return {"dX": dX, "dW1": dW1, "dW3": dW3, "dW2": dW2, "dact": dact, "db1": db1, "db3": db3, "db2": db2}

    # ---- 8-bit activation checkpoints: what backward needs of the pre-activations in 1.0625 bytes each
    def ckpt8_sizes(self):
        """Bytes of each checkpoint: one per shard (A_i), SwiGLU two (G_i, then U_i)."""
        return [n for n, in self._ckpt8]

    def _ckpt8_args(self, X, W1_i, W2_i, W3_i):
        """Checked addresses of the inputs that both passes share."""
        p, td, dev = self.plan, self.tdtype, self.workspace.device
        return (_ptr("X", X, (p.T, p.d), td, dev), _ptrs("W1_i", W1_i, self._col, td, dev),
                _ptrs("W3_i", W3_i, self._col, td, dev) if self.swiglu else None,
                _ptrs("W2_i", W2_i, self._row, td, dev))

    def forward_ckpt8(self, X, W1_i, W2_i, W3_i=None, stream=None, b1_i=None, b3_i=None, b2=None, out=None):
        """forward with the pre-activations kept as 8-bit checkpoints.  Returns (Y, ckpt); out: those two, to write
        to.  H is scratch of the call."""
        import torch
        p, td, dev = self.plan, self.tdtype, self.workspace.device
        x, w1, w3, w2 = self._ckpt8_args(X, W1_i, W2_i, W3_i)
        b1 = _ptrs("b1_i", b1_i, self._wide, td, dev) if b1_i is not None else None
        b3 = _ptrs("b3_i", b3_i, self._wide, td, dev) if b3_i is not None and self.swiglu else None
        b2 = _ptr("b2", b2, (p.d,), td, dev) if b2 is not None else None
        with _on(dev, stream):
            if out is None:
                Y = X.new_empty((p.T, p.d))
                ckpt = [X.new_empty(n, dtype=torch.uint8) for n in self._ckpt8]
                y, c = Y.data_ptr(), (ctypes.c_void_p * len(ckpt))(*[x.data_ptr() for x in ckpt])
            else:
                Y, ckpt = out
                y = _ptr("Y", Y, (p.T, p.d), td, dev)
                c = _ptrs("ckpt", ckpt, self._ckpt8, torch.uint8, dev)
            scratch, H = _pieces(self._act_bytes, dev)
            tpmlp_forward_ckpt8(p, x, w1, w3, w2, b1, b3, b2, y, c, H, self.workspace.data_ptr(), _current(dev))
        return Y, ckpt

    def backward_ckpt8(self, X, W1_i, W2_i, ckpt, dY, W3_i=None, stream=None, bias_grads=False, out=None):
        """Gradients as backward gives them (without "dact"), from the checkpoints that forward_ckpt8 wrote.  out:
        (dX, dW1, dW3, dW2) to write to (dW3: None for GeLU)."""
        import torch
        p, td, dev = self.plan, self.tdtype, self.workspace.device
        x, w1, w3, w2 = self._ckpt8_args(X, W1_i, W2_i, W3_i)
        dy = _ptr("dY", dY, (p.T, p.d), td, dev)
        c = _ptrs("ckpt", ckpt, self._ckpt8, torch.uint8, dev)
        col, row = self._col, self._row
        with _on(dev, stream):
            if out is None:
                dX = X.new_empty((p.T, p.d))
                (dW1, to1), (dW2, to2) = _new_list(X, col), _new_list(X, row)
                dW3, to3 = _new_list(X, col) if self.swiglu else (None, None)
                to = dX.data_ptr(), to1, to3, to2
            else:
                dX, dW1, dW3, dW2 = out
                to = (_ptr("dX", dX, (p.T, p.d), td, dev), _ptrs("dW1", dW1, col, td, dev),
                      _ptrs("dW3", dW3, col, td, dev) if self.swiglu else None, _ptrs("dW2", dW2, row, td, dev))
            db1 = db3 = db2 = None
            db = (None, None, None)
            if bias_grads:
                db2 = X.new_empty(p.d)
                db1, to1 = _new_list(X, self._wide)
                db3, to3 = _new_list(X, self._wide) if self.swiglu else (None, None)
                db = to1, to3, db2.data_ptr()
            scratch, at = _pieces(self._act_bytes * (3 if self.swiglu else 2), dev)  # H_i, then dact
            tpmlp_backward_ckpt8(p, x, w1, w3, w2, c, at[:p.t], dy, at[p.t:], *to, *db, self.workspace.data_ptr(),
                                 _current(dev))
        return {"dX": dX, "dW1": dW1, "dW3": dW3, "dW2": dW2, "db1": db1, "db3": db3, "db2": db2}

    def check(self, stream=None):
        tpmlp_check(self.plan, self.workspace, stream)

    # ---- sequence-parallel layout: X, dY in and Y, dX out as token stripes
    def set_sequence_stripes(self, stripe_rows: Sequence[int]):
        tpmlp_plan_set_sequence_stripes(self.plan, stripe_rows)

    def alloc_stripes(self):
        return [self._empty(r, self.plan.d) for r in self.plan.stripe_rows]

    def forward_sp(self, X_stripes, W1_i, W2_i, W3_i=None, stream=None, b1_i=None, b3_i=None, b2=None):
        """Y stripes = reduce-scatter of sum_i act(X W1_i + b1_i) W2_i (+ b2), X gathered from its stripes.
        Returns (Y_stripes, saved, H)."""
        Y_j = self.alloc_stripes()
        _, saved, H = self.alloc_forward()
        tpmlp_forward_sp(self.plan, X_stripes, W1_i, W3_i, W2_i, b1_i, b3_i, b2, Y_j, saved, H, self.workspace,
                         stream)
        return Y_j, saved, H

    def backward_sp(self, X_stripes, W1_i, W2_i, saved, H, dY_stripes, W3_i=None, stream=None, bias_grads=False):
        dact, _, dW1, dW3, dW2 = self.alloc_backward()
        dX_j = self.alloc_stripes()
        db1, db3, db2 = self.alloc_bias_grads() if bias_grads else (None, None, None)
        tpmlp_backward_sp(self.plan, X_stripes, W1_i, W3_i, W2_i, saved, H, dY_stripes, dact, dX_j, dW1, dW3, dW2,
                          db1, db3, db2, self.workspace, stream)
        return {"dX_stripes": dX_j, "dW1": dW1, "dW3": dW3, "dW2": dW2, "dact": dact, "db1": db1, "db3": db3,
                "db2": db2}


# Partial sums of the gains' gradients in an fp32 plan's workspace at most: CTAs of a launch x head_dim.
_GAIN_SUMS_BYTES = 4096 * 256 * 4


class ShardedAttentionProj:
    """Attention plan + workspace + output allocation for one shape.

    Tensors follow the C ABI: X [T, d]; Wqkv_i [d, n_i] = [WQ_i | WK_i | WV_i];
    QKV_i [T, n_i]; O_i [T, dq_i]; WO_i [dq_i, d]; Z [T, d].
    """

    def __init__(self, T: int, d: int, dq_i: Sequence[int], dkv_i: Sequence[int], dtype: str = "bf16",
                 device=None):
        import torch
        self.plan = AttnPlan(T, d, dq_i, dkv_i, dtype)
        self.device = torch.device(device or "cuda")
        self.tdtype = {"bf16": torch.bfloat16, "fp32": torch.float32}[dtype]
        # Of the size that the largest head_dim asks for, so that set_qk_norm_rope never replaces it: kernels in flight
        # and captured graphs keep its address.
        n = tpmlp_workspace_size(self.plan)
        self.workspace = torch.zeros(max(n, 256 + _GAIN_SUMS_BYTES), dtype=torch.uint8, device=self.device)
        p = self.plan  # shapes of QKV_i, [Q_i | K_i] and V_i
        self._fused, self._v = [(p.T, n) for n in p.d_i], [(p.T, k) for k in p.dkv_i]
        self._qk = [(p.T, q + k) for q, k in zip(p.dq_i, p.dkv_i)]

    def _empty(self, *shape):
        import torch
        return torch.empty(*shape, dtype=self.tdtype, device=self.device)

    def qkv_forward(self, X, Wqkv_i, out=None, stream=None):
        p = self.plan
        QKV = out if out is not None else [self._empty(p.T, n) for n in p.d_i]
        tpmlp_attn_qkv_forward(p, X, Wqkv_i, QKV, self.workspace, stream)
        return QKV

    def out_forward(self, WO_i, O_i, out=None, stream=None):
        Z = out if out is not None else self._empty(self.plan.T, self.plan.d)
        tpmlp_attn_out_forward(self.plan, WO_i, O_i, Z, self.workspace, stream)
        return Z

    def out_backward(self, WO_i, O_i, dZ, out=None, stream=None):
        p = self.plan
        dO, dWO = out if out is not None else ([self._empty(p.T, q) for q in p.dq_i],
                                               [self._empty(q, p.d) for q in p.dq_i])
        tpmlp_attn_out_backward(p, WO_i, O_i, dZ, dO, dWO, self.workspace, stream)
        return dO, dWO

    def qkv_backward(self, X, Wqkv_i, dQKV_i, out=None, stream=None):
        p = self.plan
        dX, dWqkv = out if out is not None else (self._empty(p.T, p.d), [self._empty(p.d, n) for n in p.d_i])
        tpmlp_attn_qkv_backward(p, X, Wqkv_i, dQKV_i, dX, dWqkv, self.workspace, stream)
        return dX, dWqkv

    # ---- norm of the query and key heads with the position rotation
    def set_qk_norm_rope(self, head_dim, rotary_dim=None, layout="halves", norm=True, eps=1e-6, base=10000.0,
                         inv_freq=None):
        tpmlp_attn_plan_set_qk_norm_rope(self.plan, head_dim, rotary_dim, layout, norm, eps, base, inv_freq)

    def _qk_args(self, QKV_i, positions, gq, gk, may_lack_x=False):
        """Checked addresses of the inputs that both passes share."""
        p, td, dev = self.plan, self.tdtype, self.workspace.device
        D = getattr(p, "head_dim", 0)
        if not D:
            raise ValueError("the heads are not described (set_qk_norm_rope)")
        import torch
        return (_ptrs("QKV_i", QKV_i, self._fused, td, dev) if QKV_i is not None or not may_lack_x else None,
                _ptr("positions", positions, (p.T,), torch.int64, dev) if positions is not None else None,
                _ptr("gq", gq, (D,), td, dev) if gq is not None else None,
                _ptr("gk", gk, (D,), td, dev) if gk is not None else None)

    def _in_place_or_dense(self, name, xs, fused):
        """[T, dq_i + dkv_i] tensors, or the [T, n_i] ones at the addresses `fused`."""
        p = self.plan
        if len(xs) != p.t:
            raise ValueError(f"{name}: expected {p.t} tensors, got {len(xs)}")
        shapes = [n if p.T and x.data_ptr() == f else qk for x, f, n, qk in zip(xs, fused, self._fused, self._qk)]
        return _ptrs(name, xs, shapes, self.tdtype, self.workspace.device)

    def qk_norm_rope_forward(self, QKV_i, positions=None, gq=None, gk=None, out=None, stream=None):
        """The normed and rotated heads [Q_i | K_i] of each shard.  out: [T, dq_i + dkv_i] tensors, or QKV_i itself
        (in place: the value columns stay as they are)."""
        p = self.plan
        qkv, pos, q, k = self._qk_args(QKV_i, positions, gq, gk)
        with _on(self.workspace.device, stream):
            if out is None:
                out, to = _new_list(QKV_i[0], self._qk)
            else:
                to = self._in_place_or_dense("out", out, qkv)
            tpmlp_attn_qk_norm_rope_forward(p, qkv, pos, q, k, to, _current(self.workspace.device))
        return out

    def qk_norm_rope_backward(self, QKV_i, dQK_i, positions=None, gq=None, gk=None, dV_i=None, out=None, stream=None,
                              gain_grads=None):
        """(dQKV_i, dgq, dgk) from the core's [dQ_i | dK_i] and, optionally, dV_i [T, dkv_i].  out: the dQKV_i to
        write to; their value columns stay as they are without dV_i.  dQK_i may be those tensors themselves.
        gain_grads: whether to compute dgq and dgk (None: if a gain is given).  Without a norm QKV_i is not read and may
        be None."""
        p, td, dev = self.plan, self.tdtype, self.workspace.device
        qkv, pos, q, k = self._qk_args(QKV_i, positions, gq, gk, may_lack_x=not getattr(p, "qk_norm", True))
        dv = _ptrs("dV_i", dV_i, self._v, td, dev) if dV_i is not None else None
        if dV_i is None and out is None:
            raise ValueError("dV_i, or dQKV_i that hold dV already (out), must be given")
        if gain_grads is None:
            gain_grads = gq is not None or gk is not None
        with _on(dev, stream):
            like = QKV_i[0] if QKV_i is not None else self.workspace.new_empty(0, dtype=td)
            if out is None:
                out, dqkv = _new_list(like, self._fused)
            else:
                dqkv = _ptrs("out", out, self._fused, td, dev)
            dgq = dgk = None
            if gain_grads:
                dgq, dgk = like.new_empty(p.head_dim), like.new_empty(p.head_dim)
            tpmlp_attn_qk_norm_rope_backward(p, qkv, pos, q, k, self._in_place_or_dense("dQK_i", dQK_i, dqkv), dv,
                                             dqkv, dgq, dgk, self.workspace, _current(dev))
        return out, dgq, dgk

    def check(self, stream=None):
        tpmlp_check(self.plan, self.workspace, stream)


def _make_function():
    import torch

    class TPMLPFunction(torch.autograd.Function):
        """Y = TPMLPFunction.apply(mlp, X, *W1_i, *W2_i[, *W3_i]) with the library's backward."""

        @staticmethod
        def forward(ctx, mlp: ShardedMLP, X, *weights):
            t = mlp.plan.t
            W1_i, W2_i = list(weights[:t]), list(weights[t:2 * t])
            W3_i = list(weights[2 * t:3 * t]) if mlp.swiglu else None
            Y, saved, H = mlp.forward(X.contiguous(), W1_i, W2_i, W3_i)
            ctx.mlp = mlp
            ctx.save_for_backward(X, *weights, *saved, *H)
            return Y

        @staticmethod
        def backward(ctx, dY):
            mlp = ctx.mlp
            t = mlp.plan.t
            ns = 2 * t if mlp.swiglu else t
            tensors = ctx.saved_tensors
            X = tensors[0]
            nw = 3 * t if mlp.swiglu else 2 * t
            weights = list(tensors[1:1 + nw])
            saved = list(tensors[1 + nw:1 + nw + ns])
            H = list(tensors[1 + nw + ns:])
            W1_i, W2_i = weights[:t], weights[t:2 * t]
            W3_i = weights[2 * t:] if mlp.swiglu else None
            g = mlp.backward(X, W1_i, W2_i, saved, H, dY.contiguous(), W3_i)
            grads = g["dW1"] + g["dW2"] + (g["dW3"] if mlp.swiglu else [])
            return (None, g["dX"], *grads)

    return TPMLPFunction


def _make_checkpoint_function():
    import torch

    class TPMLPCheckpointFunction(torch.autograd.Function):
        """TPMLPFunction with the pre-activations kept as 8-bit checkpoints between the passes: it saves X, the
        weights and 1.0625 bytes per pre-activation.  Without biases, as TPMLPFunction; any other number of weights is
        refused.

        In a CUDA graph capture, capture forward and backward together, and let no eager autograd graph of the same
        leaves be alive then: autograd accumulates a leaf's gradient on the stream of the first graph that used it,
        which a capture cannot take in.  ShardedMLP.forward_ckpt8 and backward_ckpt8 know no such thing."""

        @staticmethod
        def forward(ctx, mlp: ShardedMLP, X, *weights):
            t = mlp.plan.t
            n = (3 if mlp.swiglu else 2) * t
            if len(weights) != n:  # no biases here: a longer list would be computed without its rest
                names = "W1_i, W2_i, W3_i" if mlp.swiglu else "W1_i, W2_i"
                raise ValueError(f"expected {n} weights ({names}), got {len(weights)}")
            X = X.contiguous()
            W3_i = list(weights[2 * t:3 * t]) if mlp.swiglu else None
            Y, ckpt = mlp.forward_ckpt8(X, list(weights[:t]), list(weights[t:2 * t]), W3_i)
            ctx.mlp, ctx.nw = mlp, len(weights)
            ctx.save_for_backward(X, *weights, *ckpt)
            return Y

        @staticmethod
        @torch.autograd.function.once_differentiable
        def backward(ctx, dY):
            mlp, nw = ctx.mlp, ctx.nw
            t = mlp.plan.t
            X, *rest = ctx.saved_tensors
            weights, ckpt = rest[:nw], rest[nw:]
            W3_i = weights[2 * t:] if mlp.swiglu else None
            g = mlp.backward_ckpt8(X, weights[:t], weights[t:2 * t], ckpt, dY.contiguous(), W3_i)
            return (None, g["dX"], *g["dW1"], *g["dW2"], *(g["dW3"] if mlp.swiglu else []))

    return TPMLPCheckpointFunction


class _LazyFunction:
    """An autograd function that is made, and torch imported, on its first use.  What was made stays with the class, so
    that a copy of the object, or one that was pickled, is as good as the object."""

    _make, _fn = staticmethod(_make_function), None

    def __getattr__(self, name):
        cls = type(self)
        if cls._fn is None:
            cls._fn = cls._make()
        return getattr(cls._fn, name)


class _LazyCheckpointFunction(_LazyFunction):
    _make, _fn = staticmethod(_make_checkpoint_function), None


TPMLPFunction = _LazyFunction()
TPMLPCheckpointFunction = _LazyCheckpointFunction()
