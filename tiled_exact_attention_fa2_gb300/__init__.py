"""GB300 (sm_103a) FlashAttention-2: thin Python binding of the C ABI in include/fa2.h.

Every step of the computation runs in the CUDA kernels of
``libfa2_gb300.so``; this module only checks tensor metadata, allocates
outputs with torch and passes raw pointers, sizes and the current CUDA stream.
There is no fallback: if the shared library is missing, every call raises.

Build the library with ``python -c "import __graft_entry__ as g; g.build()"``
(or ``python tiled_exact_attention_fa2_gb300/_build.py``).
"""
from __future__ import annotations

import ctypes
import functools
import inspect
import math
import os
import struct
from typing import NamedTuple, Optional, Tuple

import torch

from . import _build

__all__ = [
    "FA2Error", "load_library", "fa2_fwd", "fa2_fwd_ws", "fa2_fwd_workspace_bytes", "fa2_bwd", "fa2_bwd_ws", "fa2_bwd_workspace_bytes",
    "fa2_status_string", "fa2_device_status", "fa2_abi_version", "fa2_step_from_host",
    "fa2_step_from_host_workspace_bytes",
    "fa2_bwd_stages", "fa2_bwd_noalloc", "fa2_fwd_gqa", "fa2_bwd_gqa", "fa2_fwd_splitkv",
    "fa2_fwd_varlen", "fa2_bwd_varlen", "prepared_step", "FA2_OK",
    "fa2_qk_norm_rope", "fa2_qk_norm_rope_bwd", "fa2_page_plan", "PagePlan", "fa2_kv4_cache", "fa2_kv4_page_bytes",
    "fa2_kv4_append", "fa2_kv4_gather", "fa2_kv4_attn", "fa2_kv4_attn_workspace_bytes",
]

FA2_OK = 0
_LIB: Optional[ctypes.CDLL] = None

_vp = ctypes.c_void_p
_i = ctypes.c_int
_f = ctypes.c_float
_sz = ctypes.c_size_t
_ll = ctypes.c_longlong

_SIGNATURES = {
    "fa2_fwd": (_i, [_vp, _vp, _vp, _vp, _vp, _i, _i, _i, _i, _f, _i, _vp]),
    "fa2_fwd_ws": (_i, [_vp, _vp, _vp, _vp, _vp, _i, _i, _i, _i, _f, _i, _vp, _sz, _vp]),
    "fa2_fwd_workspace_bytes": (_sz, [_i, _i, _i, _i]),
    "fa2_fwd_gqa_ws": (_i, [_vp, _vp, _vp, _vp, _vp, _i, _i, _i, _i, _i, _f, _i, _vp, _sz, _vp]),
    "fa2_bwd": (_i, [_vp, _vp, _vp, _vp, _vp, _vp, _vp, _vp, _vp, _i, _i, _i, _i, _f, _i, _vp]),
    "fa2_bwd_ws": (_i, [_vp, _vp, _vp, _vp, _vp, _vp, _vp, _vp, _vp, _i, _i, _i, _i, _f, _i, _vp, _sz, _vp]),
    "fa2_bwd_workspace_bytes": (_sz, [_i, _i, _i, _i]),
    "fa2_status_string": (ctypes.c_char_p, [_i]),
    "fa2_device_status": (_i, [ctypes.POINTER(_i), _i]),
    "fa2_abi_version": (_i, []),
    "fa2_bwd_preprocess": (_i, [_vp, _vp, _vp, _vp, _i, _i, _i, _i, _vp]),
    "fa2_bwd_main": (_i, [_vp, _vp, _vp, _vp, _vp, _vp, _vp, _vp, _vp, _i, _i, _i, _i, _f, _i, _vp]),
    "fa2_bwd_dq_convert": (_i, [_vp, _vp, _i, _i, _i, _i, _f, _vp]),
    "fa2_bwd_main_dq": (_i, [_vp, _vp, _vp, _vp, _vp, _vp, _vp, _vp, _vp, _i, _i, _i, _i, _f, _i, _i, _vp]),
    "fa2_bwd_dq_partials_bytes": (_sz, [_i, _i, _i, _i, _i]),
    "fa2_bwd_dq_reduce": (_i, [_vp, _vp, _i, _i, _i, _i, _f, _i, _vp]),
    "fa2_bwd_deterministic_workspace_bytes": (_sz, [_i, _i, _i, _i, _i]),
    "fa2_bwd_deterministic": (_i, [_vp, _vp, _vp, _vp, _vp, _vp, _vp, _vp, _vp, _i, _i, _i, _i, _f, _i, _vp, _sz,
                                   _vp]),
    "fa2_last_error_detail": (ctypes.c_char_p, []),
    "fa2_bwd_noalloc": (_i, [_vp, _vp, _vp, _vp, _vp, _vp, _vp, _vp, _vp, _i, _i, _i, _i, _f, _i, _vp]),
    "fa2_noalloc_scratch_capacity": (_sz, []),
    "fa2_step_from_host_workspace_bytes": (_sz, [_i, _i, _i, _i, ctypes.POINTER(_i), _i, _i]),
    "fa2_step_from_host": (_i, [_vp, _vp, _vp, _vp, _vp, _vp, _vp, _vp, _vp, _i, _i, _i, _i, _f, _i,
                                ctypes.POINTER(_i), _i, _i, _vp, _sz, _vp]),
    "fa2_fwd_gqa": (_i, [_vp, _vp, _vp, _vp, _vp, _i, _i, _i, _i, _i, _f, _i, _vp]),
    "fa2_bwd_gqa": (_i, [_vp, _vp, _vp, _vp, _vp, _vp, _vp, _vp, _vp, _i, _i, _i, _i, _i, _f, _i, _vp]),
    "fa2_bwd_gqa_ws": (_i, [_vp, _vp, _vp, _vp, _vp, _vp, _vp, _vp, _vp, _i, _i, _i, _i, _i, _f, _i, _vp, _sz,
                            _vp]),
    "fa2_check_wait_timeout": (_i, [_i, ctypes.POINTER(_i)]),
    "fa2_check_warp_wait": (_i, [_i, ctypes.POINTER(ctypes.c_uint)]),
    "fa2_fwd_splitkv_workspace_bytes": (_sz, [_i, _i, _i, _i, _i, _i]),
    "fa2_fwd_splitkv_suggest_splits": (_i, [_i, _i, _i, _i, _i, _i]),
    "fa2_fwd_splitkv": (_i, [_vp, _vp, _vp, _vp, _vp, _i, _i, _i, _i, _i, _i, _f, _i, _i, _vp, _sz, _vp]),
    "fa2_fwd_varlen": (_i, [_vp, _vp, _vp, _vp, _vp, _vp, _vp, _i, _i, _i, _i, _i, _i, _i, _i, _f, _i, _vp]),
    "fa2_bwd_varlen_workspace_bytes": (_sz, [_i, _i, _i]),
    "fa2_bwd_varlen": (_i, [_vp, _vp, _vp, _vp, _vp, _vp, _vp, _vp, _vp, _vp, _vp, _i, _i, _i, _i, _i, _i, _i, _i,
                            _f, _i, _vp, _sz, _vp]),
    "fa2_qk_norm_rope": (_i, [_vp, _vp, _vp, _vp, _i, _vp, _vp, _vp, _vp, _i, _i, _i, _i, _i, _i, _i, _i, _f, _vp, _vp]),
    "fa2_qk_norm_rope_bwd_workspace_bytes": (_sz, [_i]),
    "fa2_qk_norm_rope_bwd": (_i, [_vp, _vp, _vp, _vp, _vp, _vp, _i, _vp, _vp, _vp, _vp, _vp, _vp, _i, _i, _i, _i, _i, _i,
                                  _i, _i, _f, _vp, _vp, _sz, _vp]),
    "fa2_page_plan": (_i, [_vp, _vp, _vp, _vp, _vp, _vp, _vp, _vp, _vp, _vp, _i, _i, _i, _ll, _i, _i, _vp]),
    "fa2_kv4_page_bytes": (_sz, [_i, _i, _i]),
    "fa2_kv4_append": (_i, [_vp, _vp, _vp, _vp, _ll, _vp, _vp, _vp, _i, _i, _i, _i, _i, _f, _f, _vp]),
    "fa2_kv4_gather": (_i, [_vp, _ll, _vp, _ll, _vp, _vp, _vp, _i, _i, _i, _i, _i, _i, _i, _f, _f, _vp]),
    "fa2_kv4_attn_workspace_bytes": (_sz, [_i, _i, _i, _i, _i, _i]),
    "fa2_kv4_attn": (_i, [_vp, _vp, _ll, _vp, _ll, _vp, _vp, _vp, _vp, _i, _i, _i, _i, _i, _i, _i, _i, _i, _i, _f, _f, _f,
                          _i, _vp, _sz, _vp]),
}


class FA2Error(RuntimeError):
    def __init__(self, fn: str, status: int):
        self.status = status
        detail = load_library().fa2_last_error_detail().decode() if status in (6, 7) else ""
        super().__init__(f"{fn} failed with status {status}: {fa2_status_string(status)}"
                         + (f" [{detail}]" if detail else ""))


def load_library(path: Optional[str] = None) -> ctypes.CDLL:
    """Load libfa2_gb300.so (raises if it has not been built)."""
    global _LIB
    if _LIB is not None and path is None:
        return _LIB
    path = path or _build.LIB_PATH
    if not os.path.exists(path):
        raise RuntimeError(
            f"{os.path.basename(path)} is not built; run `python -c \"import __graft_entry__ as g; g.build()\"`")
    lib = ctypes.CDLL(path)
    for name, (res, args) in _SIGNATURES.items():
        fn = getattr(lib, name)
        fn.restype = res
        fn.argtypes = args
    if path == _build.LIB_PATH:
        _LIB = lib
    return lib


def fa2_status_string(status: int) -> str:
    return load_library().fa2_status_string(int(status)).decode()


def fa2_abi_version() -> int:
    return load_library().fa2_abi_version()


def fa2_device_status(reset: bool = False) -> int:
    """Device status word of the kernels (0 = every internal wait completed)."""
    v = _i(0)
    rc = load_library().fa2_device_status(ctypes.byref(v), 1 if reset else 0)
    if rc != FA2_OK:
        raise FA2Error("fa2_device_status", rc)
    return v.value


def fa2_bwd_workspace_bytes(B: int, H: int, N: int, d: int) -> int:
    return load_library().fa2_bwd_workspace_bytes(B, H, N, d)


def _shape(t: torch.Tensor, name: str):
    if t.dim() != 4:
        raise ValueError(f"{name} must be [B, H, N, d], got {tuple(t.shape)}")
    if t.dtype != torch.bfloat16:
        raise ValueError(f"{name} must be bfloat16, got {t.dtype}")
    if not t.is_cuda:
        raise ValueError(f"{name} must be a CUDA tensor")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    return tuple(t.shape)


def _stream(stream, device) -> int:
    if stream is None:
        return torch.cuda.current_stream(device).cuda_stream
    if isinstance(stream, torch.cuda.Stream):
        if device.index is not None and stream.device_index != device.index:
            raise ValueError(f"the stream belongs to cuda:{stream.device_index}, the tensors to {device}")
        return stream.cuda_stream
    return int(stream)


class _on:
    """`device` current, and the given stream torch's current one, so that what a call allocates belongs to the stream
    that uses it."""

    def __init__(self, device, stream):
        if isinstance(stream, torch.cuda.Stream) and stream.device_index != device:
            raise ValueError(f"the stream belongs to cuda:{stream.device_index}, the tensors to cuda:{device}")
        self.guards = [torch.cuda.device(device)]
        if stream is not None:
            if not isinstance(stream, torch.cuda.Stream):
                # (1 is cudaStreamLegacy, which torch would take for a number of its own)
                handle = int(stream)
                stream = torch.cuda.default_stream(device) if handle in (0, 1) else torch.cuda.ExternalStream(handle, device=device)
            self.guards.append(torch.cuda.stream(stream))

    def __enter__(self):
        for g in self.guards:
            g.__enter__()

    def __exit__(self, *exc):
        for g in reversed(self.guards):
            g.__exit__(*exc)


def _made_on_stream(fn):
    """The call made on the `stream` that it is given: what it allocates (outputs, scratch that is freed when it returns)
    belongs to that stream, so no other stream's work is given the memory while this call's is under way."""
    at = list(inspect.signature(fn).parameters).index("stream")

    @functools.wraps(fn)
    def call(*args, **kwargs):
        stream = args[at] if len(args) > at else kwargs.get("stream")
        q = args[0] if args else kwargs.get("q")
        if stream is None or not q.is_cuda:
            return fn(*args, **kwargs)
        with _on(q.get_device(), stream):
            return fn(*args, **kwargs)

    return call


def _scale(scale, d):
    return 1.0 / math.sqrt(d) if scale is None else float(scale)


@_made_on_stream
def fa2_fwd(q: torch.Tensor, k: torch.Tensor, v: torch.Tensor, o: Optional[torch.Tensor] = None,
            lse: Optional[torch.Tensor] = None, scale: Optional[float] = None, causal: bool = True,
            stream=None) -> Tuple[torch.Tensor, torch.Tensor]:
    """O [B,H,N,d] bf16 and LSE [B,H,N] fp32 of softmax(scale Q K^T) V."""
    lib = load_library()
    B, H, N, d = _shape(q, "q")
    if _shape(k, "k") != (B, H, N, d) or _shape(v, "v") != (B, H, N, d):
        raise ValueError("q, k and v must have the same shape")
    if o is None:
        o = torch.empty_like(q)
    if lse is None:
        lse = torch.empty((B, H, N), dtype=torch.float32, device=q.device)
    if lse.dtype != torch.float32 or not lse.is_contiguous() or tuple(lse.shape) != (B, H, N):
        raise ValueError("lse must be a contiguous fp32 [B, H, N] tensor")
    _shape(o, "o")
    rc = lib.fa2_fwd(q.data_ptr(), k.data_ptr(), v.data_ptr(), o.data_ptr(), lse.data_ptr(), B, H, N, d,
                     _scale(scale, d), 1 if causal else 0, _stream(stream, q.device))
    if rc != FA2_OK:
        raise FA2Error("fa2_fwd", rc)
    return o, lse


def fa2_fwd_workspace_bytes(B: int, H_kv: int, N: int, d: int) -> int:
    return load_library().fa2_fwd_workspace_bytes(B, H_kv, N, d)


@_made_on_stream
def fa2_fwd_ws(q: torch.Tensor, k: torch.Tensor, v: torch.Tensor, workspace: torch.Tensor,
               o: Optional[torch.Tensor] = None, lse: Optional[torch.Tensor] = None, scale: Optional[float] = None,
               causal: bool = True, stream=None) -> Tuple[torch.Tensor, torch.Tensor]:
    """fa2_fwd with caller-owned scratch (a CUDA byte tensor of fa2_fwd_workspace_bytes bytes)."""
    lib = load_library()
    B, H, N, d = _shape(q, "q")
    if _shape(k, "k") != (B, H, N, d) or _shape(v, "v") != (B, H, N, d):
        raise ValueError("q, k and v must have the same shape")
    o = torch.empty_like(q) if o is None else o
    lse = torch.empty((B, H, N), dtype=torch.float32, device=q.device) if lse is None else lse
    if lse.dtype != torch.float32 or not lse.is_contiguous() or tuple(lse.shape) != (B, H, N):
        raise ValueError("lse must be a contiguous fp32 [B, H, N] tensor")
    _shape(o, "o")
    rc = lib.fa2_fwd_ws(q.data_ptr(), k.data_ptr(), v.data_ptr(), o.data_ptr(), lse.data_ptr(), B, H, N, d,
                        _scale(scale, d), 1 if causal else 0, workspace.data_ptr(),
                        workspace.numel() * workspace.element_size(), _stream(stream, q.device))
    if rc != FA2_OK:
        raise FA2Error("fa2_fwd_ws", rc)
    return o, lse


def _bwd_common(q, k, v, o, dO, lse, dq, dk, dv):
    B, H, N, d = _shape(q, "q")
    for name, t in (("k", k), ("v", v), ("o", o), ("dO", dO)):
        if _shape(t, name) != (B, H, N, d):
            raise ValueError(f"{name} must have q's shape")
    if lse.dtype != torch.float32 or not lse.is_contiguous() or tuple(lse.shape) != (B, H, N):
        raise ValueError("lse must be a contiguous fp32 [B, H, N] tensor")
    dq = torch.empty_like(q) if dq is None else dq
    dk = torch.empty_like(k) if dk is None else dk
    dv = torch.empty_like(v) if dv is None else dv
    for name, t in (("dq", dq), ("dk", dk), ("dv", dv)):
        _shape(t, name)
    return (B, H, N, d), dq, dk, dv


@_made_on_stream
def fa2_bwd(q, k, v, o, dO, lse, dq=None, dk=None, dv=None, scale: Optional[float] = None,
            causal: bool = True, stream=None):
    """dQ, dK, dV (bf16) of L with dL/dO = dO; scratch is allocated stream-ordered inside the library."""
    lib = load_library()
    (B, H, N, d), dq, dk, dv = _bwd_common(q, k, v, o, dO, lse, dq, dk, dv)
    rc = lib.fa2_bwd(q.data_ptr(), k.data_ptr(), v.data_ptr(), o.data_ptr(), dO.data_ptr(), lse.data_ptr(),
                     dq.data_ptr(), dk.data_ptr(), dv.data_ptr(), B, H, N, d, _scale(scale, d),
                     1 if causal else 0, _stream(stream, q.device))
    if rc != FA2_OK:
        raise FA2Error("fa2_bwd", rc)
    return dq, dk, dv


@_made_on_stream
def fa2_bwd_ws(q, k, v, o, dO, lse, workspace: torch.Tensor, dq=None, dk=None, dv=None,
               scale: Optional[float] = None, causal: bool = True, stream=None):
    """fa2_bwd with caller-owned scratch (a CUDA byte tensor of fa2_bwd_workspace_bytes bytes)."""
    lib = load_library()
    (B, H, N, d), dq, dk, dv = _bwd_common(q, k, v, o, dO, lse, dq, dk, dv)
    rc = lib.fa2_bwd_ws(q.data_ptr(), k.data_ptr(), v.data_ptr(), o.data_ptr(), dO.data_ptr(), lse.data_ptr(),
                        dq.data_ptr(), dk.data_ptr(), dv.data_ptr(), B, H, N, d, _scale(scale, d),
                        1 if causal else 0, workspace.data_ptr(), workspace.numel() * workspace.element_size(),
                        _stream(stream, q.device))
    if rc != FA2_OK:
        raise FA2Error("fa2_bwd_ws", rc)
    return dq, dk, dv


def prepared_step(q, k, v, o, lse, dO, dq, dk, dv, fwd_workspace: torch.Tensor, bwd_workspace: torch.Tensor,
                  scale: Optional[float] = None, causal: bool = True, stream=None):
    """A callable that enqueues fa2_fwd_ws then fa2_bwd_ws on fixed buffers.

    Every argument is checked and converted to its C type once, here; each
    call of the returned function makes the two C calls with those values
    (which still validate their arguments).  For loops that run the same
    small problem many times, where marshalling arguments in Python would
    take as long as the kernels.  The tensors must stay alive (and in place)
    for as long as the callable is used.
    """
    lib = load_library()
    B, H, N, d = _shape(q, "q")
    if _shape(k, "k") != (B, H, N, d) or _shape(v, "v") != (B, H, N, d):
        raise ValueError("q, k and v must have the same shape")
    _shape(o, "o")
    _bwd_common(q, k, v, o, dO, lse, dq, dk, dv)
    vp, ci, cf, cs = ctypes.c_void_p, ctypes.c_int, ctypes.c_float, ctypes.c_size_t
    sc, cz, st = cf(_scale(scale, d)), ci(1 if causal else 0), vp(_stream(stream, q.device))
    dims = (ci(B), ci(H), ci(N), ci(d))
    fargs = (vp(q.data_ptr()), vp(k.data_ptr()), vp(v.data_ptr()), vp(o.data_ptr()), vp(lse.data_ptr()), *dims,
             sc, cz, vp(fwd_workspace.data_ptr()), cs(fwd_workspace.numel() * fwd_workspace.element_size()), st)
    bargs = (vp(q.data_ptr()), vp(k.data_ptr()), vp(v.data_ptr()), vp(o.data_ptr()), vp(dO.data_ptr()),
             vp(lse.data_ptr()), vp(dq.data_ptr()), vp(dk.data_ptr()), vp(dv.data_ptr()), *dims, sc, cz,
             vp(bwd_workspace.data_ptr()), cs(bwd_workspace.numel() * bwd_workspace.element_size()), st)
    fwd, bwd = lib.fa2_fwd_ws, lib.fa2_bwd_ws

    def step():
        rc = fwd(*fargs)
        if rc != FA2_OK:
            raise FA2Error("fa2_fwd_ws", rc)
        rc = bwd(*bargs)
        if rc != FA2_OK:
            raise FA2Error("fa2_bwd_ws", rc)

    return step


def _gqa_shapes(q, k, v):
    B, H, N, d = _shape(q, "q")
    Bk, Hkv, Nk, dk_ = _shape(k, "k")
    if (Bk, Nk, dk_) != (B, N, d) or _shape(v, "v") != (B, Hkv, N, d):
        raise ValueError("k and v must be [B, H_kv, N, d] with q's B, N and d")
    return B, H, Hkv, N, d


@_made_on_stream
def fa2_fwd_gqa(q, k, v, o=None, lse=None, scale: Optional[float] = None, causal: bool = True, stream=None):
    """Grouped-query forward: q [B,H,N,d], k/v [B,H_kv,N,d]; query head h reads K/V head h // (H // H_kv)."""
    lib = load_library()
    B, H, Hkv, N, d = _gqa_shapes(q, k, v)
    o = torch.empty_like(q) if o is None else o
    lse = torch.empty((B, H, N), dtype=torch.float32, device=q.device) if lse is None else lse
    _shape(o, "o")
    if lse.dtype != torch.float32 or not lse.is_contiguous() or tuple(lse.shape) != (B, H, N):
        raise ValueError("lse must be a contiguous fp32 [B, H, N] tensor")
    rc = lib.fa2_fwd_gqa(q.data_ptr(), k.data_ptr(), v.data_ptr(), o.data_ptr(), lse.data_ptr(), B, H, Hkv, N, d,
                         _scale(scale, d), 1 if causal else 0, _stream(stream, q.device))
    if rc != FA2_OK:
        raise FA2Error("fa2_fwd_gqa", rc)
    return o, lse


@_made_on_stream
def fa2_bwd_gqa(q, k, v, o, dO, lse, dq=None, dk=None, dv=None, scale: Optional[float] = None,
                causal: bool = True, stream=None):
    """Grouped-query backward: dk/dv [B,H_kv,N,d] are sums over each group of query heads."""
    lib = load_library()
    B, H, Hkv, N, d = _gqa_shapes(q, k, v)
    for name, t in (("o", o), ("dO", dO)):
        if _shape(t, name) != (B, H, N, d):
            raise ValueError(f"{name} must have q's shape")
    if lse.dtype != torch.float32 or not lse.is_contiguous() or tuple(lse.shape) != (B, H, N):
        raise ValueError("lse must be a contiguous fp32 [B, H, N] tensor")
    dq = torch.empty_like(q) if dq is None else dq
    dk = torch.empty_like(k) if dk is None else dk
    dv = torch.empty_like(v) if dv is None else dv
    rc = lib.fa2_bwd_gqa(q.data_ptr(), k.data_ptr(), v.data_ptr(), o.data_ptr(), dO.data_ptr(), lse.data_ptr(),
                         dq.data_ptr(), dk.data_ptr(), dv.data_ptr(), B, H, Hkv, N, d, _scale(scale, d),
                         1 if causal else 0, _stream(stream, q.device))
    if rc != FA2_OK:
        raise FA2Error("fa2_bwd_gqa", rc)
    return dq, dk, dv


@_made_on_stream
def fa2_fwd_splitkv(q, k, v, num_splits: Optional[int] = None, o=None, lse=None, workspace=None,
                    scale: Optional[float] = None, causal: bool = True, stream=None):
    """Split-KV forward for Nq <= Nk (decoding): q [B,H,Nq,d], k/v [B,H_kv,Nk,d].

    Returns (o [B,H,Nq,d] bf16, lse [B,H,Nq] fp32).  ``num_splits`` defaults
    to fa2_fwd_splitkv_suggest_splits for q's device.  ``workspace`` (a CUDA
    byte tensor) is allocated here when not given."""
    lib = load_library()
    B, H, Nq, d = _shape(q, "q")
    Bk, Hkv, Nk, dk_ = _shape(k, "k")
    if (Bk, dk_) != (B, d) or _shape(v, "v") != (B, Hkv, Nk, d):
        raise ValueError("k and v must be [B, H_kv, Nk, d] with q's B and d")
    if num_splits is None:
        sms = torch.cuda.get_device_properties(q.device).multi_processor_count
        num_splits = max(1, lib.fa2_fwd_splitkv_suggest_splits(sms, B, H, Hkv, Nq, Nk))
    o = torch.empty_like(q) if o is None else o
    lse = torch.empty((B, H, Nq), dtype=torch.float32, device=q.device) if lse is None else lse
    need = lib.fa2_fwd_splitkv_workspace_bytes(B, H, Nq, Nk, d, num_splits)
    if workspace is None and need > 0:
        workspace = torch.empty(need, dtype=torch.uint8, device=q.device)
    wptr = workspace.data_ptr() if workspace is not None else None
    wbytes = workspace.numel() * workspace.element_size() if workspace is not None else 0
    rc = lib.fa2_fwd_splitkv(q.data_ptr(), k.data_ptr(), v.data_ptr(), o.data_ptr(), lse.data_ptr(), B, H, Hkv, Nq,
                             Nk, d, _scale(scale, d), 1 if causal else 0, num_splits, wptr, wbytes,
                             _stream(stream, q.device))
    if rc != FA2_OK:
        raise FA2Error("fa2_fwd_splitkv", rc)
    return o, lse


def _packed(t, name: str):
    if t.dim() != 3:
        raise ValueError(f"{name} must be packed [total, heads, d], got {tuple(t.shape)}")
    if t.dtype != torch.bfloat16 or not t.is_cuda or not t.is_contiguous():
        raise ValueError(f"{name} must be a contiguous CUDA bfloat16 tensor")
    return tuple(t.shape)


def _cu(t, name: str):
    if t.dtype != torch.int32 or not t.is_cuda or not t.is_contiguous() or t.dim() != 1 or t.numel() < 2:
        raise ValueError(f"{name} must be a contiguous CUDA int32 tensor of B + 1 offsets")
    return t.numel() - 1


def _ptr(t):
    return t.data_ptr() if t is not None and t.numel() > 0 else None


def _varlen_shapes(q, k, v, cu_seqlens_q, cu_seqlens_k):
    tq, H, d = _packed(q, "q")
    tk, Hkv, dk_ = _packed(k, "k")
    if dk_ != d or _packed(v, "v") != (tk, Hkv, d):
        raise ValueError("k and v must be [total_k, H_kv, d] with q's d")
    B = _cu(cu_seqlens_q, "cu_seqlens_q")
    if _cu(cu_seqlens_k, "cu_seqlens_k") != B:
        raise ValueError("cu_seqlens_q and cu_seqlens_k must have the same length")
    return B, H, Hkv, tq, tk, d


def _max_len(cu, given):
    if given is not None:
        return int(given)
    return int((cu[1:] - cu[:-1]).max().item()) if cu.numel() > 1 else 0


@_made_on_stream
def fa2_fwd_varlen(q, k, v, cu_seqlens_q, cu_seqlens_k, max_seqlen_q: Optional[int] = None,
                   max_seqlen_k: Optional[int] = None, o=None, lse=None, scale: Optional[float] = None,
                   causal: bool = True, stream=None):
    """Variable-length forward on packed sequences: q [total_q,H,d], k/v [total_k,H_kv,d],
    cu_seqlens_* CUDA int32 [B+1].  Returns (o [total_q,H,d] bf16, lse [H,total_q] fp32).
    The maximum lengths are read from the offsets (a device sync) when not given."""
    lib = load_library()
    B, H, Hkv, tq, tk, d = _varlen_shapes(q, k, v, cu_seqlens_q, cu_seqlens_k)
    mq, mk = _max_len(cu_seqlens_q, max_seqlen_q), _max_len(cu_seqlens_k, max_seqlen_k)
    o = torch.empty_like(q) if o is None else o
    lse = torch.empty((H, tq), dtype=torch.float32, device=q.device) if lse is None else lse
    if _packed(o, "o") != (tq, H, d):
        raise ValueError("o must have q's shape")
    if lse.dtype != torch.float32 or not lse.is_contiguous() or tuple(lse.shape) != (H, tq):
        raise ValueError("lse must be a contiguous fp32 [H, total_q] tensor")
    rc = lib.fa2_fwd_varlen(_ptr(q), _ptr(k), _ptr(v), _ptr(o), _ptr(lse), cu_seqlens_q.data_ptr(),
                            cu_seqlens_k.data_ptr(), B, H, Hkv, tq, tk, mq, mk, d, _scale(scale, d),
                            1 if causal else 0, _stream(stream, q.device))
    if rc != FA2_OK:
        raise FA2Error("fa2_fwd_varlen", rc)
    return o, lse


@_made_on_stream
def fa2_bwd_varlen(q, k, v, o, dO, lse, cu_seqlens_q, cu_seqlens_k, max_seqlen_q: Optional[int] = None,
                   max_seqlen_k: Optional[int] = None, dq=None, dk=None, dv=None, workspace=None,
                   scale: Optional[float] = None, causal: bool = True, stream=None):
    """Variable-length backward: returns (dq [total_q,H,d], dk, dv [total_k,H_kv,d]); dk, dv
    sum over each group of query heads.  ``workspace`` is allocated here when not given."""
    lib = load_library()
    B, H, Hkv, tq, tk, d = _varlen_shapes(q, k, v, cu_seqlens_q, cu_seqlens_k)
    mq, mk = _max_len(cu_seqlens_q, max_seqlen_q), _max_len(cu_seqlens_k, max_seqlen_k)
    for name, t in (("o", o), ("dO", dO)):
        if _packed(t, name) != (tq, H, d):
            raise ValueError(f"{name} must have q's shape")
    if lse.dtype != torch.float32 or not lse.is_contiguous() or tuple(lse.shape) != (H, tq):
        raise ValueError("lse must be a contiguous fp32 [H, total_q] tensor")
    dq = torch.empty_like(q) if dq is None else dq
    dk = torch.empty_like(k) if dk is None else dk
    dv = torch.empty_like(v) if dv is None else dv
    need = lib.fa2_bwd_varlen_workspace_bytes(H, tq, d)
    if workspace is None:
        workspace = torch.empty(max(need, 1), dtype=torch.uint8, device=q.device)
    rc = lib.fa2_bwd_varlen(_ptr(q), _ptr(k), _ptr(v), _ptr(o), _ptr(dO), _ptr(lse), _ptr(dq), _ptr(dk), _ptr(dv),
                            cu_seqlens_q.data_ptr(), cu_seqlens_k.data_ptr(), B, H, Hkv, tq, tk, mq, mk, d,
                            _scale(scale, d), 1 if causal else 0, workspace.data_ptr(),
                            workspace.numel() * workspace.element_size(), _stream(stream, q.device))
    if rc != FA2_OK:
        raise FA2Error("fa2_bwd_varlen", rc)
    return dq, dk, dv


@_made_on_stream
def fa2_bwd_noalloc(q, k, v, o, dO, lse, dq=None, dk=None, dv=None, scale: Optional[float] = None,
                    causal: bool = True, stream=None):
    """fa2_bwd for callers that cannot allocate device memory: the library's
    scratch comes from a fixed 64 MiB device array shared by all calls (see
    include/fa2.h); concurrent calls on one device race."""
    lib = load_library()
    (B, H, N, d), dq, dk, dv = _bwd_common(q, k, v, o, dO, lse, dq, dk, dv)
    rc = lib.fa2_bwd_noalloc(q.data_ptr(), k.data_ptr(), v.data_ptr(), o.data_ptr(), dO.data_ptr(),
                             lse.data_ptr(), dq.data_ptr(), dk.data_ptr(), dv.data_ptr(), B, H, N, d,
                             _scale(scale, d), 1 if causal else 0, _stream(stream, q.device))
    if rc != FA2_OK:
        raise FA2Error("fa2_bwd_noalloc", rc)
    return dq, dk, dv


FA2_DQ_REDUCE, FA2_DQ_ATOMIC, FA2_DQ_SPLIT = 0, 1, 2


@_made_on_stream
def fa2_bwd_deterministic(q, k, v, o, dO, lse, dq=None, dk=None, dv=None, workspace=None,
                          scale: Optional[float] = None, causal: bool = True, stream=None):
    """Bitwise-reproducible backward (d = 128): dQ summed over key tiles in a
    fixed order.  ``workspace`` (CUDA byte tensor) is allocated here when not given."""
    lib = load_library()
    (B, H, N, d), dq, dk, dv = _bwd_common(q, k, v, o, dO, lse, dq, dk, dv)
    need = lib.fa2_bwd_deterministic_workspace_bytes(B, H, N, d, 1 if causal else 0)
    if workspace is None:
        workspace = torch.empty(max(need, 1), dtype=torch.uint8, device=q.device)
    rc = lib.fa2_bwd_deterministic(q.data_ptr(), k.data_ptr(), v.data_ptr(), o.data_ptr(), dO.data_ptr(),
                                   lse.data_ptr(), dq.data_ptr(), dk.data_ptr(), dv.data_ptr(), B, H, N, d,
                                   _scale(scale, d), 1 if causal else 0, workspace.data_ptr(),
                                   workspace.numel() * workspace.element_size(), _stream(stream, q.device))
    if rc != FA2_OK:
        raise FA2Error("fa2_bwd_deterministic", rc)
    return dq, dk, dv


def fa2_bwd_stages(q, k, v, o, dO, lse, Dvec, dq_acc, dq, dk, dv, scale: Optional[float] = None,
                   causal: bool = True, stream=None, hook=None, dq_mode: int = FA2_DQ_REDUCE):
    """fa2_bwd_ws as its three C-ABI stages; ``hook(i)`` is called before stage i
    (0: preprocess, 1: main, 2: dQ convert) and with i = 3 after the last, so a
    caller can record CUDA events between them."""
    lib = load_library()
    (B, H, N, d), dq, dk, dv = _bwd_common(q, k, v, o, dO, lse, dq, dk, dv)
    sc, st = _scale(scale, d), _stream(stream, q.device)
    hook = hook or (lambda i: None)
    hook(0)
    # (split mode: D only, the partial slots are written whole)
    acc0 = None if dq_mode == FA2_DQ_SPLIT else dq_acc.data_ptr()
    rc = lib.fa2_bwd_preprocess(o.data_ptr(), dO.data_ptr(), Dvec.data_ptr(), acc0, B, H, N, d, st)
    if rc != FA2_OK:
        raise FA2Error("fa2_bwd_preprocess", rc)
    hook(1)
    rc = lib.fa2_bwd_main_dq(q.data_ptr(), k.data_ptr(), v.data_ptr(), dO.data_ptr(), lse.data_ptr(),
                             Dvec.data_ptr(), dq_acc.data_ptr(), dk.data_ptr(), dv.data_ptr(), B, H, N, d, sc,
                             1 if causal else 0, dq_mode, st)
    if rc != FA2_OK:
        raise FA2Error("fa2_bwd_main_dq", rc)
    hook(2)
    if dq_mode == FA2_DQ_SPLIT:
        rc = lib.fa2_bwd_dq_reduce(dq_acc.data_ptr(), dq.data_ptr(), B, H, N, d, sc, 1 if causal else 0, st)
    else:
        rc = lib.fa2_bwd_dq_convert(dq_acc.data_ptr(), dq.data_ptr(), B, H, N, d, sc, st)
    if rc != FA2_OK:
        raise FA2Error("fa2_bwd_dq_convert", rc)
    hook(3)
    return dq, dk, dv


def _group_plan(BH: int, chunks: Optional[int], groups):
    """Head counts per group for fa2_step_from_host: `groups` as given,
    `chunks` equal groups, or None for the library's default plan."""
    if groups is not None:
        sizes = [int(x) for x in groups]
        if sum(sizes) != BH or min(sizes) < 1:
            raise ValueError(f"groups must be positive head counts summing to B * H = {BH}")
        return sizes
    if chunks is not None:
        n = max(1, min(BH, int(chunks)))
        return [BH * (i + 1) // n - BH * i // n for i in range(n)]
    return None


def fa2_step_from_host_workspace_bytes(B: int, H: int, N: int, d: int, groups=None, compute_streams: int = 2) -> int:
    arr, n = _int_array(groups)
    return load_library().fa2_step_from_host_workspace_bytes(B, H, N, d, arr, n, compute_streams)


def _int_array(values):
    if values is None:
        return None, 0
    return (ctypes.c_int * len(values))(*values), len(values)


def fa2_step_from_host(host: dict, causal: bool = True, scale: Optional[float] = None, stream=None,
                       chunks: Optional[int] = None, groups=None, compute_streams: int = 2,
                       workspace: Optional[torch.Tensor] = None) -> dict:
    """One forward + backward pass on host tensors (C ABI fa2_step_from_host).

    ``host`` holds CPU tensors (page-locked for overlap): bf16 q, k, v, dO
    [B, H, N, d] and outputs o, dq, dk, dv (bf16, same shape) and lse (fp32
    [B, H, N]).  The library pipelines the copies and kernels over groups of
    heads (``groups`` head counts, ``chunks`` equal groups, or its default
    plan) on ``compute_streams`` compute streams.  ``workspace`` is a CUDA
    uint8 tensor of at least fa2_step_from_host_workspace_bytes(...) bytes
    (allocated here when omitted).  Everything is enqueued on ``stream``
    (default: the current stream); synchronise it before reading ``host``.
    """
    q = host["q"]
    if q.dim() != 4 or q.dtype != torch.bfloat16 or q.is_cuda:
        raise ValueError("host['q'] must be a CPU bfloat16 [B, H, N, d] tensor")
    B, H, N, d = q.shape
    for name in ("k", "v", "dO", "o", "dq", "dk", "dv"):
        t = host[name]
        if t.shape != q.shape or t.dtype != torch.bfloat16 or t.is_cuda or not t.is_contiguous():
            raise ValueError(f"host['{name}'] must be a contiguous CPU bfloat16 tensor shaped like q")
    lse = host["lse"]
    if tuple(lse.shape) != (B, H, N) or lse.dtype != torch.float32 or lse.is_cuda or not lse.is_contiguous():
        raise ValueError("host['lse'] must be a contiguous CPU float32 [B, H, N] tensor")
    plan = _group_plan(B * H, chunks, groups)
    arr, n = _int_array(plan)
    lib = load_library()
    need = lib.fa2_step_from_host_workspace_bytes(B, H, N, d, arr, n, compute_streams)
    if need == 0:
        raise FA2Error("fa2_step_from_host_workspace_bytes", 2)
    if workspace is None:
        dev = stream.device_index if isinstance(stream, torch.cuda.Stream) else torch.cuda.current_device()
        with _on(dev, stream):
            workspace = torch.empty(need, dtype=torch.uint8, device=dev)
    st = _stream(stream, workspace.device)
    rc = lib.fa2_step_from_host(q.data_ptr(), host["k"].data_ptr(), host["v"].data_ptr(), host["dO"].data_ptr(),
                                host["o"].data_ptr(), lse.data_ptr(), host["dq"].data_ptr(), host["dk"].data_ptr(),
                                host["dv"].data_ptr(), B, H, N, d, _scale(scale, d), 1 if causal else 0, arr, n,
                                compute_streams, workspace.data_ptr(), workspace.numel(), st)
    if rc != FA2_OK:
        raise FA2Error("fa2_step_from_host", rc)
    return host


# --------------------------------------------------------------- around the attention: norm + rotation, paged 4-bit cache
# These calls are made once per layer and decoding step, where the kernels take
# a few microseconds: the checks read each tensor's metadata once, and the
# stream handle comes from torch without a Stream object.
_raw_stream = torch._C._cuda_getCurrentRawStream
_current_device = torch._C._cuda_getDevice
# A host array of strides, as the bytes of C's long longs (made in a third of the time of a ctypes array).
_pack4, _pack12, _pack18 = (struct.Struct(f"{n}q").pack for n in (4, 12, 18))


# (devices are compared by index: -1 is the CPU)
def _rows(t, name: str, dev: int):
    """((B, heads, N, d), (batch, head, token) strides) of a bf16 [B, heads, N, d] tensor, or of a packed [total, heads,
    d] one as B = 1."""
    if t.dtype is not torch.bfloat16 or t.get_device() != dev:
        raise ValueError(f"{name} must be bfloat16 on cuda:{dev}")
    shape, stride = t.shape, t.stride()
    if len(shape) == 4:
        B, h, N, d = shape
        sb, sh, sn, sd = stride
    elif len(shape) == 3:
        (N, h, d), (sn, sh, sd), B, sb = shape, stride, 1, 0
    else:
        raise ValueError(f"{name} must be [B, heads, N, d] or packed [total, heads, d], got {tuple(shape)}")
    if sd != 1 and d > 1:
        raise ValueError(f"{name}'s last dimension must be contiguous")
    return (B, h, N, d), (sb, sh, sn)


def _ints(t, name: str, dev: int, count: int, dtype=torch.int32):
    if t.dtype is not dtype or t.get_device() != dev or t.shape != (count,) or not t.is_contiguous():
        raise ValueError(f"{name} must be a contiguous {dtype} tensor of {count} entries on cuda:{dev}")


def _table(t, dev: int):
    """(rows, width, row stride) of an int32 block table."""
    if t.dtype is not torch.int32 or t.get_device() != dev or t.dim() != 2:
        raise ValueError(f"block_table must be an int32 [B, width] tensor on cuda:{dev}")
    (rows, width), (sr, sc) = t.shape, t.stride()
    if width > 1 and sc != 1:
        raise ValueError("block_table's rows must be contiguous")
    return rows, width, sr


def _gpu(t, name: str) -> int:
    dev = t.get_device()
    if dev < 0:
        raise ValueError(f"{name} must be a CUDA tensor")
    return dev


def _norm_args(q, k, q_weight, k_weight, rope, positions, interleaved, dev):
    """The checks and C arguments that the norm's two directions share: (dims, weights are fp32, strides of q and k)."""
    (B, H, N, d), sq = _rows(q, "q", dev)
    (Bk, Hkv, Nk, dk), sk = _rows(k, "k", dev)
    if Bk != B or Nk != N or dk != d or k.dim() != q.dim():
        raise ValueError("k must have q's B, N and d")
    w32 = 0
    for w in (q_weight, k_weight):
        if w is not None:
            if w.dtype is torch.float32:
                w32 = 1
            elif w.dtype is not torch.bfloat16:
                raise ValueError("a weight must be bfloat16 or float32")
            if w.shape != (d,) or w.get_device() != dev or not w.is_contiguous():
                raise ValueError("a weight must be a contiguous tensor of d values on q's device")
    if q_weight is not None and k_weight is not None and q_weight.dtype is not k_weight.dtype:
        raise ValueError("q_weight and k_weight must have the same type")
    rot = max_pos = 0
    if rope is not None:
        if rope.dtype is not torch.float32 or rope.dim() != 2 or rope.get_device() != dev or not rope.is_contiguous():
            raise ValueError("rope must be a contiguous float32 [max_positions, rot_dim] tensor on q's device")
        max_pos, rot = rope.shape
    if positions is not None:
        if (positions.dtype is not torch.int32 or positions.get_device() != dev or not positions.is_contiguous()
                or positions.shape != ((N,) if q.dim() == 3 else (B, N))):
            raise ValueError("positions must be a contiguous int32 tensor, one per token, on q's device")
    return (B, H, Hkv, N, d, rot, 1 if interleaved else 0, max_pos), w32, sq + sk


def _norm_out(like, out, name: str, dev: int):
    """(`out` checked against `like`, or a new contiguous tensor; its strides)."""
    if out is None:
        out = torch.empty(like.shape, dtype=torch.bfloat16, device=like.device)
        stride = out.stride()
        return out, (stride[:3] if len(stride) == 4 else (0, stride[1], stride[0]))
    if out.shape != like.shape:
        raise ValueError(f"{name} must have its input's shape")
    return out, _rows(out, name, dev)[1]


def _dp(t):
    return None if t is None else t.data_ptr()


def fa2_qk_norm_rope(q, k, q_weight=None, k_weight=None, rope=None, positions=None, eps: float = 1e-6,
                     interleaved: bool = False, q_out=None, k_out=None, stream=None):
    """Per-head RMS norm of q and k and the position rotation, in one pass (see include/fa2.h).

    q [B, H, N, d], k [B, H_kv, N, d] with any strides but a contiguous last
    dimension (views of a fused projection), or packed [total, heads, d].
    ``rope`` is fp32 [max_positions, rot_dim]: cosines, then sines;
    ``positions`` int32 [B, N] (packed: [total]), default 0, 1, ...  Returns
    (q_out, k_out), new contiguous tensors unless given; q_out may be q.
    """
    dev = _gpu(q, "q")
    if stream is not None or dev != _current_device():
        with _on(dev, stream):
            return fa2_qk_norm_rope(q, k, q_weight, k_weight, rope, positions, eps, interleaved, q_out, k_out)
    dims, w32, strides = _norm_args(q, k, q_weight, k_weight, rope, positions, interleaved, dev)
    q_out, sq = _norm_out(q, q_out, "q_out", dev)
    k_out, sk = _norm_out(k, k_out, "k_out", dev)
    rc = load_library().fa2_qk_norm_rope(
        q.data_ptr(), k.data_ptr(), _dp(q_weight), _dp(k_weight), w32, _dp(rope), _dp(positions), q_out.data_ptr(),
        k_out.data_ptr(), *dims, eps, _pack12(*strides, *sq, *sk), _raw_stream(dev))
    if rc != FA2_OK:
        raise FA2Error("fa2_qk_norm_rope", rc)
    return q_out, k_out


def fa2_qk_norm_rope_bwd(dq_out, dk_out, q, k, q_weight=None, k_weight=None, rope=None, positions=None,
                         eps: float = 1e-6, interleaved: bool = False, dq=None, dk=None, workspace=None, stream=None):
    """Gradient of fa2_qk_norm_rope: (dq, dk, dq_weight, dk_weight) from the gradients of its outputs.

    q and k are the forward call's inputs.  dq, dk are new contiguous tensors
    unless given (dq may be dq_out or q).  The weights' gradients are fp32,
    None where there is no weight.
    """
    dev = _gpu(q, "q")
    if stream is not None or dev != _current_device():
        with _on(dev, stream):
            return fa2_qk_norm_rope_bwd(dq_out, dk_out, q, k, q_weight, k_weight, rope, positions, eps, interleaved, dq, dk,
                                        workspace)
    dims, w32, strides = _norm_args(q, k, q_weight, k_weight, rope, positions, interleaved, dev)
    if dq_out.shape != q.shape or dk_out.shape != k.shape:
        raise ValueError("dq_out and dk_out must have q's and k's shapes")
    grads = _rows(dq_out, "dq_out", dev)[1] + _rows(dk_out, "dk_out", dev)[1]
    dq, sq = _norm_out(q, dq, "dq", dev)
    dk, sk = _norm_out(k, dk, "dk", dev)
    d = dims[4]
    lib = load_library()
    dwq = None if q_weight is None else torch.empty(d, dtype=torch.float32, device=q.device)
    dwk = None if k_weight is None else torch.empty(d, dtype=torch.float32, device=q.device)
    if workspace is not None:
        if workspace.get_device() != dev:
            raise ValueError("workspace must be on q's device")
    elif dwq is not None or dwk is not None:
        workspace = torch.empty(max(1, lib.fa2_qk_norm_rope_bwd_workspace_bytes(d)), dtype=torch.uint8, device=q.device)
    rc = lib.fa2_qk_norm_rope_bwd(
        dq_out.data_ptr(), dk_out.data_ptr(), q.data_ptr(), k.data_ptr(), _dp(q_weight), _dp(k_weight), w32, _dp(rope),
        _dp(positions), dq.data_ptr(), dk.data_ptr(), _dp(dwq), _dp(dwk), *dims, eps, _pack18(*grads, *strides, *sq, *sk),
        _dp(workspace), 0 if workspace is None else workspace.numel() * workspace.element_size(), _raw_stream(dev))
    if rc != FA2_OK:
        raise FA2Error("fa2_qk_norm_rope_bwd", rc)
    return dq, dk, dwq, dwk


class PagePlan(NamedTuple):
    """What fa2_page_plan writes besides the block table (all on the GPU; see include/fa2.h)."""
    lens: torch.Tensor          # int32 [B]
    cu_new: torch.Tensor        # int32 [B + 1]
    cu_total: torch.Tensor      # int32 [B + 1]
    slots: torch.Tensor         # int64 [max_tokens]
    positions: torch.Tensor     # int32 [max_tokens]
    pages_needed: torch.Tensor  # int32 [1]


def fa2_page_plan(cached_lens, new_lens, free_pages, block_table, page_size: int, max_tokens: int,
                  plan: Optional[PagePlan] = None, stream=None) -> PagePlan:
    """One step's page plan from request lengths, on the GPU: fills the new entries of ``block_table``
    (int32 [B, width]) and returns the rest.  ``plan``: an earlier call's result to write into."""
    dev = _gpu(cached_lens, "cached_lens")
    if stream is not None or dev != _current_device():
        with _on(dev, stream):
            return fa2_page_plan(cached_lens, new_lens, free_pages, block_table, page_size, max_tokens, plan)
    B, width, row_stride = _table(block_table, dev)
    _ints(cached_lens, "cached_lens", dev, B)
    _ints(new_lens, "new_lens", dev, B)
    num_free = free_pages.numel()
    _ints(free_pages, "free_pages", dev, num_free)
    if max_tokens < 0:
        raise ValueError("max_tokens must be at least 0")
    if plan is None:
        at = cached_lens.device  # (six allocations take less time than two and the views of their parts)
        plan = PagePlan(torch.empty(B, dtype=torch.int32, device=at), torch.empty(B + 1, dtype=torch.int32, device=at),
                        torch.empty(B + 1, dtype=torch.int32, device=at), torch.empty(max_tokens, dtype=torch.int64, device=at),
                        torch.empty(max_tokens, dtype=torch.int32, device=at), torch.empty(1, dtype=torch.int32, device=at))
    else:
        for t, name, n in zip(plan, PagePlan._fields, (B, B + 1, B + 1, max_tokens, max_tokens, 1)):
            _ints(t, "plan." + name, dev, n, torch.int64 if name == "slots" else torch.int32)
    rc = load_library().fa2_page_plan(
        cached_lens.data_ptr(), new_lens.data_ptr(), free_pages.data_ptr(), block_table.data_ptr(),
        plan.lens.data_ptr(), plan.cu_new.data_ptr(), plan.cu_total.data_ptr(), plan.slots.data_ptr(),
        plan.positions.data_ptr(), plan.pages_needed.data_ptr(), B, num_free, width, row_stride, page_size,
        max_tokens, _raw_stream(dev))
    if rc != FA2_OK:
        raise FA2Error("fa2_page_plan", rc)
    return plan


def fa2_kv4_page_bytes(H_kv: int, page_size: int, d: int) -> int:
    return load_library().fa2_kv4_page_bytes(H_kv, page_size, d)


def fa2_kv4_cache(num_pages: int, H_kv: int, page_size: int, d: int, device="cuda") -> torch.Tensor:
    """A cache of zeros: uint8 [num_pages, H_kv, page_size / 16, 18 d]."""
    if fa2_kv4_page_bytes(H_kv, page_size, d) == 0 or num_pages < 1:
        raise ValueError("page_size must be 16, 32, 64 or 128, d 16, 32, 64 or 128, and the counts at least 1")
    return torch.zeros((num_pages, H_kv, page_size // 16, 18 * d), dtype=torch.uint8, device=device)


def _cache_dims(cache):
    """(pages, H_kv, page size, d, page stride in bytes) of a cache, whose pages may lie apart."""
    if cache.dtype is not torch.uint8 or cache.dim() != 4:
        raise ValueError("cache must be a CUDA uint8 tensor [num_pages, H_kv, page_size / 16, 18 d] (fa2_kv4_cache)")
    (pages, heads, tiles, row), (s0, s1, s2, s3) = cache.shape, cache.stride()
    if row % 18 != 0 or s3 != 1 or (tiles > 1 and s2 != row) or (heads > 1 and s1 != tiles * row):
        raise ValueError("a page of the cache must be contiguous, its last dimension 18 d")
    # (one page: its stride says nothing)
    return pages, heads, tiles * 16, row // 18, s0 if pages > 1 else heads * tiles * row


def fa2_kv4_append(k, v, cache, slots, k_scale: float = 1.0, v_scale: float = 1.0, k_out=None, v_out=None,
                   stream=None) -> None:
    """Write keys and values [T, H_kv, d] bf16 (any token and head strides) to their ``slots`` (int64 [T]) of the
    4-bit cache.  ``k_out``, ``v_out``: contiguous tensors that receive the values as stored."""
    dev = _gpu(cache, "cache")
    if stream is not None or dev != _current_device():
        with _on(dev, stream):
            return fa2_kv4_append(k, v, cache, slots, k_scale, v_scale, k_out, v_out)
    pages, heads, page_size, d, page_stride = _cache_dims(cache)
    T = slots.numel()
    _ints(slots, "slots", dev, T, torch.int64)
    want = (T, heads, d)
    if k.dim() != 3 or v.dim() != 3:
        raise ValueError("k and v must be [tokens, H_kv, d]")
    (kt, kh, kd), (vt, vh, vd) = k.stride(), v.stride()
    if (k.dtype is not torch.bfloat16 or v.dtype is not torch.bfloat16 or k.get_device() != dev or v.get_device() != dev
            or k.shape != want or v.shape != want or kd != 1 or vd != 1):
        raise ValueError("k and v must be bfloat16 [tokens, H_kv, d] on the cache's device, the last dimension contiguous")
    for t in (k_out, v_out):
        if t is not None and (t.dtype is not torch.bfloat16 or t.get_device() != dev or t.shape != want or not t.is_contiguous()):
            raise ValueError("k_out and v_out must be contiguous bfloat16 tensors of k's shape")
    if T == 0:
        return
    rc = load_library().fa2_kv4_append(
        k.data_ptr(), v.data_ptr(), _pack4(kt, kh, vt, vh), cache.data_ptr(), page_stride, slots.data_ptr(), _dp(k_out),
        _dp(v_out), T, heads, pages, page_size, d, k_scale, v_scale, _raw_stream(dev))
    if rc != FA2_OK:
        raise FA2Error("fa2_kv4_append", rc)


def fa2_kv4_gather(cache, block_table, cu_seqlens, total: int, k_scale: float = 1.0, v_scale: float = 1.0, k=None,
                   v=None, stream=None):
    """The cache's keys and values as packed bf16 [total, H_kv, d] (what fa2_fwd_varlen takes as k and v with
    cu_seqlens_k = ``cu_seqlens``).  Rows outside every sequence of given k, v are left as they are."""
    dev = _gpu(cache, "cache")
    if stream is not None or dev != _current_device():
        with _on(dev, stream):
            return fa2_kv4_gather(cache, block_table, cu_seqlens, total, k_scale, v_scale, k, v)
    pages, heads, page_size, d, page_stride = _cache_dims(cache)
    B, width, row_stride = _table(block_table, dev)
    _ints(cu_seqlens, "cu_seqlens", dev, B + 1)
    for t in (k, v):
        if t is not None and (t.get_device() != dev or t.dtype is not torch.bfloat16 or t.shape != (total, heads, d)
                              or not t.is_contiguous()):
            raise ValueError("k and v must be contiguous bfloat16 [total, H_kv, d] on the cache's device")
    k = torch.empty((total, heads, d), dtype=torch.bfloat16, device=cache.device) if k is None else k
    v = torch.empty((total, heads, d), dtype=torch.bfloat16, device=cache.device) if v is None else v
    rc = load_library().fa2_kv4_gather(
        cache.data_ptr(), page_stride, block_table.data_ptr(), row_stride, cu_seqlens.data_ptr(), k.data_ptr(), v.data_ptr(), B, heads,
        total, pages, page_size, width, d, k_scale, v_scale, _raw_stream(dev))
    if rc != FA2_OK:
        raise FA2Error("fa2_kv4_gather", rc)
    return k, v


def fa2_kv4_attn_workspace_bytes(B: int, H: int, H_kv: int, max_seqlen_q: int, max_seqlen_k: int, d: int) -> int:
    """Scratch of fa2_kv4_attn for these sizes (0: none); max_seqlen_k at most width * page_size of the block table.

    A call with a shorter bound can need more (include/fa2.h has the rule); with
    max_seqlen_k = 2**30 it is what is enough under any bound.
    """
    return load_library().fa2_kv4_attn_workspace_bytes(B, H, H_kv, max_seqlen_q, max_seqlen_k, d)


def fa2_kv4_attn(q, cache, block_table, lens, cu_seqlens_q=None, max_seqlen_q: Optional[int] = None,
                 max_seqlen_k: Optional[int] = None, o=None, lse=None, workspace=None, scale: Optional[float] = None,
                 k_scale: float = 1.0, v_scale: float = 1.0, causal: bool = True, stream=None):
    """Attention of packed queries q [total_q, H, d] over the 4-bit paged cache: (o [total_q, H, d] bf16,
    lse [H, total_q] fp32).

    Request b's keys are the first lens[b] tokens of its pages block_table[b]
    (int32 [B, width]); its queries are rows cu_seqlens_q[b] .. of q, its last
    positions where ``causal``.  Without cu_seqlens_q every request has
    ``max_seqlen_q`` queries (default: total_q / B).  With cu_seqlens_q and no
    max_seqlen_q the maximum is read from the offsets (a device sync); a bound
    may be larger than any request's queries.  ``max_seqlen_k`` bounds lens (default: what block_table has room for); a
    tight bound lets short requests take a single launch without workspace.
    """
    dev = _gpu(cache, "cache")
    if stream is not None or dev != _current_device():
        with _on(dev, stream):
            return fa2_kv4_attn(q, cache, block_table, lens, cu_seqlens_q, max_seqlen_q, max_seqlen_k, o, lse, workspace,
                                scale, k_scale, v_scale, causal)
    pages, heads, page_size, d, page_stride = _cache_dims(cache)
    if q.dim() != 3 or q.dtype is not torch.bfloat16 or q.get_device() != dev or not q.is_contiguous() or q.shape[2] != d:
        raise ValueError("q must be contiguous bfloat16 [total_q, H, d] on the cache's device, with its head dim")
    tq, H, _ = q.shape
    B, width, row_stride = _table(block_table, dev)
    _ints(lens, "lens", dev, B)
    if cu_seqlens_q is not None:
        _ints(cu_seqlens_q, "cu_seqlens_q", dev, B + 1)
        mq = min(_max_len(cu_seqlens_q, max_seqlen_q), tq)
    else:
        mq = tq // max(B, 1) if max_seqlen_q is None else int(max_seqlen_q)
        if mq * B != tq:
            raise ValueError("without cu_seqlens_q every request has the same number of queries")
    if o is None:
        o = torch.empty_like(q)
    elif o.shape != q.shape or o.dtype is not torch.bfloat16 or o.get_device() != dev or not o.is_contiguous():
        raise ValueError("o must be contiguous bfloat16 with q's shape and device")
    if lse is None:
        lse = torch.empty((H, tq), dtype=torch.float32, device=cache.device)
    elif lse.dtype is not torch.float32 or lse.get_device() != dev or not lse.is_contiguous() or lse.shape != (H, tq):
        raise ValueError("lse must be a contiguous fp32 [H, total_q] tensor")
    lib = load_library()
    mk = min(width * page_size, 2 ** 31 - 1)
    if max_seqlen_k is not None and max_seqlen_k < mk:
        mk = int(max_seqlen_k)
    if workspace is None:
        need = lib.fa2_kv4_attn_workspace_bytes(B, H, heads, mq, mk, d)
        if need:
            workspace = torch.empty(need, dtype=torch.uint8, device=cache.device)
    elif workspace.get_device() != dev:
        raise ValueError("workspace must be on the cache's device")
    rc = lib.fa2_kv4_attn(
        q.data_ptr(), cache.data_ptr(), page_stride, block_table.data_ptr(), row_stride, lens.data_ptr(), _dp(cu_seqlens_q),
        o.data_ptr(), lse.data_ptr(), B, H, heads, tq, mq, mk, pages, page_size, width, d, _scale(scale, d), k_scale, v_scale, 1 if causal else 0,
        _dp(workspace), 0 if workspace is None else workspace.numel() * workspace.element_size(), _raw_stream(dev))
    if rc != FA2_OK:
        raise FA2Error("fa2_kv4_attn", rc)
    return o, lse
