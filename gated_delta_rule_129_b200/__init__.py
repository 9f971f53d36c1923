"""B200 (sm_100a) Gated DeltaNet-2 forward operator -- Python binding.

A thin ctypes layer over ``libgdn2.so`` (declared in ``include/gdn2.h``).  It
only marshals arguments: every step of the computation runs in the library's
CUDA kernels.  PyTorch supplies device memory and the current stream.  There
is no CPU fallback: if the library is missing, every call raises.

Public functions mirror the C entry points:

* :func:`chunk_fwd`        -- ``gdn2_chunk_fwd``
* :func:`chunk_prep`       -- ``gdn2_chunk_prep`` (gate prep + intra-chunk WY)
* :func:`chunk_walk`       -- ``gdn2_chunk_walk`` (state walk + output)
* :func:`chunk_plan`, :func:`chunk_fused` -- ``gdn2_chunk_plan``, ``gdn2_chunk_fused``
  (the fused prep + walk launch on its own, for timing and tests)
* :func:`recurrent_step`   -- ``gdn2_recurrent_step`` (one decode token)
* :func:`token_prologue`, :func:`token_epilogue` and their backward passes
  :func:`token_prologue_bwd`, :func:`token_epilogue_bwd` -- the token path
* :func:`act_pack`, :func:`act_unpack` -- activations kept in 8 bits
* :func:`gated_scan_fwd`, :func:`gated_scan_bwd`, :func:`gated_scan_step` -- the
  gated linear recurrence
* :func:`workspace_size`, :func:`workspace_layout`, :func:`status_string`
"""
from __future__ import annotations

import ctypes
import functools
import inspect
import os
import threading
from typing import NamedTuple

__all__ = ["chunk_fwd", "chunk_fwd_noalloc", "noalloc_status", "chunk_walk_flagged", "chunk_fwd_segmented",
           "segmented_workspace_size", "state_map", "token_prologue", "token_epilogue", "token_path_fwd", "chunk_prep", "chunk_walk", "chunk_plan", "chunk_fused",
           "recurrent_step", "workspace_size",
           "act_pack", "act_unpack", "PackedAct", "token_prologue_bwd", "token_epilogue_bwd", "token_path_bwd",
           "gated_scan_fwd", "gated_scan_bwd", "gated_scan_step", "gated_scan_chunk_states",
           "workspace_layout", "status_string", "GDN2Error", "lib_path", "load_library"]

_HERE = os.path.dirname(os.path.abspath(__file__))
_LIB_PATH = os.path.join(_HERE, "libgdn2.so")
_lock = threading.Lock()
_lib = None

GDN2_IO_F32 = 0
GDN2_IO_BF16 = 1

STATUS = {0: "GDN2_OK", 1: "GDN2_ERR_NULL", 2: "GDN2_ERR_SHAPE", 3: "GDN2_ERR_DTYPE",
          4: "GDN2_ERR_ALIGN", 5: "GDN2_ERR_SEQLENS", 6: "GDN2_ERR_WORKSPACE",
          7: "GDN2_ERR_CUDA", 8: "GDN2_ERR_DEVICE_TIMEOUT", 9: "GDN2_ERR_UNSUPPORTED"}

EXPORTED = ("gdn2_workspace_size", "gdn2_workspace_layout", "gdn2_chunk_fwd", "gdn2_chunk_fwd_noalloc",
            "gdn2_chunk_prep", "gdn2_chunk_walk", "gdn2_chunk_plan", "gdn2_chunk_fused",
            "gdn2_recurrent_step", "gdn2_status_string", "gdn2_version", "gdn2_backward_workspace_size",
            "gdn2_chunk_bwd", "gdn2_noalloc_status", "gdn2_chunk_walk_flagged",
            "gdn2_segmented_workspace_size", "gdn2_chunk_fwd_segmented", "gdn2_state_map",
            "gdn2_token_prologue", "gdn2_token_epilogue", "gdn2_act_pack", "gdn2_act_unpack",
            "gdn2_token_prologue_bwd_workspace_size", "gdn2_token_prologue_bwd",
            "gdn2_token_epilogue_bwd_workspace_size", "gdn2_token_epilogue_bwd",
            "gdn2_gated_scan_workspace_size", "gdn2_gated_scan_fwd", "gdn2_gated_scan_bwd", "gdn2_gated_scan_step")


class GDN2Error(RuntimeError):
    def __init__(self, status: int, where: str):
        self.status = status
        super().__init__(f"{where}: {STATUS.get(status, status)} ({status_string(status)})")


class Desc(ctypes.Structure):
    _fields_ = [("B", ctypes.c_int), ("T", ctypes.c_int), ("H", ctypes.c_int),
                ("dk", ctypes.c_int), ("dv", ctypes.c_int), ("num_seqs", ctypes.c_int),
                ("io", ctypes.c_int), ("workspace", ctypes.c_void_p),
                ("workspace_bytes", ctypes.c_size_t)]


class WsLayout(ctypes.Structure):
    _fields_ = [("total_bytes", ctypes.c_size_t), ("max_chunks", ctypes.c_int),
                ("factor_elem_bytes", ctypes.c_int), ("factor_set", ctypes.c_int),
                ("reserved", ctypes.c_int), ("off_W", ctypes.c_size_t),
                ("off_Ut", ctypes.c_size_t), ("off_Kbar", ctypes.c_size_t),
                ("off_Qeff", ctypes.c_size_t), ("off_Opart", ctypes.c_size_t),
                ("off_gamma_last", ctypes.c_size_t), ("off_Mp", ctypes.c_size_t),
                ("off_Nc", ctypes.c_size_t), ("off_chunk_offsets", ctypes.c_size_t),
                ("off_status", ctypes.c_size_t), ("off_fix", ctypes.c_size_t),
                ("off_sync", ctypes.c_size_t), ("off_colscale", ctypes.c_size_t)]

    def as_dict(self):
        return {name: getattr(self, name) for name, _ in self._fields_}


def lib_path() -> str:
    return _LIB_PATH


def load_library():
    """Load ``libgdn2.so``; raises if it has not been built."""
    global _lib
    with _lock:
        if _lib is not None:
            return _lib
        if not os.path.exists(_LIB_PATH):
            raise RuntimeError(f"{_LIB_PATH} is missing: build it with "
                               "`python -m gated_delta_rule_129_b200.build` (nvcc, sm_100a)")
        lib = ctypes.CDLL(_LIB_PATH)
        vp, i, f, sz = ctypes.c_void_p, ctypes.c_int, ctypes.c_float, ctypes.c_size_t
        dp = ctypes.POINTER(Desc)
        lib.gdn2_workspace_size.argtypes = [dp]
        lib.gdn2_workspace_size.restype = sz
        lib.gdn2_workspace_layout.argtypes = [dp, ctypes.POINTER(WsLayout)]
        lib.gdn2_workspace_layout.restype = i
        lib.gdn2_chunk_fwd.argtypes = [dp, vp, vp, vp, vp, vp, vp, f, vp, vp, vp, vp, vp]
        lib.gdn2_chunk_fwd.restype = i
        lib.gdn2_chunk_fwd_noalloc.argtypes = [dp, vp, vp, vp, vp, vp, vp, f, vp, vp, vp, vp, vp]
        lib.gdn2_chunk_fwd_noalloc.restype = i
        lib.gdn2_noalloc_status.argtypes = [dp, vp, vp]
        lib.gdn2_noalloc_status.restype = i
        lib.gdn2_chunk_walk_flagged.argtypes = [dp, f, vp, vp, vp, vp, ctypes.c_ulonglong, vp]
        lib.gdn2_chunk_walk_flagged.restype = i
        lib.gdn2_segmented_workspace_size.argtypes = [dp, i]
        lib.gdn2_segmented_workspace_size.restype = sz
        lib.gdn2_chunk_fwd_segmented.argtypes = [dp, vp, vp, vp, vp, vp, vp, f, vp, vp, vp, vp, i, vp]
        lib.gdn2_chunk_fwd_segmented.restype = i
        lib.gdn2_state_map.argtypes = [dp, vp, vp, vp, vp, vp, vp, vp, vp, vp, vp]
        lib.gdn2_state_map.restype = i
        lib.gdn2_token_prologue.argtypes = [dp, vp, vp, vp, vp, vp, vp, i, vp, vp, vp, vp, vp]
        lib.gdn2_token_prologue.restype = i
        lib.gdn2_token_epilogue.argtypes = [dp, vp, vp, vp, vp, vp]
        lib.gdn2_token_epilogue.restype = i
        lib.gdn2_chunk_prep.argtypes = [dp, vp, vp, vp, vp, vp, vp, vp, vp]
        lib.gdn2_chunk_prep.restype = i
        lib.gdn2_chunk_walk.argtypes = [dp, f, vp, vp, vp, vp, vp, vp]
        lib.gdn2_chunk_walk.restype = i
        lib.gdn2_chunk_plan.argtypes = [dp, vp, vp]
        lib.gdn2_chunk_plan.restype = i
        lib.gdn2_chunk_fused.argtypes = [dp, vp, vp, vp, vp, vp, vp, f, vp, vp, vp, vp, vp]
        lib.gdn2_chunk_fused.restype = i
        lib.gdn2_recurrent_step.argtypes = [dp, vp, vp, vp, vp, vp, vp, f, vp, vp, vp]
        lib.gdn2_backward_workspace_size.argtypes = [dp]
        lib.gdn2_backward_workspace_size.restype = sz
        lib.gdn2_chunk_bwd.argtypes = [dp, vp, vp, vp, vp, vp, vp, f, vp, vp, vp, vp, vp, vp, vp, vp, vp, vp, vp, vp]
        lib.gdn2_chunk_bwd.restype = i
        lib.gdn2_recurrent_step.restype = i
        ll = ctypes.c_longlong
        lib.gdn2_act_pack.argtypes = [vp, i, ll, i, vp, vp, vp]
        lib.gdn2_act_pack.restype = i
        lib.gdn2_act_unpack.argtypes = [vp, vp, ll, i, i, vp, vp]
        lib.gdn2_act_unpack.restype = i
        lib.gdn2_token_prologue_bwd_workspace_size.argtypes = [dp, i]
        lib.gdn2_token_prologue_bwd_workspace_size.restype = sz
        lib.gdn2_token_prologue_bwd.argtypes = [dp] + [vp] * 9 + [i] + [vp] * 11
        lib.gdn2_token_prologue_bwd.restype = i
        lib.gdn2_token_epilogue_bwd_workspace_size.argtypes = [dp]
        lib.gdn2_token_epilogue_bwd_workspace_size.restype = sz
        lib.gdn2_token_epilogue_bwd.argtypes = [dp] + [vp] * 10
        lib.gdn2_token_epilogue_bwd.restype = i
        lib.gdn2_gated_scan_workspace_size.argtypes = [dp]
        lib.gdn2_gated_scan_workspace_size.restype = sz
        lib.gdn2_gated_scan_fwd.argtypes = [dp] + [vp] * 9
        lib.gdn2_gated_scan_fwd.restype = i
        lib.gdn2_gated_scan_bwd.argtypes = [dp] + [vp] * 12
        lib.gdn2_gated_scan_bwd.restype = i
        lib.gdn2_gated_scan_step.argtypes = [dp] + [vp] * 6
        lib.gdn2_gated_scan_step.restype = i
        lib.gdn2_status_string.argtypes = [i]
        lib.gdn2_status_string.restype = ctypes.c_char_p
        lib.gdn2_version.argtypes = []
        lib.gdn2_version.restype = i
        _lib = lib
        return lib


def status_string(status: int) -> str:
    return load_library().gdn2_status_string(int(status)).decode()


def _check(status: int, where: str):
    if status != 0:
        raise GDN2Error(status, where)


# ------------------------------------------------------------------ helpers --

def _torch():
    import torch
    return torch


def _io_of(dtype) -> int:
    torch = _torch()
    if dtype == torch.float32:
        return GDN2_IO_F32
    if dtype == torch.bfloat16:
        return GDN2_IO_BF16
    raise TypeError(f"q/k/v must be float32 or bfloat16, got {dtype}")


def _ptr(t):
    return None if t is None else ctypes.c_void_p(t.data_ptr())


def _stream(stream):
    torch = _torch()
    s = stream if stream is not None else torch.cuda.current_stream()
    return ctypes.c_void_p(s.cuda_stream)


def make_desc(B, T, H, dk, dv, io, num_seqs=0, workspace=None, workspace_bytes=0) -> Desc:
    return Desc(int(B), int(T), int(H), int(dk), int(dv), int(num_seqs), int(io),
                None if workspace is None else ctypes.c_void_p(workspace),
                int(workspace_bytes))


def workspace_size(B, T, H, dk, dv, io=GDN2_IO_BF16, num_seqs=0) -> int:
    d = make_desc(B, T, H, dk, dv, io, num_seqs)
    return int(load_library().gdn2_workspace_size(ctypes.byref(d)))


def workspace_layout(B, T, H, dk, dv, io=GDN2_IO_BF16, num_seqs=0) -> dict:
    d = make_desc(B, T, H, dk, dv, io, num_seqs)
    lay = WsLayout()
    _check(load_library().gdn2_workspace_layout(ctypes.byref(d), ctypes.byref(lay)),
           "gdn2_workspace_layout")
    return lay.as_dict()


def _shapes(q, v, cu_seqlens):
    B, T, H, dk = q.shape
    dv = v.shape[-1]
    num_seqs = 0 if cu_seqlens is None else int(cu_seqlens.numel()) - 1
    return B, T, H, dk, dv, num_seqs


def _alloc_workspace(desc_args, device):
    torch = _torch()
    nbytes = workspace_size(*desc_args)
    if nbytes == 0:
        raise GDN2Error(2, "gdn2_workspace_size")
    return torch.empty(nbytes, dtype=torch.uint8, device=device)


def _need_contig(*ts):
    for t in ts:
        if t is not None and not t.is_contiguous():
            raise ValueError("all tensors must be contiguous")


# -------------------------------------------------------------- entry points --

def chunk_fwd(q, k, v, log_alpha, b, w, scale=None, h0=None, cu_seqlens=None, *,
              out=None, hT=None, workspace=None, output_final_state=True, stream=None):
    """Gated DeltaNet-2 chunkwise forward.  Returns ``(out, hT)``.

    ``q, k, v`` are float32 or bfloat16 ``[B, T, H, d]`` CUDA tensors;
    ``log_alpha, b, w`` float32 of the same leading shape; ``h0`` float32
    ``[N, H, dk, dv]`` or None; ``cu_seqlens`` int32 ``[N + 1]`` CUDA tensor
    or None.  ``scale`` defaults to ``dk ** -0.5``.
    """
    torch = _torch()
    B, T, H, dk, dv, ns = _shapes(q, v, cu_seqlens)
    io = _io_of(q.dtype)
    N = ns if cu_seqlens is not None else B
    if scale is None:
        scale = dk ** -0.5
    _need_contig(q, k, v, log_alpha, b, w, h0, cu_seqlens)
    if out is None:
        out = torch.empty(v.shape, dtype=q.dtype, device=q.device)
    if hT is None and output_final_state:
        hT = torch.empty((N, H, dk, dv), dtype=torch.float32, device=q.device)
    if workspace is None:
        workspace = _alloc_workspace((B, T, H, dk, dv, io, ns), q.device)
    d = make_desc(B, T, H, dk, dv, io, ns, workspace.data_ptr(), workspace.numel() * workspace.element_size())
    st = load_library().gdn2_chunk_fwd(ctypes.byref(d), _ptr(q), _ptr(k), _ptr(v), _ptr(log_alpha),
                                       _ptr(b), _ptr(w), float(scale), _ptr(h0), _ptr(cu_seqlens),
                                       _ptr(out), _ptr(hT), _stream(stream))
    _check(st, "gdn2_chunk_fwd")
    return out, hT


def chunk_plan(shape, dtype, workspace, cu_seqlens=None, *, stream=None):
    """``gdn2_chunk_plan`` for ``shape = (B, T, H, dk, dv)`` into ``workspace``."""
    B, T, H, dk, dv = shape
    ns = 0 if cu_seqlens is None else cu_seqlens.numel() - 1
    d = make_desc(B, T, H, dk, dv, _io_of(dtype), ns, workspace.data_ptr(),
                  workspace.numel() * workspace.element_size())
    _check(load_library().gdn2_chunk_plan(ctypes.byref(d), _ptr(cu_seqlens), _stream(stream)), "gdn2_chunk_plan")


def chunk_fused(q, k, v, log_alpha, b, w, scale, workspace, h0=None, cu_seqlens=None, *, out, hT=None,
                stream=None):
    """``gdn2_chunk_fused``: the fused prep + walk launch alone (run
    :func:`chunk_plan` on the same workspace first).  Raises ``GDN2Error``
    (``GDN2_ERR_UNSUPPORTED``) when the problem does not take the fused path."""
    B, T, H, dk, dv, ns = _shapes(q, v, cu_seqlens)
    _need_contig(q, k, v, log_alpha, b, w, h0, cu_seqlens)
    d = make_desc(B, T, H, dk, dv, _io_of(q.dtype), ns, workspace.data_ptr(),
                  workspace.numel() * workspace.element_size())
    st = load_library().gdn2_chunk_fused(ctypes.byref(d), _ptr(q), _ptr(k), _ptr(v), _ptr(log_alpha), _ptr(b),
                                         _ptr(w), float(scale), _ptr(h0), _ptr(cu_seqlens), _ptr(out), _ptr(hT),
                                         _stream(stream))
    _check(st, "gdn2_chunk_fused")
    return out, hT


NOALLOC_SCRATCH_BYTES = 32 << 20


def chunk_fwd_noalloc(q, k, v, log_alpha, b, w, scale=None, h0=None, cu_seqlens=None, *,
                      out=None, hT=None, output_final_state=True, stream=None):
    """``gdn2_chunk_fwd_noalloc``: like :func:`chunk_fwd`, but the library uses
    its own fixed device scratch (``NOALLOC_SCRATCH_BYTES``) instead of a
    workspace, for callers that cannot allocate device memory where they run
    the operator.  Problems whose workspace would exceed the scratch raise
    ``GDN2Error`` (``GDN2_ERR_WORKSPACE``).  Calls share the scratch, so calls
    that overlap on the GPU race; keep them on one stream.  ``out``/``hT``
    are allocated here only if not given."""
    torch = _torch()
    B, T, H, dk, dv, ns = _shapes(q, v, cu_seqlens)
    io = _io_of(q.dtype)
    N = ns if cu_seqlens is not None else B
    if scale is None:
        scale = dk ** -0.5
    _need_contig(q, k, v, log_alpha, b, w, h0, cu_seqlens)
    if out is None:
        out = torch.empty(v.shape, dtype=q.dtype, device=q.device)
    if hT is None and output_final_state:
        hT = torch.empty((N, H, dk, dv), dtype=torch.float32, device=q.device)
    d = make_desc(B, T, H, dk, dv, io, ns)
    st = load_library().gdn2_chunk_fwd_noalloc(ctypes.byref(d), _ptr(q), _ptr(k), _ptr(v), _ptr(log_alpha),
                                               _ptr(b), _ptr(w), float(scale), _ptr(h0), _ptr(cu_seqlens),
                                               _ptr(out), _ptr(hT), _stream(stream))
    _check(st, "gdn2_chunk_fwd_noalloc")
    return out, hT


def noalloc_status(q, v, cu_seqlens=None, *, stream=None):
    """``gdn2_noalloc_status``: the device status word of the last
    :func:`chunk_fwd_noalloc` call on inputs shaped like ``q``, ``v``
    (``cu_seqlens`` for a packed call), as an int32 CUDA tensor of one element
    filled on ``stream`` (0 = ok, 5 = malformed cu_seqlens, 8 = a bounded
    device wait gave up)."""
    torch = _torch()
    B, T, H, dk, dv, ns = _shapes(q, v, cu_seqlens)
    out = torch.empty(4, dtype=torch.int32, device=q.device)
    d = make_desc(B, T, H, dk, dv, _io_of(q.dtype), ns)
    _check(load_library().gdn2_noalloc_status(ctypes.byref(d), _ptr(out), _stream(stream)), "gdn2_noalloc_status")
    return out[:1]


def chunk_prep(q, k, v, log_alpha, b, w, cu_seqlens=None, *, workspace=None, stream=None):
    """Stage 1 only.  Returns the workspace tensor holding the chunk factors."""
    B, T, H, dk, dv, ns = _shapes(q, v, cu_seqlens)
    io = _io_of(q.dtype)
    _need_contig(q, k, v, log_alpha, b, w, cu_seqlens)
    if workspace is None:
        workspace = _alloc_workspace((B, T, H, dk, dv, io, ns), q.device)
    d = make_desc(B, T, H, dk, dv, io, ns, workspace.data_ptr(), workspace.numel() * workspace.element_size())
    st = load_library().gdn2_chunk_prep(ctypes.byref(d), _ptr(q), _ptr(k), _ptr(v), _ptr(log_alpha),
                                        _ptr(b), _ptr(w), _ptr(cu_seqlens), _stream(stream))
    _check(st, "gdn2_chunk_prep")
    return workspace


def chunk_walk(workspace, shape, io_dtype, scale, h0=None, cu_seqlens=None, *, out=None, hT=None,
               chunk_states=None, stream=None):
    """Stage 2 only, from a workspace filled by :func:`chunk_prep`.

    ``shape`` is ``(B, T, H, dk, dv)``; ``io_dtype`` the torch dtype of q/k/v.
    Returns ``(out, hT)``.
    """
    torch = _torch()
    B, T, H, dk, dv = shape
    ns = 0 if cu_seqlens is None else int(cu_seqlens.numel()) - 1
    N = ns if cu_seqlens is not None else B
    io = _io_of(io_dtype)
    if out is None:
        out = torch.empty((B, T, H, dv), dtype=io_dtype, device=workspace.device)
    if hT is None:
        hT = torch.empty((N, H, dk, dv), dtype=torch.float32, device=workspace.device)
    d = make_desc(B, T, H, dk, dv, io, ns, workspace.data_ptr(), workspace.numel() * workspace.element_size())
    st = load_library().gdn2_chunk_walk(ctypes.byref(d), float(scale), _ptr(h0), _ptr(cu_seqlens),
                                        _ptr(out), _ptr(hT), _ptr(chunk_states), _stream(stream))
    _check(st, "gdn2_chunk_walk")
    return out, hT


def chunk_walk_flagged(workspace, shape, io_dtype, scale, h0=None, cu_seqlens=None, *, out=None, hT=None,
                       wait_budget_ns=0, stream=None):
    """``gdn2_chunk_walk_flagged``: :func:`chunk_walk` that takes each chunk
    only once its ready flag in the workspace is raised, with every bounded
    device wait limited to ``wait_budget_ns`` (0 = 2 s).  Returns ``(out, hT)``;
    a wait that gave up shows in the workspace status word."""
    torch = _torch()
    B, T, H, dk, dv = shape
    ns = 0 if cu_seqlens is None else int(cu_seqlens.numel()) - 1
    N = ns if cu_seqlens is not None else B
    if out is None:
        out = torch.empty((B, T, H, dv), dtype=io_dtype, device=workspace.device)
    if hT is None:
        hT = torch.empty((N, H, dk, dv), dtype=torch.float32, device=workspace.device)
    d = make_desc(B, T, H, dk, dv, _io_of(io_dtype), ns, workspace.data_ptr(),
                  workspace.numel() * workspace.element_size())
    st = load_library().gdn2_chunk_walk_flagged(ctypes.byref(d), float(scale), _ptr(h0), _ptr(cu_seqlens),
                                                _ptr(out), _ptr(hT), ctypes.c_ulonglong(int(wait_budget_ns)),
                                                _stream(stream))
    _check(st, "gdn2_chunk_walk_flagged")
    return out, hT


def segmented_workspace_size(B, T, H, dk, dv, io=GDN2_IO_BF16, num_seqs=0, segment_chunks=0) -> int:
    d = make_desc(B, T, H, dk, dv, io, num_seqs)
    return int(load_library().gdn2_segmented_workspace_size(ctypes.byref(d), int(segment_chunks)))


def chunk_fwd_segmented(q, k, v, log_alpha, b, w, scale=None, h0=None, cu_seqlens=None, *, segment_chunks=0,
                        out=None, hT=None, workspace=None, output_final_state=True, stream=None):
    """``gdn2_chunk_fwd_segmented``: :func:`chunk_fwd` through the two-level
    chunk scan, each sequence split into segments of ``segment_chunks``
    64-token chunks (0 = the library's choice).  Returns ``(out, hT)``."""
    torch = _torch()
    B, T, H, dk, dv, ns = _shapes(q, v, cu_seqlens)
    io = _io_of(q.dtype)
    N = ns if cu_seqlens is not None else B
    if scale is None:
        scale = dk ** -0.5
    _need_contig(q, k, v, log_alpha, b, w, h0, cu_seqlens)
    if out is None:
        out = torch.empty(v.shape, dtype=q.dtype, device=q.device)
    if hT is None and output_final_state:
        hT = torch.empty((N, H, dk, dv), dtype=torch.float32, device=q.device)
    if workspace is None:
        nbytes = segmented_workspace_size(B, T, H, dk, dv, io, ns, segment_chunks)
        if nbytes == 0:
            raise GDN2Error(9, "gdn2_segmented_workspace_size")
        workspace = torch.empty(nbytes, dtype=torch.uint8, device=q.device)
    d = make_desc(B, T, H, dk, dv, io, ns, workspace.data_ptr(), workspace.numel() * workspace.element_size())
    st = load_library().gdn2_chunk_fwd_segmented(ctypes.byref(d), _ptr(q), _ptr(k), _ptr(v), _ptr(log_alpha),
                                                 _ptr(b), _ptr(w), float(scale), _ptr(h0), _ptr(cu_seqlens),
                                                 _ptr(out), _ptr(hT), int(segment_chunks), _stream(stream))
    _check(st, "gdn2_chunk_fwd_segmented")
    return out, hT


def state_map(q, k, v, log_alpha, b, w, cu_seqlens=None, *, phi=None, psi=None, workspace=None, stream=None):
    """``gdn2_state_map``: the affine map of every sequence, ``(phi [N, H, dk,
    dk], psi [N, H, dk, dv])`` fp32, with final state = phi @ S_start + psi."""
    torch = _torch()
    B, T, H, dk, dv, ns = _shapes(q, v, cu_seqlens)
    io = _io_of(q.dtype)
    N = ns if cu_seqlens is not None else B
    _need_contig(q, k, v, log_alpha, b, w, cu_seqlens)
    if phi is None:
        phi = torch.empty((N, H, dk, dk), dtype=torch.float32, device=q.device)
    if psi is None:
        psi = torch.empty((N, H, dk, dv), dtype=torch.float32, device=q.device)
    if workspace is None:
        workspace = _alloc_workspace((B, T, H, dk, dv, io, ns), q.device)
    d = make_desc(B, T, H, dk, dv, io, ns, workspace.data_ptr(), workspace.numel() * workspace.element_size())
    st = load_library().gdn2_state_map(ctypes.byref(d), _ptr(q), _ptr(k), _ptr(v), _ptr(log_alpha), _ptr(b),
                                       _ptr(w), _ptr(cu_seqlens), _ptr(phi), _ptr(psi), _stream(stream))
    _check(st, "gdn2_state_map")
    return phi, psi


def token_prologue(q_raw, k_raw, v_raw, conv_q, conv_k, conv_v, cu_seqlens=None, *, q=None, k=None, v=None,
                   stream=None):
    """``gdn2_token_prologue``: ``(q, k, v)`` for the operator from the
    projections' outputs (short causal convolution with weights ``conv_*``
    ``[H * d, W]`` fp32, SiLU, and L2 normalisation of q and k)."""
    torch = _torch()
    B, T, H, dk, dv, ns = _shapes(q_raw, v_raw, cu_seqlens)
    io = _io_of(q_raw.dtype)
    _need_contig(q_raw, k_raw, v_raw, conv_q, conv_k, conv_v, cu_seqlens)
    W = int(conv_q.shape[-1])
    q = torch.empty_like(q_raw) if q is None else q
    k = torch.empty_like(k_raw) if k is None else k
    v = torch.empty_like(v_raw) if v is None else v
    d = make_desc(B, T, H, dk, dv, io, ns)
    st = load_library().gdn2_token_prologue(ctypes.byref(d), _ptr(q_raw), _ptr(k_raw), _ptr(v_raw), _ptr(conv_q),
                                            _ptr(conv_k), _ptr(conv_v), W, _ptr(cu_seqlens), _ptr(q), _ptr(k), _ptr(v),
                                            _stream(stream))
    _check(st, "gdn2_token_prologue")
    return q, k, v


def token_epilogue(o, gate, norm_weight, *, out=None, stream=None):
    """``gdn2_token_epilogue``: ``rmsnorm(o) * norm_weight * sigmoid(gate)``."""
    torch = _torch()
    B, T, H, dv = o.shape
    _need_contig(o, gate, norm_weight)
    out = torch.empty_like(o) if out is None else out
    d = make_desc(B, T, H, 128, dv, _io_of(o.dtype))
    st = load_library().gdn2_token_epilogue(ctypes.byref(d), _ptr(o), _ptr(gate), _ptr(norm_weight), _ptr(out),
                                            _stream(stream))
    _check(st, "gdn2_token_epilogue")
    return out


def token_path_fwd(q_raw, k_raw, v_raw, log_alpha, b, w, gate, conv_q, conv_k, conv_v, norm_weight, scale=None,
                   h0=None, cu_seqlens=None, *, workspace=None, stream=None):
    """The operator with its token path: :func:`token_prologue`, then
    :func:`chunk_fwd`, then :func:`token_epilogue`.  Returns ``(out, hT)``
    (``out`` before the caller's output projection)."""
    q, k, v = token_prologue(q_raw, k_raw, v_raw, conv_q, conv_k, conv_v, cu_seqlens, stream=stream)
    o, hT = chunk_fwd(q, k, v, log_alpha, b, w, scale, h0, cu_seqlens, workspace=workspace, stream=stream)
    return token_epilogue(o, gate, norm_weight, out=o, stream=stream), hT


def backward_workspace_size(B, T, H, dk, dv, io=GDN2_IO_BF16, num_seqs=0) -> int:
    d = make_desc(B, T, H, dk, dv, io, num_seqs)
    return int(load_library().gdn2_backward_workspace_size(ctypes.byref(d)))


def chunk_bwd(q, k, v, log_alpha, b, w, scale, dO, h0=None, dhT=None, cu_seqlens=None, *, workspace=None,
              stream=None):
    """``gdn2_chunk_bwd``: gradients of :func:`chunk_fwd`'s ``(out, hT)``
    contracted with ``dO`` (``[B, T, H, dv]``, the dtype of ``q``) and ``dhT``
    (``[N, H, dk, dv]`` fp32 or None).  Returns a dict of fp32 tensors
    ``q, k, v, log_alpha, b, w`` (input shapes) and ``h0`` ``[N, H, dk, dv]``."""
    torch = _torch()
    B, T, H, dk, dv, ns = _shapes(q, v, cu_seqlens)
    io = _io_of(q.dtype)
    N = ns if cu_seqlens is not None else B
    _need_contig(q, k, v, log_alpha, b, w, h0, cu_seqlens, dO, dhT)
    if workspace is None:
        nbytes = backward_workspace_size(B, T, H, dk, dv, io, ns)
        if nbytes == 0:
            raise GDN2Error(2, "gdn2_backward_workspace_size")
        workspace = torch.empty(nbytes, dtype=torch.uint8, device=q.device)
    f32 = dict(dtype=torch.float32, device=q.device)
    g = {n: torch.empty(t.shape, **f32) for n, t in (("q", q), ("k", k), ("v", v), ("log_alpha", log_alpha),
                                                       ("b", b), ("w", w))}
    g["h0"] = torch.empty((N, H, dk, dv), **f32)
    d = make_desc(B, T, H, dk, dv, io, ns, workspace.data_ptr(), workspace.numel() * workspace.element_size())
    st = load_library().gdn2_chunk_bwd(ctypes.byref(d), _ptr(q), _ptr(k), _ptr(v), _ptr(log_alpha), _ptr(b),
                                       _ptr(w), float(scale), _ptr(h0), _ptr(cu_seqlens), _ptr(dO), _ptr(dhT),
                                       _ptr(g["q"]), _ptr(g["k"]), _ptr(g["v"]), _ptr(g["log_alpha"]), _ptr(g["b"]),
                                       _ptr(g["w"]), _ptr(g["h0"]), _stream(stream))
    _check(st, "gdn2_chunk_bwd")
    return g


def recurrent_step(q, k, v, log_alpha, b, w, scale, state, *, out=None, stream=None):
    """One decode token; ``state`` ``[B, H, dk, dv]`` fp32 is updated in place.

    ``q, k, log_alpha, b`` are ``[B, H, dk]``; ``v, w`` ``[B, H, dv]``.
    Returns ``out`` ``[B, H, dv]``.
    """
    torch = _torch()
    Bn, H, dk = q.shape
    dv = v.shape[-1]
    io = _io_of(q.dtype)
    _need_contig(q, k, v, log_alpha, b, w, state)
    if out is None:
        out = torch.empty((Bn, H, dv), dtype=q.dtype, device=q.device)
    d = make_desc(Bn, 1, H, dk, dv, io)
    st = load_library().gdn2_recurrent_step(ctypes.byref(d), _ptr(q), _ptr(k), _ptr(v), _ptr(log_alpha),
                                            _ptr(b), _ptr(w), float(scale), _ptr(state), _ptr(out),
                                            _stream(stream))
    _check(st, "gdn2_recurrent_step")
    return out


# ------------------------------------------- training: checked entry points --

_IO = {}   # torch dtype -> gdn2_io_dtype, filled at the first call


def _io(dtype):
    if not _IO:
        torch = _torch()
        _IO.update({torch.float32: GDN2_IO_F32, torch.bfloat16: GDN2_IO_BF16})
    io = _IO.get(dtype)
    return _io_of(dtype) if io is None else io   # _io_of refuses any other


def _expect(name, t, shape, dtype, device):
    """One tensor argument: its type, shape, device and layout."""
    if t.dtype is dtype and t.shape == shape and t.device == device and t.is_contiguous():
        return
    if t.dtype != dtype:
        raise TypeError(f"{name} must be {dtype}, got {t.dtype}")
    if tuple(t.shape) != tuple(shape):
        raise ValueError(f"{name} must have shape {tuple(shape)}, got {tuple(t.shape)}")
    if t.device != device:
        raise ValueError(f"{name} is on {t.device}, expected {device}")
    raise ValueError(f"{name} must be contiguous")


def _cuda_device(name, t):
    if not t.is_cuda:
        raise ValueError(f"{name} must be a CUDA tensor, got one on {t.device}")
    return t.device


def _num_seqs(cu_seqlens, B, device):
    """0 for dense rows; the packed sequences' number, with cu_seqlens checked."""
    if cu_seqlens is None:
        return 0
    if B != 1:
        raise ValueError(f"a packed call has one row, got {B}")
    if cu_seqlens.dim() != 1 or cu_seqlens.numel() < 2:
        raise ValueError(f"cu_seqlens must have shape [num_seqs + 1], got {tuple(cu_seqlens.shape)}")
    _expect("cu_seqlens", cu_seqlens, cu_seqlens.shape, _torch().int32, device)
    return cu_seqlens.numel() - 1


def _on_stream(f):
    """``f`` with a ``stream`` argument: the whole call, its outputs and its
    workspace included, belongs to that stream, so that no block of memory is
    handed out again while the stream still uses it."""
    lead = next(iter(inspect.signature(f).parameters))   # a tensor or a PackedAct: it says where the call belongs

    @functools.wraps(f)
    def call(*args, stream=None, **kw):
        if stream is None:
            return f(*args, **kw)
        first = args[0] if args else kw.get(lead)
        first = first[0] if isinstance(first, (tuple, list)) and first else first
        device = getattr(first, "device", None)
        if device is None:
            return f(*args, **kw)   # which says what is wrong with it
        if device != stream.device:
            raise ValueError(f"stream is on {stream.device}, the tensors on {device}")
        with _torch().cuda.stream(stream):
            return f(*args, **kw)
    return call


def _call(where, device, *args):
    """The library's function ``where`` on ``args`` and ``device``'s current
    stream, with ``device`` current."""
    torch = _torch()
    fn, index = getattr(_lib or load_library(), where), device.index
    stream = torch._C._cuda_getCurrentRawStream(index)
    if index == torch.cuda.current_device():
        st = fn(*args, stream)
    else:
        with torch.cuda.device(device):
            st = fn(*args, stream)
    if st != 0:
        raise GDN2Error(st, where)


def _addr(t):
    return None if t is None else t.data_ptr()


@functools.lru_cache(maxsize=1024)
def _size_of(where, *sizes):
    """A workspace size of the library: ``where`` of make_desc(*sizes[:7]) (a pure
    function of its arguments) and what else it takes."""
    d = make_desc(*sizes[:7])
    return int(getattr(load_library(), where)(ctypes.byref(d), *sizes[7:]))


def _scratch(where, workspace, device, *sizes):
    """A descriptor of ``sizes`` with the caller's workspace, checked, or a new
    one, and the workspace tensor; a size of 0 is the library's answer to sizes
    it does not take."""
    if workspace is None:
        nbytes = _size_of(where, *sizes)
        if nbytes == 0:
            raise GDN2Error(2, where)
        torch = _torch()
        workspace = torch.empty(nbytes, dtype=torch.uint8, device=device)
    elif workspace.device != device or not workspace.is_contiguous():
        raise ValueError(f"workspace must be a contiguous tensor on {device}")
    else:
        nbytes = workspace.numel() * workspace.element_size()
    B, T, H, dk, dv, io, ns = sizes[:7]
    return Desc(B, T, H, dk, dv, ns, io, workspace.data_ptr(), nbytes), workspace


class PackedAct(NamedTuple):
    """An activation in 8 bits: ``codes`` int8 of the activation's shape and
    ``exps`` uint8 ``[..., ceil(D / 128)]``; a value is ``code * 2 ** (exp - 127)``."""
    codes: object
    exps: object


def _blocks(d):
    return (d + 127) // 128


def _long_rows(name, t):
    """``t``'s rows and their length for the library, whose rows are under 2^31
    values long: rows of whole blocks go as rows of one block, stored alike."""
    D = t.shape[-1]
    if D % 128 != 0:
        raise ValueError(f"{name} has rows of D = {D} values; past 2^31 D must be a multiple of 128")
    return t.numel() // 128, 128


@_on_stream
def act_pack(x, *, out=None):
    """``gdn2_act_pack``: ``x`` (float32 or bfloat16 ``[..., D]``) in 8 bits, one
    power of two per 128 values of a row.  Returns a :class:`PackedAct`, or
    fills ``out``."""
    torch = _torch()
    dev = _cuda_device("x", x)
    io = _io(x.dtype)
    if x.dim() < 1 or x.shape[-1] < 1:
        raise ValueError(f"x must have shape [..., D] with D >= 1, got {tuple(x.shape)}")
    _need_contig(x)
    D = x.shape[-1]
    rows, cols = (x.numel() // D, D) if D < 1 << 31 else _long_rows("x", x)
    eshape = (*x.shape[:-1], _blocks(D))
    if out is None:
        out = PackedAct(torch.empty_like(x, dtype=torch.int8), torch.empty(eshape, dtype=torch.uint8, device=dev))
    else:
        out = PackedAct(*out)
        _expect("out.codes", out.codes, x.shape, torch.int8, dev)
        _expect("out.exps", out.exps, eshape, torch.uint8, dev)
    _call("gdn2_act_pack", dev, x.data_ptr(), io, rows, cols, out.codes.data_ptr(), out.exps.data_ptr())
    return out


@_on_stream
def act_unpack(packed, dtype=None, *, out=None):
    """``gdn2_act_unpack``: the values of a :class:`PackedAct` as ``dtype``
    (float32 or bfloat16; bfloat16 if not given), or into ``out``."""
    torch = _torch()
    codes, exps = packed
    dev = _cuda_device("codes", codes)
    if codes.dim() < 1 or codes.shape[-1] < 1:
        raise ValueError(f"codes must have shape [..., D] with D >= 1, got {tuple(codes.shape)}")
    D = codes.shape[-1]
    _expect("codes", codes, codes.shape, torch.int8, dev)
    _expect("exps", exps, (*codes.shape[:-1], _blocks(D)), torch.uint8, dev)
    rows, cols = (codes.numel() // D, D) if D < 1 << 31 else _long_rows("codes", codes)
    dtype = dtype if dtype is not None else torch.bfloat16 if out is None else out.dtype
    io = _io(dtype)
    if out is None:
        out = torch.empty_like(codes, dtype=dtype)
    else:
        _expect("out", out, codes.shape, dtype, dev)
    _call("gdn2_act_unpack", dev, codes.data_ptr(), exps.data_ptr(), rows, cols, io, out.data_ptr())
    return out


def _kept(name, x, dtype, device):
    """``(data, exps)`` of a kept activation, a tensor or a PackedAct, checked."""
    torch = _torch()
    if isinstance(x, tuple):
        codes, exps = x
        _expect(f"{name}.codes", codes, codes.shape, torch.int8, device)
        _expect(f"{name}.exps", exps, (*codes.shape[:-1], _blocks(codes.shape[-1])), torch.uint8, device)
        return codes, exps
    _expect(name, x, x.shape, dtype, device)
    return x, None


@_on_stream
def token_prologue_bwd(q_raw, k_raw, v_raw, conv_q, conv_k, conv_v, dq, dk, dv, cu_seqlens=None, *, dtype=None,
                       workspace=None):
    """``gdn2_token_prologue_bwd``: gradients of :func:`token_prologue`'s
    ``(q, k, v)`` contracted with ``dq, dk, dv`` (fp32, as :func:`chunk_bwd`
    returns them).  ``q_raw, k_raw, v_raw`` are the forward call's inputs, or
    all three their :class:`PackedAct`; ``dtype`` is the type of those inputs
    and of their gradients (needed when they are packed; bfloat16 if not given).
    Returns a dict ``q_raw, k_raw, v_raw`` (that dtype) and ``conv_q, conv_k,
    conv_v`` (fp32)."""
    torch = _torch()
    packed = [isinstance(x, tuple) for x in (q_raw, k_raw, v_raw)]
    if any(packed) and not all(packed):
        raise ValueError("q_raw, k_raw and v_raw must all be packed, or none")
    first = q_raw[0] if packed[0] else q_raw
    dev = _cuda_device("q_raw", first)
    if dtype is None:
        dtype = torch.bfloat16 if packed[0] else q_raw.dtype
    io = _io(dtype)
    (xq, eq), (xk, ek), (xv, ev) = (_kept(n, x, dtype, dev) for n, x in (("q_raw", q_raw), ("k_raw", k_raw),
                                                                         ("v_raw", v_raw)))
    if xq.dim() != 4 or xv.dim() != 4 or xk.shape != xq.shape or xv.shape[:3] != xq.shape[:3]:
        raise ValueError(f"q_raw, k_raw, v_raw must be [B, T, H, d] alike, got {tuple(xq.shape)}, "
                         f"{tuple(xk.shape)}, {tuple(xv.shape)}")
    B, T, H, dk_ = xq.shape
    dv_ = xv.shape[-1]
    ns = _num_seqs(cu_seqlens, B, dev)
    W = conv_q.shape[-1]
    f32 = torch.float32
    for n, t, shape in (("conv_q", conv_q, (H * dk_, W)), ("conv_k", conv_k, (H * dk_, W)),
                        ("conv_v", conv_v, (H * dv_, W)), ("dq", dq, xq.shape), ("dk", dk, xq.shape),
                        ("dv", dv, xv.shape)):
        _expect(n, t, shape, f32, dev)
    d, workspace = _scratch("gdn2_token_prologue_bwd_workspace_size", workspace, dev, B, T, H, dk_, dv_, io, ns, W)
    like = torch.empty_like
    g = dict(q_raw=like(dq, dtype=dtype), k_raw=like(dk, dtype=dtype), v_raw=like(dv, dtype=dtype), conv_q=like(conv_q),
             conv_k=like(conv_k), conv_v=like(conv_v))
    _call("gdn2_token_prologue_bwd", dev, ctypes.byref(d), xq.data_ptr(),
          xk.data_ptr(), xv.data_ptr(), _addr(eq), _addr(ek), _addr(ev), conv_q.data_ptr(), conv_k.data_ptr(), conv_v.data_ptr(), W,
          _addr(cu_seqlens), dq.data_ptr(), dk.data_ptr(), dv.data_ptr(), *map(_addr, g.values()))
    return g


@_on_stream
def token_epilogue_bwd(o, gate, norm_weight, dout, *, workspace=None):
    """``gdn2_token_epilogue_bwd``: gradients of :func:`token_epilogue`'s result
    contracted with ``dout``.  ``o`` and ``gate`` are the forward call's inputs
    or their :class:`PackedAct`.  Returns a dict ``o``, ``gate`` (the dtype of
    ``dout``) and ``norm_weight`` (fp32)."""
    torch = _torch()
    dev = _cuda_device("dout", dout)
    io = _io(dout.dtype)
    if dout.dim() != 4:
        raise ValueError(f"dout must be [B, T, H, dv], got {tuple(dout.shape)}")
    _expect("dout", dout, dout.shape, dout.dtype, dev)
    (xo, eo), (xg, eg) = (_kept(n, x, dout.dtype, dev) for n, x in (("o", o), ("gate", gate)))
    if xo.shape != dout.shape or xg.shape != dout.shape:
        raise ValueError(f"o and gate must have dout's shape {tuple(dout.shape)}, got {tuple(xo.shape)} and "
                         f"{tuple(xg.shape)}")
    B, T, H, dv = dout.shape
    _expect("norm_weight", norm_weight, (dv,), torch.float32, dev)
    d, workspace = _scratch("gdn2_token_epilogue_bwd_workspace_size", workspace, dev, B, T, H, dv, dv, io, 0)
    g = dict(o=torch.empty_like(dout), gate=torch.empty_like(dout), norm_weight=torch.empty_like(norm_weight))
    _call("gdn2_token_epilogue_bwd", dev, ctypes.byref(d), xo.data_ptr(),
          _addr(eo), xg.data_ptr(), _addr(eg), norm_weight.data_ptr(), dout.data_ptr(), *map(_addr, g.values()))
    return g


@_on_stream
def token_path_bwd(q_raw, k_raw, v_raw, log_alpha, b, w, gate, conv_q, conv_k, conv_v, norm_weight, dout, scale=None,
                   h0=None, dhT=None, cu_seqlens=None, *, o=None):
    """Gradients of :func:`token_path_fwd`'s ``(out, hT)`` contracted with
    ``dout`` and ``dhT``: the prologue again for q, k, v, then
    :func:`token_epilogue_bwd`, :func:`chunk_bwd` and :func:`token_prologue_bwd`.

    ``q_raw, k_raw, v_raw``, ``gate`` and ``o`` (:func:`chunk_fwd`'s output
    before the epilogue; computed again if not given) are the forward pass's
    activations or their :class:`PackedAct`.  Returns a dict ``q_raw, k_raw,
    v_raw, gate`` (``dout``'s dtype) and ``log_alpha, b, w, h0, conv_q, conv_k,
    conv_v, norm_weight`` (fp32)."""
    torch = _torch()
    dev = _cuda_device("dout", dout)
    dtype, f32 = dout.dtype, torch.float32
    _io(dtype)
    raw = dict(q_raw=q_raw, k_raw=k_raw, v_raw=v_raw)
    kept = {n: _kept(n, x, dtype, dev)[0] for n, x in dict(raw, gate=gate).items()}
    qs, vs = kept["q_raw"].shape, kept["v_raw"].shape
    if len(qs) != 4 or len(vs) != 4 or kept["k_raw"].shape != qs or vs[:3] != qs[:3]:
        raise ValueError(f"q_raw, k_raw, v_raw must be [B, T, H, d] alike, got {tuple(qs)}, "
                         f"{tuple(kept['k_raw'].shape)}, {tuple(vs)}")
    B, T, H, dk = qs
    dv, W = vs[3], conv_q.shape[-1]
    N = _num_seqs(cu_seqlens, B, dev) or B
    _expect("gate", kept["gate"], vs, kept["gate"].dtype, dev)
    _expect("dout", dout, vs, dtype, dev)
    if o is not None:
        _expect("o", _kept("o", o, dtype, dev)[0], vs, o[0].dtype if isinstance(o, tuple) else dtype, dev)
    for n, t, shape in (("log_alpha", log_alpha, qs), ("b", b, qs), ("w", w, vs), ("conv_q", conv_q, (H * dk, W)),
                        ("conv_k", conv_k, (H * dk, W)), ("conv_v", conv_v, (H * dv, W)),
                        ("norm_weight", norm_weight, (dv,)), ("h0", h0, (N, H, dk, dv)), ("dhT", dhT, (N, H, dk, dv))):
        if t is not None or n not in ("h0", "dhT"):
            _expect(n, t, shape, f32, dev)
    with torch.cuda.device(dev):
        plain = [act_unpack(x, dtype) if isinstance(x, tuple) else x for x in raw.values()]
        q, k, v = token_prologue(*plain, conv_q, conv_k, conv_v, cu_seqlens)
        if scale is None:
            scale = dk ** -0.5
        if o is None:
            o = chunk_fwd(q, k, v, log_alpha, b, w, scale, h0, cu_seqlens, output_final_state=False)[0]
        e = token_epilogue_bwd(o, gate, norm_weight, dout)
        c = chunk_bwd(q, k, v, log_alpha, b, w, scale, e["o"], h0, dhT, cu_seqlens)
        # all packed or none, as the kernel reads them
        same = raw.values() if len({isinstance(x, tuple) for x in raw.values()}) == 1 else plain
        p = token_prologue_bwd(*same, conv_q, conv_k, conv_v, c["q"], c["k"], c["v"], cu_seqlens, dtype=dtype)
    return dict(p, gate=e["gate"], norm_weight=e["norm_weight"], log_alpha=c["log_alpha"], b=c["b"], w=c["w"],
                h0=c["h0"])


def _scan_args(v, log_alpha, w, cu_seqlens):
    """Checked arguments of the gated scan: sizes, device, shape of the states."""
    torch = _torch()
    dev = _cuda_device("v", v)
    io = _io(v.dtype)
    if v.dim() != 4:
        raise ValueError(f"v must be [B, T, H, dv], got {tuple(v.shape)}")
    _expect("v", v, v.shape, v.dtype, dev)
    _expect("log_alpha", log_alpha, v.shape, torch.float32, dev)
    _expect("w", w, v.shape, torch.float32, dev)
    B, T, H, dv = v.shape
    ns = _num_seqs(cu_seqlens, B, dev)
    return (B, T, H, dv, dv, io, ns), dev, (ns if ns else B, H, dv)


def gated_scan_chunk_states(v, cu_seqlens=None):
    """An uninitialised ``chunk_states`` tensor for :func:`gated_scan_fwd` and
    :func:`gated_scan_bwd` on ``v`` ``[B, T, H, dv]``: ``[max_chunks, H, dv]`` fp32."""
    torch = _torch()
    B, T, H, dv = v.shape
    n = B * ((T + 63) // 64) if cu_seqlens is None else T // 64 + cu_seqlens.numel() - 1
    return torch.empty((n, H, dv), dtype=torch.float32, device=v.device)


@_on_stream
def gated_scan_fwd(v, log_alpha, w, h0=None, cu_seqlens=None, *, out=None, hT=None, chunk_states=None,
                   workspace=None, output_final_state=True):
    """``gdn2_gated_scan_fwd``: ``h_t = exp(log_alpha_t) h_{t-1} + w_t v_t`` per
    channel.  Returns ``(out, hT)`` with ``out`` every ``h_t``.

    ``v`` is float32 or bfloat16 ``[B, T, H, dv]``, ``log_alpha`` and ``w``
    float32 of that shape, ``h0`` float32 ``[N, H, dv]`` or None; ``chunk_states``
    (:func:`gated_scan_chunk_states`) receives the state at the start of every
    64-token chunk, for :func:`gated_scan_bwd`.  A malformed ``cu_seqlens`` (and a
    device wait that gave up) leaves the outputs unspecified and a status other
    than 0 in the first int32 of a ``workspace`` that is given."""
    torch = _torch()
    sizes, dev, sshape = _scan_args(v, log_alpha, w, cu_seqlens)
    f32 = torch.float32
    if h0 is not None:
        _expect("h0", h0, sshape, f32, dev)
    if out is None:
        out = torch.empty_like(v)
    else:
        _expect("out", out, v.shape, v.dtype, dev)
    if hT is not None:
        _expect("hT", hT, sshape, f32, dev)
    elif output_final_state:
        hT = w.new_empty(sshape)
    if chunk_states is not None:
        _expect_states(chunk_states, v, cu_seqlens, dev)
    d, workspace = _scratch("gdn2_gated_scan_workspace_size", workspace, dev, *sizes)
    _call("gdn2_gated_scan_fwd", dev, ctypes.byref(d), v.data_ptr(),
          log_alpha.data_ptr(), w.data_ptr(), _addr(h0), _addr(cu_seqlens), out.data_ptr(), _addr(hT), _addr(chunk_states))
    return out, hT


def _expect_states(chunk_states, v, cu_seqlens, dev):
    B, T, H, dv = v.shape
    n = B * ((T + 63) // 64) if cu_seqlens is None else T // 64 + cu_seqlens.numel() - 1
    _expect("chunk_states", chunk_states, (n, H, dv), _torch().float32, dev)


@_on_stream
def gated_scan_bwd(v, log_alpha, w, dO, h0=None, dhT=None, cu_seqlens=None, *, chunk_states=None, workspace=None):
    """``gdn2_gated_scan_bwd``: gradients of :func:`gated_scan_fwd`'s ``(out,
    hT)`` contracted with ``dO`` (the shape and dtype of ``v``) and ``dhT``
    (``[N, H, dv]`` fp32 or None).  ``chunk_states`` as that call on the same
    inputs left them; if not given they are computed again from ``h0`` (a
    ``workspace`` that is given then holds the status of both calls, 0 if both
    went well).  Returns a dict of fp32 tensors ``v, log_alpha, w`` and ``h0``."""
    torch = _torch()
    sizes, dev, sshape = _scan_args(v, log_alpha, w, cu_seqlens)
    f32 = torch.float32
    _expect("dO", dO, v.shape, v.dtype, dev)
    if h0 is not None:
        _expect("h0", h0, sshape, f32, dev)
    if dhT is not None:
        _expect("dhT", dhT, sshape, f32, dev)
    given = workspace is not None
    d, workspace = _scratch("gdn2_gated_scan_workspace_size", workspace, dev, *sizes)
    r = ctypes.byref(d)
    again = None   # with the caller's workspace: that of the forward call, whose status word is to stay
    if chunk_states is None:
        chunk_states = gated_scan_chunk_states(v, cu_seqlens)
        d0, again = _scratch("gdn2_gated_scan_workspace_size", None, dev, *sizes) if given else (d, None)
        _call("gdn2_gated_scan_fwd", dev, ctypes.byref(d0), v.data_ptr(), log_alpha.data_ptr(), w.data_ptr(),
              _addr(h0), _addr(cu_seqlens), None, None, _addr(chunk_states))
    else:
        _expect_states(chunk_states, v, cu_seqlens, dev)
    like = torch.empty_like
    g = dict(v=like(w), log_alpha=like(w), w=like(w), h0=w.new_empty(sshape))
    _call("gdn2_gated_scan_bwd", dev, r, v.data_ptr(), log_alpha.data_ptr(), w.data_ptr(),
          _addr(chunk_states), _addr(cu_seqlens), dO.data_ptr(), _addr(dhT), *map(_addr, g.values()))
    if again is not None:
        word = workspace.view(-1).view(torch.uint8)[:4].view(torch.int32)
        torch.maximum(word, again[:4].view(torch.int32), out=word)
    return g


@_on_stream
def gated_scan_step(v, log_alpha, w, state, *, out=None):
    """``gdn2_gated_scan_step``: one token; ``state`` ``[B, H, dv]`` fp32 is
    updated in place.  ``v`` ``[B, H, dv]``; ``log_alpha, w`` fp32 of that shape.
    Returns ``out`` ``[B, H, dv]``, the new states in the dtype of ``v``."""
    torch = _torch()
    dev = _cuda_device("v", v)
    io = _io(v.dtype)
    if v.dim() != 3:
        raise ValueError(f"v must be [B, H, dv], got {tuple(v.shape)}")
    _expect("v", v, v.shape, v.dtype, dev)
    for n, t in (("log_alpha", log_alpha), ("w", w), ("state", state)):
        _expect(n, t, v.shape, torch.float32, dev)
    if out is None:
        out = torch.empty_like(v)
    else:
        _expect("out", out, v.shape, v.dtype, dev)
    B, H, dv = v.shape
    d = Desc(B, 1, H, dv, dv, 0, io, None, 0)
    _call("gdn2_gated_scan_step", dev, ctypes.byref(d), v.data_ptr(),
          log_alpha.data_ptr(), w.data_ptr(), state.data_ptr(), out.data_ptr())
    return out
