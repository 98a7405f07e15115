"""Binding of ``libkda_layer.so``: the operators of a KDA layer around the decode step.

``kda_scan`` / ``kda_scan_backward`` (``include/layer/kda_scan.h``) run the
recurrence over long packed sequences and its gradients.  Like the rest of the
package the functions only marshal torch tensors; there is no fallback.
"""
from __future__ import annotations

import ctypes
import math
import os
import threading

import torch

__all__ = ["kda_scan", "kda_scan_backward", "scan_workspace_bytes", "scan_error", "layer_library", "LAYER_LIBRARY_PATH",
           "LAYER_SYMBOLS"]

LAYER_LIBRARY_PATH = os.path.join(os.path.dirname(os.path.abspath(__file__)), "libkda_layer.so")

_P, _I, _I32, _F = ctypes.c_void_p, ctypes.c_int64, ctypes.c_int32, ctypes.c_float


class ScanArgs(ctypes.Structure):
    """ctypes mirror of ``kda_scan_args``."""
    _fields_ = [("q", _P), ("q_row_stride", _I), ("k", _P), ("k_row_stride", _I), ("v", _P), ("v_row_stride", _I),
                ("g", _P), ("g_row_stride", _I), ("beta", _P), ("beta_row_stride", _I), ("cu_seqlens", _P),
                ("initial_state", _P), ("final_state", _P), ("slot_idx", _P), ("num_slots", _I),
                ("out", _P), ("out_row_stride", _I), ("workspace", _P), ("workspace_bytes", _I),
                ("N", _I), ("T", _I), ("HV", _I), ("K", _I), ("V", _I), ("scale", _F), ("save", _I32)]


class ScanGrads(ctypes.Structure):
    """ctypes mirror of ``kda_scan_grads``."""
    _fields_ = [("d_out", _P), ("d_out_row_stride", _I), ("d_final_state", _P),
                ("dq", _P), ("dq_row_stride", _I), ("dk", _P), ("dk_row_stride", _I), ("dv", _P), ("dv_row_stride", _I),
                ("dg", _P), ("dg_row_stride", _I), ("dbeta", _P), ("dbeta_row_stride", _I),
                ("d_initial_state", _P), ("saved", _I32)]


# Every symbol the headers under include/layer/ declare, with its ctypes signature.
LAYER_SYMBOLS = {
    "kda_scan_workspace_bytes": ([_I, _I, _I32, _I, _I, _I, _I32], ctypes.c_int64),
    "kda_scan": ([ctypes.POINTER(ScanArgs), _P], ctypes.c_int),
    "kda_scan_backward": ([ctypes.POINTER(ScanArgs), ctypes.POINTER(ScanGrads), _P], ctypes.c_int),
}

_lock = threading.Lock()
_lib = None


def layer_library() -> ctypes.CDLL:
    """The loaded library (raises if it has not been built)."""
    global _lib
    lib = _lib
    if lib is not None:
        return lib
    with _lock:
        if _lib is None:
            if not os.path.exists(LAYER_LIBRARY_PATH):
                raise RuntimeError(f"{LAYER_LIBRARY_PATH} is missing: build it with "
                                   "`python -m linear_attention_recurrent_decode_b200.build` (no fallback exists)")
            lib = ctypes.CDLL(LAYER_LIBRARY_PATH)
            for name, (argtypes, restype) in LAYER_SYMBOLS.items():
                fn = getattr(lib, name)
                fn.argtypes = argtypes
                fn.restype = restype
            _lib = lib
    return _lib


def _raise(status, where):
    from . import KdaError
    raise KdaError(status, where)


def _stream(stream):
    from . import _stream_handle
    return _stream_handle(stream)


def _on_device(tensors):
    """The current device index; every given tensor must be on it."""
    dev = torch.cuda.current_device() if torch.cuda.is_available() else -1
    for name, t in tensors.items():
        if t is None:
            continue
        if not isinstance(t, torch.Tensor):
            raise TypeError(f"{name} must be a torch.Tensor")
        if not t.is_cuda:
            raise ValueError(f"{name} must be on a CUDA device")
        if t.get_device() != dev:
            raise ValueError(f"{name} is on cuda:{t.get_device()}, the current device is cuda:{dev}")
    return dev


def _row_stride(t, name, dtype, lead, inner):
    """Row stride of a [*lead, *inner] tensor whose rows are evenly strided and dense inside."""
    if t.dtype != dtype:
        raise TypeError(f"{name} must be {dtype}, got {t.dtype}")
    if tuple(t.shape) != (*lead, *inner):
        raise ValueError(f"{name} must have shape {(*lead, *inner)}, got {tuple(t.shape)}")
    want = 1
    for d in range(t.dim() - 1, len(lead) - 1, -1):
        if t.shape[d] > 1 and t.stride(d) != want:
            raise ValueError(f"{name}: each row must be contiguous")
        want *= t.shape[d]
    # the innermost leading dimension longer than 1 sets the stride, the outer ones have to follow it
    rs, rows = None, 1
    for d in range(len(lead) - 1, -1, -1):
        if lead[d] > 1:
            if rs is None:
                rs = t.stride(d)
            elif t.stride(d) != rs * rows:
                raise ValueError(f"{name}: rows must be evenly strided")
        rows *= lead[d]
    return want if rs is None else rs


def _state(t, name, blocks, HV, K, V):
    if t.dtype != torch.float32 or not t.is_contiguous():
        raise TypeError(f"{name} must be a contiguous float32 tensor")
    if t.dim() != 4 or tuple(t.shape[1:]) != (HV, K, V) or (blocks is not None and t.shape[0] != blocks):
        raise ValueError(f"{name} must be [{'blocks' if blocks is None else blocks}, {HV}, {K}, {V}], got {tuple(t.shape)}")
    return t.data_ptr()


def scan_workspace_bytes(T: int, N: int, HV: int, K: int = 128, V: int = 128, *, packed: bool = True,
                         training: bool = False) -> int:
    """Device workspace of ``kda_scan`` for ``N`` sequences: ``T`` is the number of rows of the packed form,
    the tokens of each sequence of the dense one.  ``training``: for ``save=True`` and for the backward pass."""
    n = layer_library().kda_scan_workspace_bytes(N, T, int(packed), HV, K, V, int(training))
    if n < 0:
        raise ValueError(f"kda_scan does not support T={T}, N={N}, HV={HV}, K={K}, V={V}")
    return n


def _scan_args(q, k, v, g, beta, initial_state, cu_seqlens, scale, workspace, training, slot_idx=None):
    if not isinstance(q, torch.Tensor) or not isinstance(v, torch.Tensor):
        raise TypeError("q and v must be torch.Tensors")
    lead_dims = 1 if cu_seqlens is not None else 2
    if q.dim() != lead_dims + 2 or v.dim() != lead_dims + 2:
        raise ValueError("q, k, v must be [rows, HV, K|V] with cu_seqlens, [N, T, HV, K|V] without")
    _on_device(dict(q=q, k=k, v=v, g=g, beta=beta, initial_state=initial_state, cu_seqlens=cu_seqlens, workspace=workspace,
                    slot_idx=slot_idx))
    lead, (HV, K), V = tuple(q.shape[:lead_dims]), q.shape[lead_dims:], v.shape[-1]
    if cu_seqlens is not None:
        if cu_seqlens.dtype != torch.int32 or cu_seqlens.dim() != 1 or cu_seqlens.numel() < 1 or not cu_seqlens.is_contiguous():
            raise TypeError("cu_seqlens must be a contiguous int32 [N + 1] tensor")
        N, T = cu_seqlens.numel() - 1, lead[0]
    else:
        N, T = lead
    bf, f32 = torch.bfloat16, torch.float32
    a = ScanArgs()
    a.q, a.q_row_stride = q.data_ptr(), _row_stride(q, "q", bf, lead, (HV, K))
    a.k, a.k_row_stride = k.data_ptr(), _row_stride(k, "k", bf, lead, (HV, K))
    a.v, a.v_row_stride = v.data_ptr(), _row_stride(v, "v", bf, lead, (HV, V))
    a.g, a.g_row_stride = g.data_ptr(), _row_stride(g, "g", f32, lead, (HV, K))
    a.beta, a.beta_row_stride = beta.data_ptr(), _row_stride(beta, "beta", f32, lead, (HV,))
    if cu_seqlens is not None:
        a.cu_seqlens = cu_seqlens.data_ptr()
    need = scan_workspace_bytes(T, N, HV, K, V, packed=cu_seqlens is not None, training=training)
    if workspace is None:
        workspace = torch.empty(max(need, 16), dtype=torch.uint8, device=q.device)
    if workspace.dtype != torch.uint8 or not workspace.is_contiguous():
        raise TypeError("workspace must be a contiguous uint8 tensor")
    a.workspace, a.workspace_bytes = workspace.data_ptr(), workspace.numel()
    a.N, a.T, a.HV, a.K, a.V = N, T, HV, K, V
    a.scale = float(1.0 / math.sqrt(K) if scale is None else scale)
    return a, lead, (N, HV, K, V), workspace


def kda_scan(q, k, v, g, beta, initial_state=None, *, cu_seqlens=None, slot_idx=None, final_state=None, out=None,
             scale: float | None = None, workspace=None, save: bool = False, stream=None):
    """The recurrence over whole sequences (``kda_scan`` of the C ABI); returns ``(out, final_state)``.

    Packed: q, k ``[rows, HV, K]``, v ``[rows, HV, V]`` (bf16), g ``[rows, HV, K]``, beta ``[rows, HV]`` (fp32) with
    ``cu_seqlens`` (device int32 ``[N + 1]``).  Dense: the same with ``[N, T, ...]`` and no ``cu_seqlens``.  Rows may be
    strided views (slices of one packed buffer).  Rows outside every sequence are neither read nor written.

    States are fp32 ``[N, HV, K, V]``; ``initial_state=None`` starts from zeros, ``final_state`` is allocated if not
    given.  For serving, ``slot_idx`` (device int32 ``[N]``) names blocks of a pool: ``initial_state`` is the pool,
    updated in place unless another ``final_state`` pool is given; a slot outside it makes the sequence inactive (zero
    outputs).  ``workspace``: a device uint8 tensor of :func:`scan_workspace_bytes` bytes (allocated if not given);
    ``save=True`` (training size) keeps in it what :func:`kda_scan_backward` reads."""
    a, lead, (N, HV, K, V), workspace = _scan_args(q, k, v, g, beta, initial_state, cu_seqlens, scale, workspace, save, slot_idx)
    _on_device(dict(final_state=final_state, out=out))
    blocks = N
    if slot_idx is not None:
        if initial_state is None:
            raise ValueError("slot_idx needs initial_state, the state pool")
        if slot_idx.dtype != torch.int32 or tuple(slot_idx.shape) != (N,) or not slot_idx.is_contiguous():
            raise TypeError(f"slot_idx must be a contiguous int32 [{N}] tensor")
        blocks = initial_state.shape[0]
        a.slot_idx, a.num_slots = slot_idx.data_ptr(), blocks
        if final_state is None:
            final_state = initial_state
    if final_state is None:
        final_state = torch.empty((N, HV, K, V), dtype=torch.float32, device=q.device)
    if initial_state is not None:
        a.initial_state = _state(initial_state, "initial_state", blocks, HV, K, V)
    a.final_state = _state(final_state, "final_state", blocks, HV, K, V)
    if out is None:
        out = torch.empty((*lead, HV, V), dtype=torch.bfloat16, device=q.device)
    a.out, a.out_row_stride = out.data_ptr(), _row_stride(out, "out", torch.bfloat16, lead, (HV, V))
    a.save = int(save)
    st = layer_library().kda_scan(ctypes.byref(a), _stream(stream))
    if st:
        _raise(st, "kda_scan")
    return out, final_state


def kda_scan_backward(d_out, q, k, v, g, beta, initial_state=None, *, d_final_state=None, cu_seqlens=None,
                      scale: float | None = None, workspace=None, saved: bool = False, dq=None, dk=None, dv=None, dg=None,
                      dbeta=None, d_initial_state=None, stream=None):
    """Gradients of :func:`kda_scan`: returns ``(dq, dk, dv, dg, dbeta, d_initial_state)``.

    ``d_out`` (bf16, like ``out``) and ``d_final_state`` (fp32, like the states; None: zeros) are the loss's gradients.
    The forward call's inputs, ``cu_seqlens`` and ``scale`` are given again.  With ``saved=True``, ``workspace`` is the
    one a ``kda_scan(..., save=True)`` of the same inputs left; otherwise the forward pass is computed again first.
    Gradients are allocated if not given; given ones may be strided views.  Gradient rows outside every sequence are left
    as they were."""
    if saved and workspace is None:
        raise ValueError("saved=True needs the forward call's workspace")
    a, lead, (N, HV, K, V), workspace = _scan_args(q, k, v, g, beta, initial_state, cu_seqlens, scale, workspace, True)
    _on_device(dict(d_out=d_out, d_final_state=d_final_state, dq=dq, dk=dk, dv=dv, dg=dg, dbeta=dbeta,
                    d_initial_state=d_initial_state))
    bf, f32 = torch.bfloat16, torch.float32
    if initial_state is not None:
        a.initial_state = _state(initial_state, "initial_state", N, HV, K, V)
    d = ScanGrads()
    d.d_out, d.d_out_row_stride = d_out.data_ptr(), _row_stride(d_out, "d_out", bf, lead, (HV, V))
    if d_final_state is not None:
        d.d_final_state = _state(d_final_state, "d_final_state", N, HV, K, V)
    got = []
    for name, t, dtype, inner in (("dq", dq, bf, (HV, K)), ("dk", dk, bf, (HV, K)), ("dv", dv, bf, (HV, V)),
                                  ("dg", dg, f32, (HV, K)), ("dbeta", dbeta, f32, (HV,))):
        if t is None:
            t = torch.empty((*lead, *inner), dtype=dtype, device=q.device)
        setattr(d, name, t.data_ptr())
        setattr(d, name + "_row_stride", _row_stride(t, name, dtype, lead, inner))
        got.append(t)
    if d_initial_state is None:
        d_initial_state = torch.empty((N, HV, K, V), dtype=f32, device=q.device)
    d.d_initial_state = _state(d_initial_state, "d_initial_state", N, HV, K, V)
    d.saved = int(saved)
    st = layer_library().kda_scan_backward(ctypes.byref(a), ctypes.byref(d), _stream(stream))
    if st:
        _raise(st, "kda_scan_backward")
    return (*got, d_initial_state)


def scan_error(workspace) -> int:
    """The error word of a workspace that the caller zeroed before the calls it watches: 1 if a kernel gave up a
    bounded wait.  Waits for the device's work in flight."""
    return int(workspace[:4].view(torch.int32).item())
