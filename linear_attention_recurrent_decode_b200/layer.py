"""Binding of ``libkda_layer.so``: the operators of a KDA layer around the decode step.

``kda_scan`` / ``kda_scan_backward`` (``include/layer/kda_scan.h``) run the
recurrence over long packed sequences and its gradients;
``kda_qk_norm_rope`` / ``kda_qk_norm_rope_backward`` (``include/layer/kda_qk.h``)
the per-head norm of its queries and keys with the position rotation.  Like the
rest of the package the functions only marshal torch tensors; there is no
fallback.  No call records an autograd graph, whatever its inputs require: a
program that trains calls the backward functions itself, for instance in the
``backward`` of a ``torch.autograd.Function`` of its own (once differentiable).
"""
from __future__ import annotations

import ctypes
import functools
import math
import os
import threading

import torch

__all__ = ["kda_scan", "kda_scan_backward", "scan_workspace_bytes", "scan_error", "kda_qk_norm_rope", "kda_qk_norm_rope_backward",
           "rope_frequencies", "layer_library", "LAYER_LIBRARY_PATH", "LAYER_SYMBOLS"]

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


class QkTensor(ctypes.Structure):
    """ctypes mirror of ``kda_qk_tensor``."""
    _fields_ = [("x", _P), ("x_row_stride", _I), ("y", _P), ("y_row_stride", _I), ("dy", _P), ("dy_row_stride", _I),
                ("dx", _P), ("dx_row_stride", _I), ("weight", _P), ("dweight", _P), ("heads", _I)]


class QkArgs(ctypes.Structure):
    """ctypes mirror of ``kda_qk_args``."""
    _fields_ = [("q", QkTensor), ("k", QkTensor), ("rows", _I), ("D", _I), ("rot", _I), ("positions", _P), ("inv_freq", _P),
                ("positions_64", _I32), ("norm", _I32), ("interleaved", _I32), ("eps", _F), ("rope_scale", _F),
                ("workspace", _P), ("workspace_bytes", _I)]


QK_NORMS = {"none": 0, "l2": 1, "rms": 2}

# Every symbol the headers under include/layer/ declare, with its ctypes signature.
LAYER_SYMBOLS = {
    "kda_scan_workspace_bytes": ([_I, _I, _I32, _I, _I, _I, _I32], ctypes.c_int64),
    "kda_scan": ([ctypes.POINTER(ScanArgs), _P], ctypes.c_int),
    "kda_scan_backward": ([ctypes.POINTER(ScanArgs), ctypes.POINTER(ScanGrads), _P], ctypes.c_int),
    "kda_qk_workspace_bytes": ([_I], ctypes.c_int64),
    "kda_qk_norm_rope": ([ctypes.POINTER(QkArgs), _P], ctypes.c_int),
    "kda_qk_norm_rope_backward": ([ctypes.POINTER(QkArgs), _P], ctypes.c_int),
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


# The per-call path below is kept to a few microseconds: one comparison per tensor, the reason only on failure.
_BF16, _F32 = torch.bfloat16, torch.float32


def _device() -> int:
    """The current device's index (-2 without CUDA, which no tensor's is: every one is then refused)."""
    return torch.cuda.current_device() if torch.cuda.is_initialized() or torch.cuda.is_available() else -2


def _on_stream(call):
    """Runs a call given a ``stream`` with that stream current, so that what it allocates belongs to the stream too."""
    @functools.wraps(call)
    def run(*args, stream=None, **kwargs):
        if stream is None:
            return call(*args, **kwargs)
        from . import _stream_handle
        handle = _stream_handle(stream).value or 0  # refuses another device's stream
        with torch.cuda.stream(torch.cuda.ExternalStream(handle) if handle else torch.cuda.default_stream()):
            return call(*args, **kwargs)
    return run


def _on_device(t, name, dev):
    """Refuses a tensor that is not on the current device."""
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    if t.get_device() != dev or not t.is_cuda:
        if not t.is_cuda:
            raise ValueError(f"{name} must be on a CUDA device")
        raise ValueError(f"{name} is on cuda:{t.get_device()}, the current device is cuda:{dev}")


def _row_stride(t, name, dtype, shape, lead, dev):
    """Row stride of a tensor of this shape whose rows (over the first ``lead`` dimensions) are evenly strided and
    dense inside."""
    if type(t) is not torch.Tensor or t.get_device() != dev:
        _on_device(t, name, dev)
    if t.dtype != dtype:
        raise TypeError(f"{name} must be {dtype}, got {t.dtype}")
    if t.shape != shape:
        raise ValueError(f"{name} must have shape {tuple(shape)}, got {tuple(t.shape)}")
    if t.is_contiguous():
        return shape[-1] if lead == len(shape) - 1 else shape[-1] * shape[-2]  # rows of one or two dimensions
    want, strides = 1, t.stride()
    if lead == 1 and len(strides) == 3 and shape[0] > 1 and strides[2] == 1 and strides[1] == shape[2]:
        return strides[0]  # columns of one packed buffer
    for d in range(len(shape) - 1, lead - 1, -1):
        if shape[d] > 1 and strides[d] != want:
            raise ValueError(f"{name}: each row must be contiguous")
        want *= shape[d]
    # the innermost leading dimension longer than 1 sets the stride, the outer ones have to follow it
    rs, rows = None, 1
    for d in range(lead - 1, -1, -1):
        if shape[d] > 1:
            if rs is None:
                rs = strides[d]
            elif strides[d] != rs * rows:
                raise ValueError(f"{name}: rows must be evenly strided")
        rows *= shape[d]
    return want if rs is None else rs


def _empty(x, shape=None, dtype=None):
    """A contiguous tensor of x's (or this) shape and type on x's device."""
    if shape is None:
        return torch.empty_like(x, dtype=dtype, memory_format=torch.contiguous_format)
    return x.new_empty(shape, dtype=dtype)


def _state(t, name, blocks, HV, K, V, dev):
    if not (type(t) is torch.Tensor and t.get_device() == dev):
        _on_device(t, name, dev)
    if t.dtype != _F32 or not t.is_contiguous():
        raise TypeError(f"{name} must be a contiguous float32 tensor")
    if t.dim() != 4 or t.shape[1:] != (HV, K, V) or (blocks is not None and t.shape[0] != blocks):
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


def _scan_args(q, k, v, g, beta, cu_seqlens, scale, workspace, training):
    """The arguments both calls share, the leading shape, (N, HV, K, V), the workspace and the current device."""
    if not isinstance(q, torch.Tensor) or not isinstance(v, torch.Tensor):
        raise TypeError("q and v must be torch.Tensors")
    n = 1 if cu_seqlens is not None else 2
    if q.dim() != n + 2 or v.dim() != n + 2:
        raise ValueError("q, k, v must be [rows, HV, K|V] with cu_seqlens, [N, T, HV, K|V] without")
    dev, qs, vs = _device(), q.shape, v.shape
    lead, HV, K, V = qs[:n], qs[n], qs[n + 1], vs[n + 1]
    a = ScanArgs()
    if cu_seqlens is not None:
        _on_device(cu_seqlens, "cu_seqlens", dev)
        if cu_seqlens.dtype != torch.int32 or cu_seqlens.dim() != 1 or cu_seqlens.numel() < 1 or not cu_seqlens.is_contiguous():
            raise TypeError("cu_seqlens must be a contiguous int32 [N + 1] tensor")
        N, T = cu_seqlens.numel() - 1, lead[0]
        a.cu_seqlens = cu_seqlens.data_ptr()
    else:
        N, T = lead
    a.q_row_stride = _row_stride(q, "q", _BF16, qs, n, dev)
    a.k_row_stride = _row_stride(k, "k", _BF16, qs, n, dev)
    a.v_row_stride = _row_stride(v, "v", _BF16, (*lead, HV, V), n, dev)
    a.g_row_stride = _row_stride(g, "g", _F32, qs, n, dev)
    a.beta_row_stride = _row_stride(beta, "beta", _F32, qs[:-1], n, dev)
    a.q, a.k, a.v, a.g, a.beta = q.data_ptr(), k.data_ptr(), v.data_ptr(), g.data_ptr(), beta.data_ptr()
    if workspace is None:
        need = scan_workspace_bytes(T, N, HV, K, V, packed=cu_seqlens is not None, training=training)
        workspace = q.new_empty(max(need, 16), dtype=torch.uint8)
    else:
        _on_device(workspace, "workspace", dev)
        if workspace.dtype != torch.uint8 or not workspace.is_contiguous():
            raise TypeError("workspace must be a contiguous uint8 tensor")
    a.workspace, a.workspace_bytes = workspace.data_ptr(), workspace.numel()
    a.N, a.T, a.HV, a.K, a.V = N, T, HV, K, V
    a.scale = 1.0 / math.sqrt(K) if scale is None else scale
    return a, lead, (N, HV, K, V), workspace, dev


@_on_stream
def kda_scan(q, k, v, g, beta, initial_state=None, *, cu_seqlens=None, slot_idx=None, final_state=None, out=None,
             scale: float | None = None, workspace=None, save: bool = False, stream=None):
    """The recurrence over whole sequences (``kda_scan`` of the C ABI); returns ``(out, final_state)``, without an autograd
    graph.

    Packed: q, k ``[rows, HV, K]``, v ``[rows, HV, V]`` (bf16), g ``[rows, HV, K]``, beta ``[rows, HV]`` (fp32) with
    ``cu_seqlens`` (device int32 ``[N + 1]``).  Dense: the same with ``[N, T, ...]`` and no ``cu_seqlens``.  Rows may be
    strided views (slices of one packed buffer).  Rows outside every sequence are neither read nor written: in an ``out``
    allocated here they hold anything.

    States are fp32 ``[N, HV, K, V]``; ``initial_state=None`` starts from zeros, ``final_state`` is allocated if not
    given.  For serving, ``slot_idx`` (device int32 ``[N]``) names blocks of a pool: ``initial_state`` is the pool,
    updated in place unless another ``final_state`` pool is given; a slot outside it makes the sequence inactive (zero
    outputs).  ``workspace``: a device uint8 tensor of :func:`scan_workspace_bytes` bytes (allocated if not given);
    ``save=True`` (training size) keeps in it what :func:`kda_scan_backward` reads."""
    a, lead, (N, HV, K, V), workspace, dev = _scan_args(q, k, v, g, beta, cu_seqlens, scale, workspace, save)
    blocks = N
    if slot_idx is not None:
        if initial_state is None:
            raise ValueError("slot_idx needs initial_state, the state pool")
        _on_device(slot_idx, "slot_idx", dev)
        _on_device(initial_state, "initial_state", dev)
        if slot_idx.dtype != torch.int32 or slot_idx.shape != (N,) or not slot_idx.is_contiguous():
            raise TypeError(f"slot_idx must be a contiguous int32 [{N}] tensor")
        blocks = initial_state.shape[0]
        a.slot_idx, a.num_slots = slot_idx.data_ptr(), blocks
        if final_state is None:
            final_state = initial_state
    if initial_state is not None:
        a.initial_state = _state(initial_state, "initial_state", blocks, HV, K, V, dev)
    if final_state is None:
        final_state = _empty(q, (N, HV, K, V), _F32) if initial_state is None else _empty(initial_state)
    a.final_state = _state(final_state, "final_state", blocks, HV, K, V, dev)
    if out is None:
        out = _empty(v)
    a.out_row_stride = _row_stride(out, "out", _BF16, v.shape, len(lead), dev)
    a.out = out.data_ptr()
    a.save = bool(save)
    st = layer_library().kda_scan(ctypes.byref(a), torch._C._cuda_getCurrentRawStream(dev))
    if st:
        _raise(st, "kda_scan")
    return out, final_state


@_on_stream
def kda_scan_backward(d_out, q, k, v, g, beta, initial_state=None, *, d_final_state=None, cu_seqlens=None,
                      scale: float | None = None, workspace=None, saved: bool = False, dq=None, dk=None, dv=None, dg=None,
                      dbeta=None, d_initial_state=None, stream=None):
    """Gradients of :func:`kda_scan`: returns ``(dq, dk, dv, dg, dbeta, d_initial_state)``.

    ``d_out`` (bf16, like ``out``) and ``d_final_state`` (fp32, like the states; None: zeros) are the loss's gradients.
    The forward call's inputs, ``cu_seqlens`` and ``scale`` are given again.  With ``saved=True``, ``workspace`` is the
    one a ``kda_scan(..., save=True)`` of the same inputs left (364 KB for every 64 tokens and head); otherwise the forward
    pass is computed again first, about 1.8 times the time.
    Gradients are allocated if not given; given ones may be strided views.  Gradient rows outside every sequence are left
    as they were, and hold anything if allocated here: where a batch is padded and all rows are summed over later, give
    zeroed gradients."""
    if saved and workspace is None:
        raise ValueError("saved=True needs the forward call's workspace")
    a, lead, (N, HV, K, V), workspace, dev = _scan_args(q, k, v, g, beta, cu_seqlens, scale, workspace, True)
    n = len(lead)
    if initial_state is not None:
        a.initial_state = _state(initial_state, "initial_state", N, HV, K, V, dev)
    d = ScanGrads()
    d.d_out_row_stride = _row_stride(d_out, "d_out", _BF16, v.shape, n, dev)
    d.d_out = d_out.data_ptr()
    if d_final_state is not None:
        d.d_final_state = _state(d_final_state, "d_final_state", N, HV, K, V, dev)
    if dq is None:
        dq = _empty(q)
    if dk is None:
        dk = _empty(q)
    if dv is None:
        dv = _empty(v)
    if dg is None:
        dg = _empty(g)
    if dbeta is None:
        dbeta = _empty(beta)
    d.dq_row_stride = _row_stride(dq, "dq", _BF16, q.shape, n, dev)
    d.dk_row_stride = _row_stride(dk, "dk", _BF16, q.shape, n, dev)
    d.dv_row_stride = _row_stride(dv, "dv", _BF16, v.shape, n, dev)
    d.dg_row_stride = _row_stride(dg, "dg", _F32, g.shape, n, dev)
    d.dbeta_row_stride = _row_stride(dbeta, "dbeta", _F32, beta.shape, n, dev)
    d.dq, d.dk, d.dv, d.dg, d.dbeta = dq.data_ptr(), dk.data_ptr(), dv.data_ptr(), dg.data_ptr(), dbeta.data_ptr()
    if d_initial_state is None:
        d_initial_state = _empty(q, (N, HV, K, V), _F32)
    d.d_initial_state = _state(d_initial_state, "d_initial_state", N, HV, K, V, dev)
    d.saved = bool(saved)
    st = layer_library().kda_scan_backward(ctypes.byref(a), ctypes.byref(d), torch._C._cuda_getCurrentRawStream(dev))
    if st:
        _raise(st, "kda_scan_backward")
    return dq, dk, dv, dg, dbeta, d_initial_state


def scan_error(workspace) -> int:
    """The error word of a workspace that the caller zeroed before the calls it watches: 1 if a kernel gave up a
    bounded wait.  Waits for the device's work in flight."""
    return int(workspace[:4].view(torch.int32).item())


def rope_frequencies(rot: int, base: float = 10000.0, *, factor: float = 1.0, trained_context: int | None = None,
                     fast_turns: float = 32.0, slow_turns: float = 1.0, device=None):
    """``(inv_freq, rope_scale)`` of a rotation of ``rot`` components: ``base ** (-2 i / rot)`` in float64.

    ``factor`` > 1 stretches the positions for contexts that much longer than the model was trained on: without
    ``trained_context`` every frequency is divided by it; with it only those that make fewer than ``slow_turns`` turns in
    ``trained_context`` tokens, those that make more than ``fast_turns`` stay, a linear ramp over the pair index lies
    between, and ``rope_scale`` is ``0.1 ln(factor) + 1`` (the ramped scaling published as YaRN)."""
    if rot < 0 or rot % 2:
        raise ValueError(f"rot must be even and >= 0, got {rot}")
    if factor < 1.0 or base <= 1.0:
        raise ValueError("factor must be >= 1 and base > 1")
    freq = float(base) ** (-torch.arange(0, rot, 2, dtype=torch.float64) / max(rot, 1))
    scale = 1.0
    if factor > 1.0 and trained_context is None:
        freq = freq / factor
    elif factor > 1.0:
        def pair_of(turns):  # the (fractional) pair that makes this many turns in the trained context
            return rot * math.log(trained_context / (turns * 2 * math.pi)) / (2 * math.log(base))
        lo, hi = max(math.floor(pair_of(fast_turns)), 0), min(math.ceil(pair_of(slow_turns)), rot - 1)
        ramp = ((torch.arange(rot // 2, dtype=torch.float64) - lo) / max(hi - lo, 1e-3)).clamp(0, 1)
        freq = freq * (1 - ramp) + freq / factor * ramp
        scale = 0.1 * math.log(factor) + 1.0
    return (freq if device is None else freq.to(device)), scale


def _qk_args(q, k, norm, eps, q_weight, k_weight, positions, inv_freq, interleaved, rope_scale):
    """The arguments both calls share, the number of leading dimensions, D, and the current device."""
    if not isinstance(q, torch.Tensor) or q.dim() < 3:
        raise TypeError("q must be a torch.Tensor [..., heads, D]")
    if norm not in QK_NORMS:
        raise ValueError(f"norm must be one of {', '.join(QK_NORMS)}, got {norm!r}")
    dev, D, n = _device(), q.shape[-1], q.dim() - 2
    lead = q.shape[:n]
    a = QkArgs()
    a.rows = math.prod(lead)
    a.D, a.norm, a.eps, a.rope_scale, a.interleaved = D, QK_NORMS[norm], eps, rope_scale, bool(interleaved)
    for name, x, w, t in (("q", q, q_weight, a.q), ("k", k, k_weight, a.k)):
        if x is None:
            if w is not None:
                raise ValueError(f"{name}_weight without {name}")
            continue
        if not isinstance(x, torch.Tensor) or x.dim() != q.dim() or x.shape[:-2] != lead or x.shape[-1] != D:
            raise ValueError(f"{name} must be [{', '.join(map(str, lead))}, heads, {D}]")
        t.x_row_stride = _row_stride(x, name, _BF16, x.shape, n, dev)
        t.heads, t.x = x.shape[-2], x.data_ptr()
        if w is not None:
            _on_device(w, name + "_weight", dev)
            if w.dtype != _BF16 or w.shape != (D,) or not w.is_contiguous():
                raise TypeError(f"{name}_weight must be a contiguous bfloat16 [{D}] tensor")
            if norm == "none":
                raise ValueError(f"{name}_weight needs a norm")
            t.weight = w.data_ptr()
    if inv_freq is not None:
        _on_device(inv_freq, "inv_freq", dev)
        if inv_freq.dtype != torch.float64 or inv_freq.dim() != 1 or not inv_freq.is_contiguous():
            raise TypeError("inv_freq must be a contiguous float64 [rot / 2] tensor")
        if positions is None:
            raise ValueError("inv_freq needs positions")
        _on_device(positions, "positions", dev)
        if positions.dtype not in (torch.int32, torch.int64) or positions.shape != lead or not positions.is_contiguous():
            raise TypeError(f"positions must be a contiguous int32 or int64 tensor of shape {tuple(lead)}")
        a.rot = 2 * inv_freq.numel()
        a.inv_freq, a.positions, a.positions_64 = inv_freq.data_ptr(), positions.data_ptr(), positions.dtype == torch.int64
    elif positions is not None:
        raise ValueError("positions need inv_freq")
    return a, n, D, dev


@_on_stream
def kda_qk_norm_rope(q, k=None, *, norm: str = "l2", eps: float = 1e-6, q_weight=None, k_weight=None, positions=None,
                     inv_freq=None, interleaved: bool = False, rope_scale: float = 1.0, q_out=None, k_out=None, stream=None):
    """Per-head norm of queries and keys and the position rotation in one pass; returns ``(q, k)`` as the decode step,
    the prefill and the scan take them (``k`` None if not given).

    q ``[..., heads, D]``, k ``[..., k_heads, D]`` (bf16; rows may be strided views of one packed buffer).  ``norm``:
    ``"l2"`` x / sqrt(sum x^2 + eps), ``"rms"`` x / sqrt(mean x^2 + eps), ``"none"``; ``q_weight`` / ``k_weight`` (bf16
    ``[D]``) multiply after it.  ``inv_freq`` (float64 ``[rot / 2]``, :func:`rope_frequencies`, ``rot`` a multiple of 16)
    turns the first ``rot`` components of each head by ``positions`` (int32 or int64, the leading shape) in halves or ``interleaved`` pairs, times
    ``rope_scale``.  Outputs are allocated if not given; ``q_out=q`` / ``k_out=k`` work in place."""
    a, n, D, dev = _qk_args(q, k, norm, eps, q_weight, k_weight, positions, inv_freq, interleaved, rope_scale)
    got = []
    for name, x, y, t in (("q_out", q, q_out, a.q), ("k_out", k, k_out, a.k)):
        if x is None:
            if y is not None:
                raise ValueError("k_out without k")
        elif y is None:
            y = _empty(x)
            t.y, t.y_row_stride = y.data_ptr(), t.heads * D
        else:
            t.y_row_stride = _row_stride(y, name, _BF16, x.shape, n, dev)
            t.y = y.data_ptr()
        got.append(y)
    st = layer_library().kda_qk_norm_rope(ctypes.byref(a), torch._C._cuda_getCurrentRawStream(dev))
    if st:
        _raise(st, "kda_qk_norm_rope")
    return tuple(got)


@_on_stream
def kda_qk_norm_rope_backward(d_q_out, d_k_out, q, k=None, *, norm: str = "l2", eps: float = 1e-6, q_weight=None,
                              k_weight=None, positions=None, inv_freq=None, interleaved: bool = False,
                              rope_scale: float = 1.0, dq=None, dk=None, workspace=None, stream=None):
    """Gradients of :func:`kda_qk_norm_rope` from those of its outputs: returns ``(dq, dk, d_q_weight, d_k_weight)``, the
    last two fp32 ``[D]`` (None without the weight).  q, k and the options are the forward call's; ``dq`` / ``dk`` are
    allocated if not given (``dq=d_q_out`` / ``dk=d_k_out`` work in place), and so is ``workspace`` (device uint8, 4096 D
    bytes), used only with weights."""
    a, n, D, dev = _qk_args(q, k, norm, eps, q_weight, k_weight, positions, inv_freq, interleaved, rope_scale)
    got, dws = [], []
    for name, x, dy, dx, w, t in (("q", q, d_q_out, dq, q_weight, a.q), ("k", k, d_k_out, dk, k_weight, a.k)):
        dw = None
        if x is None:
            if dy is not None or dx is not None:
                raise ValueError("gradients of k without k")
        else:
            t.dy_row_stride = _row_stride(dy, f"d_{name}_out", _BF16, x.shape, n, dev)
            t.dy = dy.data_ptr()
            if dx is None:
                dx = _empty(x)
                t.dx, t.dx_row_stride = dx.data_ptr(), t.heads * D
            else:
                t.dx_row_stride = _row_stride(dx, "d" + name, _BF16, x.shape, n, dev)
                t.dx = dx.data_ptr()
            if w is not None:
                dw = x.new_empty(D, dtype=_F32)
                t.dweight = dw.data_ptr()
        got.append(dx)
        dws.append(dw)
    if q_weight is not None or k_weight is not None:
        if workspace is None:
            workspace = q.new_empty(max(layer_library().kda_qk_workspace_bytes(D), 16), dtype=torch.uint8)
        else:
            _on_device(workspace, "workspace", dev)
            if workspace.dtype != torch.uint8 or not workspace.is_contiguous():
                raise TypeError("workspace must be a contiguous uint8 tensor")
        a.workspace, a.workspace_bytes = workspace.data_ptr(), workspace.numel()
    st = layer_library().kda_qk_norm_rope_backward(ctypes.byref(a), torch._C._cuda_getCurrentRawStream(dev))
    if st:
        _raise(st, "kda_qk_norm_rope_backward")
    return (*got, *dws)
