"""The gated delta rule with one decay per value head and token (scalar gate):
binding of the kda_gdn_* entry points. Argument marshalling only, as the rest
of this package; the kernels are in csrc/kda_gdn_*.hip.

Per value head, S FP32 [K, V]:
    S_t = e^{g_t} (I - beta_t k_t k_t^T) S_{t-1} + beta_t k_t v_t^T,   o_t = S_t^T q_t / sqrt(K)

  chunk_gdn       chunked forward (prefill, training; K and V in {64, 128})
  chunk_gdn_bwd   its backward
  recurrent_gdn   token-sequential forward (decode; K and V up to 256)
"""
from __future__ import annotations

import ctypes
from typing import Optional, Tuple

import torch

from . import (KDA_BF16, KDA_FP32, KDA_GATE_NAT, KDA_GATE_RAW, KdaDims, KdaError, _cu_dims, _I32_MAX, _lib,
               _nbytes)


def _ptr(t):
    """A tensor's address (None passes): what a c_void_p argument takes."""
    return None if t is None else t.data_ptr()


_DT = {torch.bfloat16: KDA_BF16, torch.float32: KDA_FP32}


class KdaGdnGate(ctypes.Structure):
    """kda_gdn_gate: the gate operand of the scalar-gate entry points."""
    _fields_ = [("x", ctypes.c_void_p), ("A_log", ctypes.c_void_p), ("dt_bias", ctypes.c_void_p),
                ("dtype", ctypes.c_int32), ("kind", ctypes.c_int32)]


def _stream_of(index: int) -> int:
    return torch.cuda.current_stream(index).cuda_stream


# the same handle without a Stream object around it: 0.1 instead of 2.8 us, of
# a single-token call's 12
_stream_of = getattr(torch._C, "_cuda_getCurrentRawStream", _stream_of)


class _OnDevice:
    """Makes a tensor's device the current one for the call (stream, launch)."""

    def __init__(self, t: torch.Tensor):
        self._index = t.get_device()

    def __enter__(self):
        self._old = torch.cuda.current_device()
        if self._old != self._index:
            torch.cuda.set_device(self._index)
        return _stream_of(self._index)

    def __exit__(self, *exc):
        if self._old != self._index:
            torch.cuda.set_device(self._old)


def _want(t, name, shape, dtype, device):
    """A contiguous tensor of exactly this shape, dtype and device (None passes)."""
    if t is None or (type(t) is torch.Tensor and t.dtype is dtype and t.shape == shape and t.device == device
                     and t.is_contiguous()):
        return
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    if t.dtype != dtype:
        raise TypeError(f"{name} must be {dtype}, got {t.dtype}")
    if t.shape != shape:
        raise ValueError(f"{name} must have shape {tuple(shape)}, got {tuple(t.shape)}")
    if t.device != device:
        raise ValueError(f"{name} is on {t.device}, the first input on {device}")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")


def _check_args(q, k, v, gate, beta, initial_state, cu_seqlens, raw, A_log, dt_bias, o=None, final_state=None,
                do=None, dht=None):
    """Every dtype, shape, device and layout the C ABI cannot see. Returns the
    kda_dims and kda_gdn_gate of the call."""
    for t, n in ((q, "q"), (k, "k"), (v, "v"), (beta, "beta"), (gate, "gate")):
        if not isinstance(t, torch.Tensor):
            raise TypeError(f"{n} must be a torch.Tensor")
    if q.dim() != 4 or v.dim() != 4:
        raise ValueError("q must be [B, T, H, K] and v [B, T, HV, V]")
    B, T, H, K = q.shape
    HV, V = v.shape[2], v.shape[3]
    if H < 1 or HV < 1 or HV % H != 0:
        raise ValueError(f"HV ({HV}) must be a positive multiple of H ({H})")
    dt, dev = q.dtype, q.device
    if dt not in _DT:
        raise TypeError(f"q must be bfloat16 or float32, got {dt}")
    if gate.dtype not in (torch.float32, dt):
        raise TypeError(f"gate must be float32 or {dt}, got {gate.dtype}")
    if not raw and (A_log is not None or dt_bias is not None):
        raise ValueError("A_log and dt_bias need use_gate_in_kernel=True (a raw gate input)")
    N = _cu_dims(cu_seqlens, B)
    if max(B, T, H, HV, K, V, N) > _I32_MAX:
        raise ValueError("every size must fit the C ABI's int32 fields")
    sv, sb, st, gdt = (B, T, HV, V), (B, T, HV), (N, HV, K, V), gate.dtype
    _want(q, "q", (B, T, H, K), dt, dev)
    _want(k, "k", (B, T, H, K), dt, dev)
    _want(v, "v", sv, dt, dev)
    _want(beta, "beta", sb, dt, dev)
    _want(gate, "gate", sb, gdt, dev)
    if cu_seqlens is not None:
        _want(cu_seqlens, "cu_seqlens", (N + 1,), torch.int32, dev)
    _want(A_log, "A_log", (HV,), gdt, dev)
    _want(dt_bias, "dt_bias", (HV,), gdt, dev)
    _want(initial_state, "initial_state", st, torch.float32, dev)
    _want(final_state, "final_state", st, torch.float32, dev)
    _want(o, "o", sv, dt, dev)
    _want(do, "do", sv, dt, dev)
    _want(dht, "dht", st, torch.float32, dev)
    if not q.is_cuda:
        raise ValueError("q must be a device tensor")
    g = KdaGdnGate(gate.data_ptr(), None if A_log is None else A_log.data_ptr(),
                   None if dt_bias is None else dt_bias.data_ptr(), _DT[gdt],
                   KDA_GATE_RAW if raw else KDA_GATE_NAT)
    return KdaDims(B, T, N, H, HV, K, V), g


def chunk_gdn_workspace_bytes(q: torch.Tensor, v: torch.Tensor, cu_seqlens=None, backward: bool = False) -> int:
    """Workspace bytes of chunk_gdn, or (backward=True) of chunk_gdn_bwd. 0 for
    sizes the chunked kernels do not take."""
    B, T, H, K = q.shape
    d = KdaDims(B, T, _cu_dims(cu_seqlens, B), H, v.shape[2], K, v.shape[3])
    return int(_lib().kda_gdn_chunk_workspace_bytes(ctypes.byref(d), _DT[q.dtype], int(bool(backward))))


def _workspace(ws, need, like, name="workspace"):
    if ws is None:
        return torch.empty(max(need, 1), device=like.device, dtype=torch.uint8)
    if not isinstance(ws, torch.Tensor) or ws.device != like.device or not ws.is_contiguous():
        raise ValueError(f"{name} must be a contiguous tensor on {like.device}")
    return ws


def chunk_gdn(q, k, v, gate, beta, initial_state=None, *, cu_seqlens=None, output_final_state: bool = False,
              use_gate_in_kernel: bool = False, A_log: Optional[torch.Tensor] = None,
              dt_bias: Optional[torch.Tensor] = None, qk_l2norm: bool = False,
              o: Optional[torch.Tensor] = None, final_state: Optional[torch.Tensor] = None,
              workspace: Optional[torch.Tensor] = None) -> Tuple[torch.Tensor, Optional[torch.Tensor]]:
    """Chunked forward (kda_gdn_chunk_fwd). q, k [B, T, H, K], v [B, T, HV, V]
    and beta [B, T, HV] in one dtype (bfloat16 or float32); gate [B, T, HV] in
    float32 or that dtype: the natural-log gate g, or with
    use_gate_in_kernel=True the raw input x of g = -exp(A_log) softplus(x +
    dt_bias) (A_log, dt_bias [HV] in the gate's dtype, each optional).
    qk_l2norm=True normalises q and k in the kernel. cu_seqlens packs sequences
    into one batch row as in chunk_kda. A `workspace` passed in must hold
    chunk_gdn_workspace_bytes(); calls that may overlap need one each.
    Returns (o, final_state or None)."""
    d, g = _check_args(q, k, v, gate, beta, initial_state, cu_seqlens, use_gate_in_kernel, A_log, dt_bias, o,
                       final_state)
    dt, lib = _DT[q.dtype], _lib()
    if o is None:
        o = torch.empty_like(v)
    if not output_final_state:
        final_state = None
    elif final_state is None:
        final_state = torch.empty((d.N, d.HV, d.K, d.V), device=q.device, dtype=torch.float32)
    ws = _workspace(workspace, lib.kda_gdn_chunk_workspace_bytes(ctypes.byref(d), dt, 0), q)
    with _OnDevice(q) as stream:
        rc = lib.kda_gdn_chunk_fwd(ctypes.byref(d), dt, _ptr(q), _ptr(k), _ptr(v), ctypes.byref(g),
                                   int(bool(qk_l2norm)), _ptr(beta), _ptr(initial_state), _ptr(cu_seqlens),
                                   int(bool(output_final_state)), _ptr(o), _ptr(final_state), _ptr(ws), _nbytes(ws), stream)
    if rc:
        raise KdaError("kda_gdn_chunk_fwd", rc)
    return o, final_state


def chunk_gdn_bwd(q, k, v, gate, beta, initial_state, do, dht=None, *, cu_seqlens=None,
                  use_gate_in_kernel: bool = False, A_log: Optional[torch.Tensor] = None,
                  dt_bias: Optional[torch.Tensor] = None, qk_l2norm: bool = False,
                  workspace: Optional[torch.Tensor] = None):
    """Backward of chunk_gdn (kda_gdn_chunk_bwd): inputs as there, do like v and
    dht like the states or None. Returns a dict: dq, dk, dv, dbeta like their
    tensors, dg like `gate` (the gradient of what `gate` holds: g, or the raw
    x), dA_log and ddt_bias where those parameters are given (else None), and
    dh0 where initial_state is (else None). A `workspace` passed in must hold
    chunk_gdn_workspace_bytes(..., backward=True)."""
    if not isinstance(do, torch.Tensor):
        raise TypeError("do must be a torch.Tensor")
    d, g = _check_args(q, k, v, gate, beta, initial_state, cu_seqlens, use_gate_in_kernel, A_log, dt_bias, do=do,
                       dht=dht)
    dt, lib = _DT[q.dtype], _lib()
    # packed inputs get zeros in the capacity tail, which no kernel touches
    new = torch.empty_like if cu_seqlens is None else torch.zeros_like
    dq, dk, dv, dg, dbeta = new(q), new(k), new(v), new(gate), new(beta)
    dA = None if A_log is None else torch.empty_like(A_log)
    ddt = None if dt_bias is None else torch.empty_like(dt_bias)
    dh0 = None if initial_state is None else torch.empty_like(initial_state)
    ws = _workspace(workspace, lib.kda_gdn_chunk_workspace_bytes(ctypes.byref(d), dt, 1), q)
    with _OnDevice(q) as stream:
        rc = lib.kda_gdn_chunk_bwd(ctypes.byref(d), dt, _ptr(q), _ptr(k), _ptr(v), ctypes.byref(g),
                                   int(bool(qk_l2norm)), _ptr(beta), _ptr(initial_state), _ptr(cu_seqlens),
                                   _ptr(do), _ptr(dht), _ptr(dq), _ptr(dk), _ptr(dv), _ptr(dg), _ptr(dbeta),
                                   _ptr(dh0), _ptr(dA), _ptr(ddt), _ptr(ws), _nbytes(ws), stream)
    if rc:
        raise KdaError("kda_gdn_chunk_bwd", rc)
    return dict(dq=dq, dk=dk, dv=dv, dg=dg, dbeta=dbeta, dA_log=dA, ddt_bias=ddt, dh0=dh0)


def recurrent_gdn(q, k, v, gate, beta, initial_state=None, *, cu_seqlens=None, output_final_state: bool = False,
                  use_gate_in_kernel: bool = False, A_log: Optional[torch.Tensor] = None,
                  dt_bias: Optional[torch.Tensor] = None, qk_l2norm: bool = False,
                  o: Optional[torch.Tensor] = None,
                  final_state: Optional[torch.Tensor] = None) -> Tuple[torch.Tensor, Optional[torch.Tensor]]:
    """Token-sequential forward (kda_gdn_recurrent_fwd), FP32 compute: decode
    and short sequences. Arguments as chunk_gdn; pass final_state=initial_state
    to update the states in place. Inference only: inputs that require grad are
    rejected (use chunk_gdn for training)."""
    for t in (q, k, v, gate, beta, initial_state, A_log, dt_bias):
        if isinstance(t, torch.Tensor) and t.requires_grad:
            raise RuntimeError("recurrent_gdn is inference-only; inputs require grad (use chunk_gdn)")
    d, g = _check_args(q, k, v, gate, beta, initial_state, cu_seqlens, use_gate_in_kernel, A_log, dt_bias, o,
                       final_state)
    if o is None:
        o = torch.empty_like(v)
    if not output_final_state:
        final_state = None
    elif final_state is None:
        final_state = torch.empty((d.N, d.HV, d.K, d.V), device=q.device, dtype=torch.float32)
    with _OnDevice(q) as stream:
        rc = _lib().kda_gdn_recurrent_fwd(ctypes.byref(d), _DT[q.dtype], _ptr(q), _ptr(k), _ptr(v),
                                          ctypes.byref(g), int(bool(qk_l2norm)), _ptr(beta), _ptr(initial_state),
                                          _ptr(cu_seqlens), int(bool(output_final_state)), _ptr(o),
                                          _ptr(final_state), stream)
    if rc:
        raise KdaError("kda_gdn_recurrent_fwd", rc)
    return o, final_state
