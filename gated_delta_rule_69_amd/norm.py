"""Output norm of a linear-attention layer: binding of kda_norm_fwd and
kda_norm_bwd (csrc/kda_norm.hip). Argument marshalling only.

    n = (x - mu) / sqrt(mean((x - mu)^2) + eps)      (mu = 0 for kind "rms")
    y = (n weight + bias) act(gate)                  (no factor without a gate)

over the last dimension of x.
"""
from __future__ import annotations

import ctypes
from typing import Optional

import torch

from . import KdaError, _cu_dims, _lib, _nbytes
from .gdn import _DT, _OnDevice, _ptr, _want, _workspace

_KINDS = {"rms": 0, "layer": 1}
_ACTS = {"silu": 0, "sigmoid": 1}


class KdaNorm(ctypes.Structure):
    """kda_norm: parameters of the output norm."""
    _fields_ = [("weight", ctypes.c_void_p), ("bias", ctypes.c_void_p), ("param_dtype", ctypes.c_int32),
                ("D", ctypes.c_int32), ("kind", ctypes.c_int32), ("activation", ctypes.c_int32),
                ("eps", ctypes.c_float)]


def _check_args(x, weight, bias, gate, kind, activation, eps, cu_seqlens, **like_x):
    """Checks everything the C ABI cannot see; returns (kda_norm, rows, N, rows per token)."""
    if not isinstance(x, torch.Tensor):
        raise TypeError("x must be a torch.Tensor")
    if x.dtype not in _DT:
        raise TypeError(f"x must be bfloat16 or float32, got {x.dtype}")
    if x.dim() < 1 or x.shape[-1] < 1:
        raise ValueError("x must be [..., D] with D >= 1")
    if kind not in _KINDS:
        raise ValueError(f"kind must be one of {sorted(_KINDS)}, got {kind!r}")
    if activation not in _ACTS:
        raise ValueError(f"activation must be one of {sorted(_ACTS)}, got {activation!r}")
    D, dev = x.shape[-1], x.device
    pdt = torch.float32
    for t, n in ((weight, "weight"), (bias, "bias")):
        if t is not None:
            if not isinstance(t, torch.Tensor):
                raise TypeError(f"{n} must be a torch.Tensor")
            if t.dtype not in (torch.float32, x.dtype):
                raise TypeError(f"{n} must be float32 or {x.dtype}, got {t.dtype}")
            pdt = t.dtype
    _want(x, "x", x.shape, x.dtype, dev)
    _want(weight, "weight", (D,), pdt, dev)
    _want(bias, "bias", (D,), pdt, dev)
    _want(gate, "gate", x.shape, x.dtype, dev)
    for n, t in like_x.items():
        _want(t, n, x.shape, x.dtype, dev)
    rows, N, rpt = x.numel() // D, 0, 1
    if cu_seqlens is not None:
        if x.dim() < 3:
            raise ValueError("with cu_seqlens x is a packed batch [1, T, ..., D]")
        N = _cu_dims(cu_seqlens, x.shape[0])
        _want(cu_seqlens, "cu_seqlens", (N + 1,), torch.int32, dev)
        for s in x.shape[2:-1]:
            rpt *= s
        if rpt < 1:
            raise ValueError("a packed batch needs at least one row per token")
    if not x.is_cuda:
        raise ValueError("x must be a device tensor")
    p = KdaNorm(None if weight is None else weight.data_ptr(), None if bias is None else bias.data_ptr(), _DT[pdt],
                D, _KINDS[kind], _ACTS[activation], float(eps))
    return p, rows, N, rpt


def gated_norm(x, weight=None, bias=None, gate=None, *, kind: str = "rms", activation: str = "silu",
               eps: float = 1e-5, cu_seqlens=None, out: Optional[torch.Tensor] = None) -> torch.Tensor:
    """y = (n(x) weight + bias) act(gate) over the last dimension (1 .. 8192) of
    x (kda_norm_fwd). kind "rms" or "layer"; weight and bias [D] in float32 or
    x's dtype, both optional; gate like x or None (then no factor), activation
    "silu" or "sigmoid". With cu_seqlens x is a packed batch [1, T, ..., D] (a
    scan's output): rows behind the last sequence are neither read nor written.
    `out` may be x or gate."""
    p, rows, N, rpt = _check_args(x, weight, bias, gate, kind, activation, eps, cu_seqlens, out=out)
    if out is None:
        out = torch.empty_like(x)
    with _OnDevice(x) as stream:
        rc = _lib().kda_norm_fwd(_DT[x.dtype], rows, ctypes.byref(p), _ptr(cu_seqlens), N, rpt, _ptr(x), _ptr(gate),
                                 _ptr(out), stream)
    if rc:
        raise KdaError("kda_norm_fwd", rc)
    return out


def gated_norm_bwd(x, dy, weight=None, bias=None, gate=None, *, kind: str = "rms", activation: str = "silu",
                   eps: float = 1e-5, cu_seqlens=None, workspace: Optional[torch.Tensor] = None):
    """Gradients of gated_norm (kda_norm_bwd) from dy like x: a dict with dx and
    dgate (None without a gate) like x, dweight and dbias like their parameters
    (None where absent). With cu_seqlens the rows behind the last sequence add
    nothing to dweight and dbias, and their dx and dgate are zero."""
    if not isinstance(dy, torch.Tensor):
        raise TypeError("dy must be a torch.Tensor")
    p, rows, N, rpt = _check_args(x, weight, bias, gate, kind, activation, eps, cu_seqlens, dy=dy)
    new = torch.empty_like if cu_seqlens is None else torch.zeros_like
    dx, dz = new(x), None if gate is None else new(gate)
    dw = None if weight is None else torch.empty_like(weight)
    db = None if bias is None else torch.empty_like(bias)
    ws = None
    if dw is not None or db is not None:
        ws = _workspace(workspace, int(_lib().kda_norm_bwd_workspace_bytes(ctypes.byref(p))), x)
    with _OnDevice(x) as stream:
        rc = _lib().kda_norm_bwd(_DT[x.dtype], rows, ctypes.byref(p), _ptr(cu_seqlens), N, rpt, _ptr(x), _ptr(gate),
                                 _ptr(dy), _ptr(dx), _ptr(dz), _ptr(dw), _ptr(db), _ptr(ws), _nbytes(ws), stream)
    if rc:
        raise KdaError("kda_norm_bwd", rc)
    return dict(dx=dx, dweight=dw, dbias=db, dgate=dz)
