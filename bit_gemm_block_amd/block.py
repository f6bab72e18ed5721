"""Operators that stand beside the W4A4 linear layer in a transformer block.

Binding of include/w4a4_block.h (in libw4a4.so): argument marshalling only, on
the current HIP stream of the tensors' device.

* adapter_add: low-rank adapters of many requests beside a shared projection;
* norm_residual: norms before and after a block, its gate and residual scale;
* gated_activation: act(gate) * up between two projections.

Activations are matrices with contiguous rows (any row distance: column slices
are taken as they are); weights, norm parameters and workspaces are contiguous.
Outputs that the caller does not pass are allocated with torch.
"""
from __future__ import annotations

import ctypes
import os
import re
from typing import List, Optional, Tuple

import torch

from . import w4a4 as _w

HEADER = os.path.join(os.path.dirname(_w.PKG), "include", "w4a4_block.h")

_NORMS = {"none": 0, "rms": 1, "layer": 2}
_ACTS = {"silu": 0, "gelu": 1, "gelu_tanh": 2, "relu": 3}
_DT = {torch.float32: _w.F32, torch.float16: _w.F16}

_P, _I64, _INT, _F = ctypes.c_void_p, ctypes.c_int64, ctypes.c_int, ctypes.c_float
_SIGS = {
    "w4a4_adapter_workspace_size": (ctypes.c_size_t, [_I64, _I64, _I64]),
    "w4a4_adapter_add": (_INT, [_P, _INT, _I64, _P, _P, _I64, _I64, _P, _P, _P, _I64, _I64, _I64,
                                _P, _I64, _P, _I64, _P, ctypes.c_size_t, _P]),
    "w4a4_norm_residual": (_INT, [_P, _INT, _I64, _P, _INT, _I64, _INT, _P, _P, _P, _INT, _I64,
                                  _I64, _F, _INT, _P, _P, _INT, _F, _F, _I64, _I64, _P, _I64, _P,
                                  _INT, _I64, _P]),
    "w4a4_gated_activation": (_INT, [_P, _I64, _P, _I64, _INT, _INT, _I64, _I64, _P, _I64, _INT,
                                     _P]),
}
_lib: Optional[ctypes.CDLL] = None


def lib() -> ctypes.CDLL:
    """The loaded C library (raises if it has not been built)."""
    global _lib
    if _lib is None:
        l = _w.lib()
        for name, (res, args) in _SIGS.items():
            f = getattr(l, name)
            f.restype = res
            f.argtypes = args
        _lib = l
    return _lib


def header_functions() -> List[str]:
    """Names of the functions include/w4a4_block.h declares."""
    with open(HEADER) as f:
        return sorted(set(re.findall(r"^\s*(?:int|size_t)\s+(w4a4_\w+)\s*\(", f.read(), re.M)))


def _dt(t: torch.Tensor) -> int:
    d = _DT.get(t.dtype)
    if d is None:
        raise TypeError(f"unsupported dtype {t.dtype}")
    return d


def _rows(t: torch.Tensor, name: str, device, M: int, C: int) -> int:
    """The row distance of a device matrix [M, C] with contiguous rows."""
    if t.device != device or device.type != "cuda":
        raise ValueError(f"{name} must be a device tensor, on the device of the others")
    if t.dim() != 2 or t.shape[0] != M or t.shape[1] != C:
        raise ValueError(f"{name} must be [{M}, {C}], not {list(t.shape)}")
    s0, s1 = t.stride()
    if C > 1 and s1 != 1:
        raise ValueError(f"{name} must have contiguous rows")
    if M <= 1 or C == 0:
        return max(s0, C)
    if s0 < C:
        raise ValueError(f"{name} must have rows that do not overlap")
    return s0


def _whole(t: torch.Tensor, name: str, device, dtype, shape) -> int:
    """The address of a contiguous device tensor of this dtype and shape."""
    if t.device != device:
        raise ValueError(f"{name} must be on the device of the others")
    if t.dtype != dtype:
        raise TypeError(f"{name} must be {dtype}, not {t.dtype}")
    if tuple(t.shape) != shape:
        raise ValueError(f"{name} must be {list(shape)}, not {list(t.shape)}")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    return t.data_ptr()


def _call(fn: str, device, *args) -> None:
    if device.index != torch.cuda.current_device():
        with torch.cuda.device(device):
            return _call(fn, device, *args)
    status = getattr(_lib or lib(), fn)(*args, torch.cuda.current_stream(device).cuda_stream)
    if status != _w.OK:
        raise _w.W4A4Error(fn[5:], status)


# ---- low-rank adapters of many requests ---------------------------------------
def adapter_workspace_size(M: int, K: int, rank: int) -> int:
    return int(lib().w4a4_adapter_workspace_size(M, K, rank))


def adapter_workspace(M: int, K: int, rank: int, device) -> torch.Tensor:
    """A workspace for adapter_add calls of these sizes (contents unspecified)."""
    return torch.empty((max(adapter_workspace_size(M, K, rank), 1),), dtype=torch.uint8,
                       device=device)


def adapter_add(y: Optional[torch.Tensor], x: torch.Tensor, At: torch.Tensor, Bt: torch.Tensor,
                index: torch.Tensor, ranks: Optional[torch.Tensor] = None,
                scales: Optional[torch.Tensor] = None, out: Optional[torch.Tensor] = None,
                workspace: Optional[torch.Tensor] = None) -> torch.Tensor:
    """out[m] = y[m] + scales[a] (x[m] . At[a]^T) . Bt[a]^T with a = index[m];
    rows whose index is outside [0, adapters) get y[m].

    x [M, K] and the stacked transposed factors At [adapters, rank, K],
    Bt [adapters, N, rank] in fp16 or fp32; y (or None: zero) and out [M, N]
    float32, out may be y; index [M], ranks [adapters] (the columns in use)
    int32, scales [adapters] float32."""
    dev = x.device
    L, R, K = At.shape
    M = x.shape[0]
    N = Bt.shape[1]
    ldx = _rows(x, "x", dev, M, K)
    at = _whole(At, "At", dev, x.dtype, (L, R, K))
    bt = _whole(Bt, "Bt", dev, x.dtype, (L, N, R))
    ix = _whole(index, "index", dev, torch.int32, (M,))
    rk = None if ranks is None else _whole(ranks, "ranks", dev, torch.int32, (L,))
    sc = None if scales is None else _whole(scales, "scales", dev, torch.float32, (L,))
    if out is None:
        out = torch.empty((M, N), dtype=torch.float32, device=dev)
    for t, name in ((y, "y"), (out, "out")):
        if t is not None and t.dtype != torch.float32:
            raise TypeError(f"{name} must be float32, not {t.dtype}")
    ldo = _rows(out, "out", dev, M, N)
    ldy = N if y is None else _rows(y, "y", dev, M, N)
    if workspace is None:
        workspace = adapter_workspace(M, K, R, dev)
    elif workspace.device != dev or not workspace.is_contiguous():
        raise ValueError("workspace must be contiguous, on the device of the others")
    _call("w4a4_adapter_add", dev, x.data_ptr(), _dt(x), ldx, at, bt, L, R, ix, rk, sc, M, N, K,
          None if y is None else y.data_ptr(), ldy, out.data_ptr(), ldo, workspace.data_ptr(),
          workspace.numel() * workspace.element_size())
    return out


# ---- norms before and after a block ---------------------------------------------
def norm_residual(h: Optional[torch.Tensor], y: Optional[torch.Tensor] = None, *,
                  post_norm: str = "none", post_weight: Optional[torch.Tensor] = None,
                  post_bias: Optional[torch.Tensor] = None, gate: Optional[torch.Tensor] = None,
                  gate_rows: int = 1, residual_scale: float = 1.0, pre_norm: str = "none",
                  pre_weight: Optional[torch.Tensor] = None,
                  pre_bias: Optional[torch.Tensor] = None, weight_offset: float = 0.0,
                  eps: float = 1e-6, x_dtype: Optional[torch.dtype] = torch.float16,
                  h_out: Optional[torch.Tensor] = None, x_out: Optional[torch.Tensor] = None,
                  want_h: Optional[bool] = None) -> Tuple[Optional[torch.Tensor], Optional[torch.Tensor]]:
    """(h', x): h' = h + residual_scale * gate * norm_post(y), x = norm_pre(h').

    h (the residual stream) and y (the block's output) are [M, C], either may
    be None; gate [ceil(M / gate_rows), C], row g for rows [g gate_rows,
    (g + 1) gate_rows); weights and biases [C] in one dtype.  Norms are "none",
    "rms" or "layer", scaled by weight_offset + weight.  h' has h's dtype (y's
    without h) and is made when y is given (want_h overrides); x has x_dtype
    (None, with pre_norm "none": no x)."""
    ref = h if h is not None else y
    if ref is None:
        raise ValueError("h or y must be given")
    dev = ref.device
    M, C = ref.shape
    if post_norm not in _NORMS or pre_norm not in _NORMS:
        raise ValueError('norms are "none", "rms" or "layer"')
    ldh = C if h is None else _rows(h, "h", dev, M, C)
    ldy = C if y is None else _rows(y, "y", dev, M, C)
    pd = None
    params = []
    for t, name in ((post_weight, "post_weight"), (post_bias, "post_bias"),
                    (pre_weight, "pre_weight"), (pre_bias, "pre_bias")):
        if t is None:
            params.append(None)
            continue
        pd = t.dtype if pd is None else pd
        params.append(_whole(t, name, dev, pd, (C,)))
    gd, ldg, gp = _w.F32, C, None
    if gate is not None:
        if gate_rows < 1:
            raise ValueError("gate_rows must be positive")
        ldg = _rows(gate, "gate", dev, -(-M // gate_rows), C)
        gd, gp = _dt(gate), gate.data_ptr()
    if h_out is None and (want_h if want_h is not None else y is not None):
        h_out = torch.empty((M, C), dtype=ref.dtype, device=dev)
    if h_out is not None and h_out.dtype != ref.dtype:
        raise TypeError("h_out must have h's dtype (y's without h)")
    if x_out is None and x_dtype is not None:
        x_out = torch.empty((M, C), dtype=x_dtype, device=dev)
    _call("w4a4_norm_residual", dev,
          None if h is None else h.data_ptr(), _dt(ref), ldh,
          None if y is None else y.data_ptr(), _w.F32 if y is None else _dt(y), ldy,
          _NORMS[post_norm], params[0], params[1], gp, gd, ldg, gate_rows, residual_scale,
          _NORMS[pre_norm], params[2], params[3], _w.F32 if pd is None else _DT.get(pd, -1),
          weight_offset, eps, M, C,
          None if h_out is None else h_out.data_ptr(),
          C if h_out is None else _rows(h_out, "h_out", dev, M, C),
          None if x_out is None else x_out.data_ptr(),
          _w.F32 if x_out is None else _dt(x_out),
          C if x_out is None else _rows(x_out, "x_out", dev, M, C))
    return h_out, x_out


# ---- gated activation -------------------------------------------------------------
def gated_activation(gate: torch.Tensor, up: Optional[torch.Tensor], act: str = "silu",
                     out_dtype: torch.dtype = torch.float16,
                     out: Optional[torch.Tensor] = None) -> torch.Tensor:
    """act(gate) * up (up None: act(gate)) of [M, F] matrices in fp16 or fp32,
    for instance the two halves of a projection y: y[:, :F], y[:, F:].  act is
    "silu", "gelu", "gelu_tanh" or "relu"."""
    a = _ACTS.get(act)
    if a is None:
        raise ValueError(f"act must be one of {sorted(_ACTS)}")
    dev = gate.device
    M, F = gate.shape
    ldg = _rows(gate, "gate", dev, M, F)
    ldu = F
    if up is not None:
        ldu = _rows(up, "up", dev, M, F)
        if up.dtype != gate.dtype:
            raise TypeError("gate and up must have one dtype")
    if out is None:
        out = torch.empty((M, F), dtype=out_dtype, device=dev)
    _call("w4a4_gated_activation", dev, gate.data_ptr(), ldg,
          None if up is None else up.data_ptr(), ldu, _dt(gate), a, M, F, out.data_ptr(),
          _rows(out, "out", dev, M, F), _dt(out))
    return out
