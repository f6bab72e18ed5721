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
import functools
import os
import re
import struct
from typing import List, Optional, Tuple

import torch

from . import w4a4 as _w

HEADER = os.path.join(os.path.dirname(_w.PKG), "include", "w4a4_block.h")

_NORMS = {"none": 0, "rms": 1, "layer": 2}
_ACTS = {"silu": 0, "gelu": 1, "gelu_tanh": 2, "relu": 3}
_PARAMS = ("post_weight", "post_bias", "pre_weight", "pre_bias")
_DT = {torch.float32: _w.F32, torch.float16: _w.F16}

# The raw handle of a device's current stream (torch's own accessor where there
# is one: the Stream object costs another microsecond).
_stream = getattr(torch._C, "_cuda_getCurrentRawStream",
                  lambda d: torch.cuda.current_stream(d).cuda_stream)
_current_device = torch.cuda.current_device

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
            if res is _INT:
                f = getattr(l, name + "_packed")
                f.restype, f.argtypes = _INT, [ctypes.c_char_p]
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


def _rows(t: torch.Tensor, name: str, dev: int, shape) -> int:
    """The row distance of a device matrix of this shape with contiguous rows."""
    if t.shape != shape:
        raise ValueError(f"{name} must be {list(shape)}, not {list(t.shape)}")
    s0, s1 = t.stride()
    M, C = shape
    if t.get_device() != dev or dev < 0:
        raise ValueError(f"{name} must be a device tensor, on the device of the others")
    if s1 == 1 and s0 >= C:
        return s0
    if C > 1 and s1 != 1:
        raise ValueError(f"{name} must have contiguous rows")
    if M > 1 and C > 0 and s0 < C:
        raise ValueError(f"{name} must have rows that do not overlap")
    return s0 if s0 >= C else C


def _whole(t: torch.Tensor, name: str, dev: int, dtype, shape) -> int:
    """The address of a contiguous device tensor of this dtype and shape."""
    if t.get_device() != dev:
        raise ValueError(f"{name} must be on the device of the others")
    if t.dtype is not dtype:
        raise TypeError(f"{name} must be {dtype}, not {t.dtype}")
    if t.shape != shape:
        raise ValueError(f"{name} must be {list(shape)}, not {list(t.shape)}")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    return t.data_ptr()


class _Entry:
    """An entry point of the library, called on a device's current stream with
    its arguments packed in one buffer: a quarter of the host time of
    converting them one by one."""

    def __init__(self, name: str, form: str):
        self.name, self.pack, self.f = name, struct.Struct(form).pack, None

    def __call__(self, dev: int, *args) -> None:
        if self.f is None:
            self.f = getattr(lib(), f"w4a4_{self.name}_packed")
        if dev == _current_device():
            status = self.f(self.pack(*args, _stream(dev)))
        else:
            with torch.cuda.device(dev):
                status = self.f(self.pack(*args, _stream(dev)))
        if status:
            raise _w.W4A4Error(self.name, status)


_adapter_add = _Entry("adapter_add", "=20q")
_norm_residual = _Entry("norm_residual", "=13qd4q2d8q")
_gated_activation = _Entry("gated_activation", "=12q")


# ---- low-rank adapters of many requests ---------------------------------------
@functools.lru_cache(maxsize=1024)
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
    dev = x.get_device()
    L, R, K = At.shape
    M = x.shape[0]
    N = Bt.shape[1]
    dt = x.dtype
    ldx = _rows(x, "x", dev, (M, K))
    at = _whole(At, "At", dev, dt, (L, R, K))
    bt = _whole(Bt, "Bt", dev, dt, (L, N, R))
    ix = _whole(index, "index", dev, torch.int32, (M,))
    rk = 0 if ranks is None else _whole(ranks, "ranks", dev, torch.int32, (L,))
    sc = 0 if scales is None else _whole(scales, "scales", dev, torch.float32, (L,))
    yp, ldy = 0, N
    if y is not None:
        if y.dtype is not torch.float32:
            raise TypeError(f"y must be float32, not {y.dtype}")
        yp, ldy = y.data_ptr(), _rows(y, "y", dev, (M, N))
    ldo = N
    if out is None:
        out = x.new_empty((M, N), dtype=torch.float32) if ldy != N or y is None else torch.empty_like(y)
    else:
        if out.dtype is not torch.float32:
            raise TypeError(f"out must be float32, not {out.dtype}")
        ldo = _rows(out, "out", dev, (M, N))
    if workspace is None:
        workspace = index.new_empty((adapter_workspace_size(M, K, R) + 3) // 4)
    elif workspace.get_device() != dev or not workspace.is_contiguous():
        raise ValueError("workspace must be contiguous, on the device of the others")
    _adapter_add(dev, x.data_ptr(), _dt(x), ldx, at, bt, L, R, ix, rk, sc, M, N, K, yp, ldy,
                 out.data_ptr(), ldo, workspace.data_ptr(), workspace.nbytes)
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
    dev, dt = ref.get_device(), ref.dtype
    shape = M, C = ref.shape
    post, pre = _NORMS.get(post_norm), _NORMS.get(pre_norm)
    if post is None or pre is None:
        raise ValueError('norms are "none", "rms" or "layer"')
    hp, hd, ldh = 0, _dt(ref), C
    if h is not None:
        hp, ldh = h.data_ptr(), _rows(h, "h", dev, shape)
    yp, yd, ldy = 0, _w.F32, C
    if y is not None:
        yp, yd, ldy = y.data_ptr(), _dt(y), _rows(y, "y", dev, shape)
    pdt, p = None, [0, 0, 0, 0]
    for i, t in enumerate((post_weight, post_bias, pre_weight, pre_bias)):
        if t is not None:
            pdt = pdt or t.dtype
            p[i] = _whole(t, _PARAMS[i], dev, pdt, (C,))
    gp, gd, ldg = 0, _w.F32, C
    if gate is not None:
        if gate_rows < 1:
            raise ValueError("gate_rows must be positive")
        gp, gd, ldg = gate.data_ptr(), _dt(gate), _rows(gate, "gate", dev, (-(-M // gate_rows), C))
    op, ldho = 0, C
    if h_out is not None:
        if h_out.dtype is not dt:
            raise TypeError("h_out must have h's dtype (y's without h)")
        op, ldho = h_out.data_ptr(), _rows(h_out, "h_out", dev, shape)
    elif want_h or (want_h is None and y is not None):
        h_out = ref.new_empty(shape)
        op = h_out.data_ptr()
    xp, xd, ldx = 0, _w.F32, C
    if x_out is not None:
        xp, xd, ldx = x_out.data_ptr(), _dt(x_out), _rows(x_out, "x_out", dev, shape)
    elif x_dtype is not None:
        x_out = ref.new_empty(shape, dtype=x_dtype)
        xp, xd = x_out.data_ptr(), _dt(x_out)
    _norm_residual(dev, hp, hd, ldh, yp, yd, ldy, post, p[0], p[1], gp, gd, ldg, gate_rows,
                   residual_scale, pre, p[2], p[3], _DT.get(pdt, _w.F32 if pdt is None else -1),
                   weight_offset, eps, M, C, op, ldho, xp, xd, ldx)
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
    dev = gate.get_device()
    shape = M, F = gate.shape
    ldg = _rows(gate, "gate", dev, shape)
    up_ptr, ldu = 0, F
    if up is not None:
        up_ptr, ldu = up.data_ptr(), _rows(up, "up", dev, shape)
        if up.dtype is not gate.dtype:
            raise TypeError("gate and up must have one dtype")
    ldo = F
    if out is None:
        out = gate.new_empty(shape, dtype=out_dtype)
    else:
        ldo = _rows(out, "out", dev, shape)
    _gated_activation(dev, gate.data_ptr(), ldg, up_ptr, ldu, _dt(gate), a, M, F, out.data_ptr(),
                      ldo, _dt(out))
    return out
