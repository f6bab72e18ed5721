"""Operators that stand beside the W4A4 linear layer in a transformer block.

Binding of include/w4a4_block.h (in libw4a4.so): argument marshalling only, on
the current HIP stream of the tensors' device.

* adapter_add: low-rank adapters of many requests beside a shared projection;
* norm_residual: norms before and after a block, its gate and residual scale;
* gated_activation: act(gate) * up between two projections.

Activations are matrices with contiguous rows (any row distance: column slices
are taken as they are); weights, norm parameters and workspaces are contiguous.
Outputs that the caller does not pass are allocated with torch.  Tensors of a
wrong shape or device raise ValueError, of a wrong dtype TypeError, and what the
library refuses raises W4A4Error with its status, before anything is enqueued.

The checks and calls are compiled (_block.so, csrc/block_binding.cpp): a small
call costs 4 to 8 us of host time in place of the 7 to 13 us that it takes
through ctypes.
"""
from __future__ import annotations

import ctypes
import os
import re
from typing import List, Optional, Tuple

import torch

from . import w4a4 as _w

BINDING_PATH = os.path.join(_w.PKG, "_block.so")
HEADER = os.path.join(os.path.dirname(_w.PKG), "include", "w4a4_block.h")

_NORMS = {"none": 0, "rms": 1, "layer": 2}
_ACTS = {"silu": 0, "gelu": 1, "gelu_tanh": 2, "relu": 3}

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
_binding = None


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


def binding():
    """The compiled binding (raises if it has not been built)."""
    global _binding
    if _binding is None:
        _w.lib()
        if not os.path.exists(BINDING_PATH):
            raise RuntimeError(f"{BINDING_PATH} is missing: build it with "
                               "`python -m bit_gemm_block_amd.build`")
        from . import _block
        _block.set_error(_w.W4A4Error)
        _binding = _block
    return _binding


def header_functions() -> List[str]:
    """Names of the functions include/w4a4_block.h declares."""
    with open(HEADER) as f:
        return sorted(set(re.findall(r"^\s*(?:int|size_t)\s+(w4a4_\w+)\s*\(", f.read(), re.M)))


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
    return (_binding or binding()).adapter_add(y, x, At, Bt, index, ranks, scales, out, workspace)


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
    post, pre = _NORMS.get(post_norm), _NORMS.get(pre_norm)
    if post is None or pre is None:
        raise ValueError('norms are "none", "rms" or "layer"')
    return (_binding or binding()).norm_residual(
        h, y, post, post_weight, post_bias, gate, gate_rows, residual_scale, pre, pre_weight,
        pre_bias, weight_offset, eps, x_dtype, h_out, x_out,
        y is not None if want_h is None else want_h)


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
    return (_binding or binding()).gated_activation(gate, up, a, out_dtype, out)
