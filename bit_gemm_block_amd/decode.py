"""Operators of a decoding step beside the W4A4 linear layer.

Binding of include/w4a4_decode.h (in libw4a4.so): argument marshalling only, on
the current HIP stream of the tensors' device.

* qlinear_w4a16: a projection of a few rows by 4-bit weights, the activations
  not quantized (the same stored weights as the layer's);
* KVCache, cache_write, cache_read: keys and values in pages, quantized to 4 or
  8 bits as they are written, and read back;
* cache_attention: attention of a batch over that cache, in which a prefix that
  all sequences share is computed once for all.

Activations are matrices with contiguous rows (any row distance: column slices
are taken as they are), all heads of a token side by side; index arrays are
contiguous int32 device tensors, so that a captured call follows their values.
Outputs that the caller does not pass are allocated with torch.  Tensors of a
wrong shape or device raise ValueError, of a wrong dtype TypeError, and what the
library refuses raises W4A4Error with its status, before anything is enqueued.
"""
from __future__ import annotations

import ctypes
import os
import re
from dataclasses import dataclass
from typing import List, Optional, Tuple

import torch

from . import block as _b
from . import w4a4 as _w

HEADER = os.path.join(os.path.dirname(_w.PKG), "include", "w4a4_decode.h")

_LAYOUTS = {"rowmajor": _w.WEIGHTS_ROWMAJOR, "tiled": _w.WEIGHTS_TILED}


class CacheStruct(ctypes.Structure):
    """w4a4_cache of the header."""
    _fields_ = [("k", ctypes.c_void_p), ("v", ctypes.c_void_p), ("k_scale", ctypes.c_void_p),
                ("v_scale", ctypes.c_void_p), ("pages", ctypes.c_int64), ("heads", ctypes.c_int64),
                ("page_size", ctypes.c_int64), ("head_dim", ctypes.c_int64), ("bits", ctypes.c_int)]


_P, _I64, _INT, _F, _SZ = ctypes.c_void_p, ctypes.c_int64, ctypes.c_int, ctypes.c_float, ctypes.c_size_t
_C = ctypes.POINTER(CacheStruct)
_SIGS = {
    "w4a16_qlinear_workspace_size": (_SZ, [_I64, _I64, _I64]),
    "w4a16_qlinear_forward": (_INT, [_P, _INT, _I64, _P, _INT, _P, _INT, _I64, _I64, _I64, _I64, _P, _INT, _I64, _P,
                                     _SZ, _P]),
    "w4a4_cache_write": (_INT, [_C, _P, _I64, _P, _I64, _INT, _P, _I64, _P]),
    "w4a4_cache_read": (_INT, [_C, _P, _I64, _P, _I64, _P, _I64, _INT, _P]),
    "w4a4_cache_attention_workspace_size": (_SZ, [_C, _I64, _I64, _I64, _I64, _I64, _I64]),
    "w4a4_cache_attention": (_INT, [_C, _P, _INT, _I64, _I64, _I64, _P, _I64, _I64, _P, _P, _I64, _INT, _P, _I64, _P,
                                    _F, _P, _INT, _I64, _P, _SZ, _P]),
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
    """Names of the functions include/w4a4_decode.h declares."""
    with open(HEADER) as f:
        return sorted(set(re.findall(r"^\s*(?:int|size_t)\s+(w4a\d+_\w+)\s*\(", f.read(), re.M)))


# ---- projections with unquantized activations -----------------------------------
def qlinear_w4a16_workspace_size(M: int, N: int, K: int) -> int:
    return int(lib().w4a16_qlinear_workspace_size(M, N, K))


def qlinear_w4a16_workspace(M: int, N: int, K: int, device) -> torch.Tensor:
    """A workspace for qlinear_w4a16 calls of up to M rows (contents unspecified)."""
    return torch.empty((max(qlinear_w4a16_workspace_size(M, N, K), 1),), dtype=torch.uint8, device=device)


def qlinear_w4a16(x: torch.Tensor, wq: torch.Tensor, w_scale: torch.Tensor, w_group: int = 0,
                  w_layout: str = "tiled", out_dtype: torch.dtype = torch.float32,
                  out: Optional[torch.Tensor] = None, workspace: Optional[torch.Tensor] = None) -> torch.Tensor:
    """y[m, n] = sum_j w_scale[n, j] sum_{k in group j} x[m, k] q[n, k].

    x [M, K] fp16 or fp32, meant for few rows; codes wq and scales w_scale ([N],
    or [N, K / w_group]) as w4a4.quantize_weight_int4 makes them in layout
    "rowmajor" or "tiled".  Weights prepared with a Hadamard block take rotated
    activations (w4a4.hadamard_rotate)."""
    layout = _LAYOUTS.get(w_layout)
    if layout is None:
        raise ValueError(f"w_layout must be one of {sorted(_LAYOUTS)}")
    return (_b._binding or _b.binding()).qlinear_w4a16(x, wq, w_scale, w_group, layout, out_dtype, out, workspace)


# ---- the quantized cache ------------------------------------------------------------
@dataclass
class KVCache:
    """Keys and values in pages: codes k, v uint8 [pages, heads, page_size,
    head_dim * bits / 8] and scales k_scale, v_scale float32 [pages, heads,
    page_size].  A token's slot is page * page_size + its offset in the page."""
    k: torch.Tensor
    v: torch.Tensor
    k_scale: torch.Tensor
    v_scale: torch.Tensor
    bits: int = 4

    @classmethod
    def empty(cls, pages: int, heads: int, page_size: int, head_dim: int, bits: int = 4, device="cuda") -> "KVCache":
        """A cache with unspecified contents (bits 4 or 8; head_dim 64, 128 or
        256; page_size a power of two from 16)."""
        if bits not in (4, 8):
            raise ValueError("bits must be 4 or 8")
        codes = lambda: torch.empty((pages, heads, page_size, head_dim * bits // 8), dtype=torch.uint8,  # noqa: E731
                                    device=device)
        scales = lambda: torch.empty((pages, heads, page_size), dtype=torch.float32, device=device)  # noqa: E731
        return cls(codes(), codes(), scales(), scales(), bits)

    @property
    def head_dim(self) -> int:
        return self.k.shape[3] * 8 // self.bits

    def struct(self) -> CacheStruct:
        pages, heads, page_size, _ = self.k.shape
        return CacheStruct(self.k.data_ptr(), self.v.data_ptr(), self.k_scale.data_ptr(), self.v_scale.data_ptr(),
                           pages, heads, page_size, self.head_dim, self.bits)


def cache_write(cache: KVCache, k: torch.Tensor, v: torch.Tensor, slots: torch.Tensor) -> None:
    """Quantizes k and v ([T, heads * head_dim], fp16 or fp32) into the tokens'
    slots (int32 [T]; a slot outside the cache: not written; each at most once
    in a call), one scale per token and head."""
    (_b._binding or _b.binding()).cache_write(cache.k, cache.v, cache.k_scale, cache.v_scale, cache.bits, k, v, slots)


def cache_read(cache: KVCache, slots: torch.Tensor, out_dtype: torch.dtype = torch.float16,
               k: Optional[torch.Tensor] = None, v: Optional[torch.Tensor] = None, want_k: bool = True,
               want_v: bool = True) -> Tuple[Optional[torch.Tensor], Optional[torch.Tensor]]:
    """(k, v) [T, heads * head_dim]: the values in slots (int32 [T]); zeros
    where a slot is outside the cache."""
    return (_b._binding or _b.binding()).cache_read(cache.k, cache.v, cache.k_scale, cache.v_scale, cache.bits, slots,
                                                    out_dtype, k, v, want_k, want_v)


# ---- attention over the cache ----------------------------------------------------------
def cache_attention_workspace_size(cache: KVCache, tokens: int, q_heads: int, seqs: int, table_width: int,
                                   max_q: int = 1, prefix_width: int = 0) -> int:
    return int(lib().w4a4_cache_attention_workspace_size(ctypes.byref(cache.struct()), tokens, q_heads, seqs,
                                                         table_width, max_q, prefix_width))


def cache_attention_workspace(cache: KVCache, tokens: int, q_heads: int, seqs: int, table_width: int, max_q: int = 1,
                              prefix_width: int = 0) -> torch.Tensor:
    """A workspace for cache_attention calls of these sizes (contents unspecified).
    Smaller sizes may need a larger one."""
    n = cache_attention_workspace_size(cache, tokens, q_heads, seqs, table_width, max_q, prefix_width)
    return torch.empty((max(n, 1),), dtype=torch.uint8, device=cache.k.device)


def cache_attention(q: torch.Tensor, cache: KVCache, tables: torch.Tensor, lengths: torch.Tensor, *,
                    q_start: Optional[torch.Tensor] = None, max_q: int = 1, causal: bool = True,
                    prefix_table: Optional[torch.Tensor] = None, prefix_length: Optional[torch.Tensor] = None,
                    scale: Optional[float] = None, out_dtype: torch.dtype = torch.float16,
                    out: Optional[torch.Tensor] = None, workspace: Optional[torch.Tensor] = None) -> torch.Tensor:
    """softmax(scale q k^T) v of a batch over the cache, [tokens, q_heads * head_dim].

    q [tokens, q_heads * head_dim] fp16 or fp32; query head h reads cache head
    h / (q_heads / heads).  Sequence s has lengths[s] tokens, in the pages
    tables[s] (int32 [S, pages]); a page outside the cache holds nothing.  Its
    queries are rows [q_start[s], q_start[s + 1]) of q, at most max_q, the last
    of which is its last token (causal: a query sees up to its own position);
    without q_start row s is sequence s.  Rows of no sequence are left as they
    are.  prefix_table (int32 [pages]) and prefix_length (int32 [1]): tokens in
    front of every sequence, which all its queries see.  scale None:
    head_dim ** -0.5."""
    return (_b._binding or _b.binding()).cache_attention(
        q, cache.k, cache.v, cache.k_scale, cache.v_scale, cache.bits, tables, lengths, q_start, max_q, causal,
        prefix_table, prefix_length, scale, out_dtype, out, workspace)
