"""float64 references of the operators beside the layer (adapters, norms joined
with gate and residual, gated activation), straight from their formulas."""
from __future__ import annotations

import math

import numpy as np


def adapter_add(y, x, At, Bt, index, ranks=None, scales=None):
    """y [M, N] (or None), x [M, K], At [L, R, K], Bt [L, N, R], index [M]."""
    L, R, _ = At.shape
    out = np.zeros((x.shape[0], Bt.shape[1])) if y is None else y.astype(np.float64).copy()
    for m, a in enumerate(index):
        if not 0 <= a < L:
            continue
        r = R if ranks is None else min(max(int(ranks[a]), 0), R)
        if r == 0:
            continue
        t = At[a, :r].astype(np.float64) @ x[m].astype(np.float64)
        s = 1.0 if scales is None else float(scales[a])
        out[m] += s * (Bt[a][:, :r].astype(np.float64) @ t)
    return out


def adapter_add_scale(y, x, At, Bt, index, ranks=None, scales=None):
    """The sums of absolute values behind adapter_add's three roundings: of the
    products x A (carried through |B|), of t B, and of the result."""
    L, R, K = At.shape
    M, N = x.shape[0], Bt.shape[1]
    first, second = np.zeros((M, N)), np.zeros((M, N))
    for m, a in enumerate(index):
        if not 0 <= a < L:
            continue
        r = R if ranks is None else min(max(int(ranks[a]), 0), R)
        if r == 0:
            continue
        A, B = At[a, :r].astype(np.float64), np.abs(Bt[a][:, :r].astype(np.float64))
        xm = x[m].astype(np.float64)
        s = 1.0 if scales is None else abs(float(scales[a]))
        t = np.abs(A @ xm)
        first[m] = s * (B @ (np.abs(A) @ np.abs(xm)))
        second[m] = s * (B @ np.full(r, t.max()))
    return first, second


def norm(v, kind, weight=None, bias=None, offset=0.0, eps=1e-6):
    v = np.asarray(v, np.float64)
    if kind == "none":
        return v
    if kind == "layer":
        v = v - v.mean(axis=1, keepdims=True)
    v = v / np.sqrt(np.mean(v * v, axis=1, keepdims=True) + eps)
    if weight is not None:
        v = v * (offset + weight.astype(np.float64))
    if bias is not None:
        v = v + bias.astype(np.float64)
    return v


def norm_residual(h, y, post="none", post_w=None, post_b=None, gate=None, gate_rows=1, rs=1.0,
                  pre="none", pre_w=None, pre_b=None, offset=0.0, eps=1e-6):
    """(h', x)."""
    out = 0.0 if h is None else h.astype(np.float64)
    if y is not None:
        v = norm(y, post, post_w, post_b, offset, eps)
        if gate is not None:
            v = v * gate.astype(np.float64)[np.arange(y.shape[0]) // gate_rows]
        out = out + rs * v
    return out, norm(out, pre, pre_w, pre_b, offset, eps)


def activation(g, act):
    g = np.asarray(g, np.float64)
    if act == "silu":
        return g / (1.0 + np.exp(-g))
    if act == "gelu":
        return 0.5 * g * np.vectorize(math.erfc, otypes=[np.float64])(-g / math.sqrt(2.0))
    if act == "gelu_tanh":
        return g / (1.0 + np.exp(-2.0 * math.sqrt(2.0 / math.pi) * (g + 0.044715 * g ** 3)))
    return np.maximum(g, 0.0)
