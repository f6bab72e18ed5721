"""float64 references of the operators of a decoding step (products with 4-bit
weights, the quantized cache, attention over it), straight from their formulas."""
from __future__ import annotations

import numpy as np


def unpack(codes, bits):
    """Bytes to signed codes: nibbles, the even element low, or int8."""
    codes = np.ascontiguousarray(codes)
    if bits == 8:
        return codes.view(np.int8).astype(np.int64)
    lo, hi = codes & 15, codes >> 4
    q = np.stack((lo, hi), axis=-1).reshape(codes.shape[:-1] + (2 * codes.shape[-1],)).astype(np.int64)
    return np.where(q > 7, q - 16, q)


def pack(q, bits):
    if bits == 8:
        return q.astype(np.int8).view(np.uint8)
    q = (q.astype(np.int64) & 15).astype(np.uint8)
    return q[..., 0::2] | (q[..., 1::2] << 4)


def tile(wq):
    """Row-major packed weights [N, K / 2] to tiles of 16 rows and 128 channels."""
    N, B = wq.shape
    t = np.concatenate((wq, np.zeros((-N % 16, B), np.uint8))).reshape(-1, 16, B // 64, 4, 16)
    return np.ascontiguousarray(t.transpose(0, 2, 3, 1, 4)).reshape(-1, B)


def qlinear_w4a16(x, wq, w_scale, group):
    """(y, sum of absolute products): x [M, K], row-major codes, scales."""
    q = unpack(wq, 4).astype(np.float64)
    s = w_scale.astype(np.float64).reshape(q.shape[0], -1)
    w = q * np.repeat(s, group or q.shape[1], axis=1)
    x = x.astype(np.float64)
    return x @ w.T, np.abs(x) @ np.abs(w).T


def quantize(x, bits):
    """(codes, scales) of rows: s = max|x| / qmax and x / s rounded to float32, as
    the definition says (a float64 quotient of float32 values, rounded again, is
    their float32 quotient)."""
    top = 7 if bits == 4 else 127
    x = x.astype(np.float64)
    s = (np.max(np.abs(x), axis=-1) / top).astype(np.float32)
    with np.errstate(divide="ignore", invalid="ignore"):
        q = np.rint((x / s.astype(np.float64)[..., None]).astype(np.float32).astype(np.float64))
    return np.where(s[..., None] > 0, np.clip(q, -top, top), 0).astype(np.int64), s


def tokens(codes, scale, table, length, bits):
    """The values and visibility of positions [0, length) of a table's pages,
    [heads, length, D] and [length]."""
    pages, heads, page, _ = codes.shape
    length = min(max(int(length), 0), len(table) * page)
    at = np.arange(length)
    p = np.asarray(table, np.int64)[at // page] if length else np.zeros(0, np.int64)
    seen = (p >= 0) & (p < pages)
    p = np.where(seen, p, 0)
    v = unpack(codes[p, :, at % page], bits).astype(np.float64) * scale[p, :, at % page].astype(np.float64)[..., None]
    return v.transpose(1, 0, 2), seen


def attention(q, cache, tables, lengths, q_start=None, max_q=1, causal=True, prefix_table=None, prefix_length=0,
              scale=None, out=None):
    """out [T, Hq D] (rows of no sequence as `out` has them) and, for error
    bounds, sum_j p_j |v_j|, max_j over the visible of sum |q_d k_jd| scale.
    cache: (k, v, k_scale, v_scale, bits) as numpy arrays."""
    kc, vc, ks, vs, bits = cache
    H = kc.shape[1]
    D = kc.shape[3] * 8 // bits
    T, G = q.shape[0], q.shape[1] // (H * D)
    scale = D ** -0.5 if scale is None else scale
    out = np.full((T, q.shape[1]), np.nan) if out is None else out.astype(np.float64).copy()
    size, reach = np.zeros(out.shape), np.zeros((T, H * G))
    q = q.astype(np.float64).reshape(T, H, G, D)
    with np.errstate(invalid="ignore"):
        front = [tokens(c, s, prefix_table, prefix_length, bits) for c, s in ((kc, ks), (vc, vs))] if prefix_table is not None else None
        for s in range(len(tables)):
            a, b = (s, s + 1) if q_start is None else (int(q_start[s]), int(q_start[s + 1]))
            (k, seen), (v, _) = (tokens(c, sc, tables[s], lengths[s], bits) for c, sc in ((kc, ks), (vc, vs)))
            L = k.shape[1]
            for i in range(min(b - a, max_q)):
                end = min(max(L - (b - a) + i + 1, 0), L) if causal else L
                keep = np.nonzero(seen[:end])[0]
                kk, vv = k[:, keep], v[:, keep]
                if front is not None:
                    f = np.nonzero(front[0][1])[0]
                    kk, vv = np.concatenate((front[0][0][:, f], kk), 1), np.concatenate((front[1][0][:, f], vv), 1)
                for h in range(H):
                    if kk.shape[1] == 0:
                        out[a + i, h * G * D:(h + 1) * G * D] = 0.0
                        continue
                    t = scale * (q[a + i, h] @ kk[h].T)
                    p = np.exp(t - t.max(axis=1, keepdims=True))
                    p /= p.sum(axis=1, keepdims=True)
                    out[a + i, h * G * D:(h + 1) * G * D] = (p @ vv[h]).reshape(-1)
                    size[a + i, h * G * D:(h + 1) * G * D] = (p @ np.abs(vv[h])).reshape(-1)
                    reach[a + i, h * G:(h + 1) * G] = (abs(scale) * (np.abs(q[a + i, h]) @ np.abs(kk[h]).T)).max(axis=1)
    return out, size, reach
