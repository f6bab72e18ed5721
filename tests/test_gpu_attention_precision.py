"""cache_attention with float32 outputs is no less exact than the formula in float32
operations, on the GPU.

Norm of the error over the norm of the output, against 64 bits, beside that of
numpy's float32 products, exp and sums on the same values.  Both round a score's
sum, its exponent, the sums over the tokens and the result to float32.  The kernel
rounds a score once for each 16 or 32 products at most and numpy no less often; a
query's and a weight's pair add 2^-23 each, as do the power of two and the
quotient.  So its error is at most as large, up to what a norm over some thousand
outputs varies: a half more is allowed.
"""
import numpy as np
import pytest

from oracle import decode_oracle as O
from test_gpu_attention import check, make_cache, queries, tables_of

pytestmark = pytest.mark.gpu


def in_float32(q, cache, tables, lengths, n, prefix, P):
    kc, vc, ks, vs, bits = cache
    H, D = kc.shape[1], kc.shape[3] * 8 // bits
    G = q.shape[1] // (H * D)
    q = q.astype(np.float32).reshape(len(q), H, G, D)
    out = np.zeros(q.shape, np.float32)
    front = [O.tokens(c, s, prefix, P, bits)[0] for c, s in ((kc, ks), (vc, vs))]
    for s, L in enumerate(lengths):
        k, v = (np.concatenate((f, O.tokens(c, sc, tables[s], L, bits)[0]), 1).astype(np.float32)
                for f, (c, sc) in zip(front, ((kc, ks), (vc, vs))))
        for h in range(H):
            for i in range(n):
                end = P + L - n + i + 1
                t = (q[s * n + i, h] @ k[h, :end].T) * np.float32(D ** -0.5)
                p = np.exp(t - t.max(axis=1, keepdims=True))
                out[s * n + i, h] = (p @ v[h, :end]) / p.sum(axis=1, keepdims=True)
    return out.reshape(len(q), -1)


# One query and many (a tile that waves share, and rows of their own), a prefix.
@pytest.mark.parametrize("dim,bits", [(64, 4), (64, 8), (128, 4), (128, 8), (256, 4), (256, 8)])
@pytest.mark.parametrize("dt", ["f16", "f32"])
@pytest.mark.parametrize("n,group,prefix", [(1, 4, 0), (1, 1, 0), (30, 4, 0), (1, 4, 900), (1, 12, 900)])
def test_no_less_exact_than_float32(dim, bits, dt, n, group, prefix):
    print("attention precision", dim, bits, dt, n, group, prefix, flush=True)
    heads, page, lengths = 4, 32, [1500, 300, 2200, 777]
    pages = sum(-(-L // page) for L in lengths) + 29
    cache = make_cache(pages, heads, page, dim, bits, dim + bits + n)
    tables, rest = tables_of(pages, lengths, page, np.random.default_rng(n))
    S = len(lengths)
    q = queries(S * n, heads * group, dim, dt, n + group)
    kw = dict(prefix_table=rest, prefix_length=prefix) if prefix else {}
    kw.update(q_start=np.arange(S + 1) * n, max_q=n)
    got = check(q, cache, tables, lengths, **kw)
    ref, _, _ = O.attention(q, cache[0], tables, lengths, **kw)
    plain = in_float32(q, cache[0], tables, lengths, n, rest, prefix)
    off, plain_off = (float(np.linalg.norm(a - ref) / np.linalg.norm(ref)) for a in (got, plain))
    print("  off by %.2e, float32 by %.2e" % (off, plain_off), flush=True)
    assert off <= 1.5 * plain_off
