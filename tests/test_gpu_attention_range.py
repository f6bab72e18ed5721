"""cache_attention at the ends of float32's range, on the GPU: values of very
different sizes among tokens of like scores, and scores far below zero.

Bar of both: scores that are equal are equal as they are computed, so that every
weight is the same, and exact; what is left of the bar in test_gpu_attention.py
are the weights' pair, 2^-20, and the sums, 8 u (tokens / 32 + 64), of sum p |v|,
and a weight's cut-off, 2^-33 of the row's largest for each token.
"""
import numpy as np
import pytest
import torch

from bit_gemm_block_amd import decode as D
from oracle import decode_oracle as O
from test_gpu_attention import U, dev, host, tables_of

pytestmark = pytest.mark.gpu


def run(codes, ks, vs, bits, tables, lengths, q, **kw):
    """Outputs and reference of a cache with keys that are 1 in channel 0."""
    k, v = codes
    arrays = (O.pack(k, bits), O.pack(v, bits), ks, vs, bits)
    cache = D.KVCache(*(dev(t) for t in arrays[:4]), bits)
    ref, size, _ = O.attention(q, arrays, tables, lengths, **kw)
    g = {n: dev(np.asarray(c, np.int32)) if n in ("q_start", "prefix_table") else c for n, c in kw.items()}
    if "prefix_length" in kw:
        g["prefix_length"] = dev(np.array([kw["prefix_length"]], np.int32))
    got = host(D.cache_attention(dev(q), cache, dev(tables), dev(np.asarray(lengths, np.int32)),
                                 out_dtype=torch.float32, **g)).astype(np.float64)
    n = tables.shape[1] * ks.shape[2] * 2
    tol = size * (2.0 ** -20 + 8 * U * (n / 32 + 64)) + 2.0 ** -33 * n * size.max(axis=1, keepdims=True)
    return got, ref, tol


@pytest.mark.parametrize("large", [60, 70, 90, 99])
@pytest.mark.parametrize("n", [1, 6, 40])
@pytest.mark.parametrize("bits", [4, 8])
def test_large_values_among_zeros(bits, n, large):
    # Tokens whose values are zero (an all-zero row has scale zero), or tiny, in
    # front of ones of 2^large: all count alike in the sum of the weights.  In one
    # wave's tokens, in some waves' only, in other runs, and in front of a prefix.
    print("attention far values", bits, n, large, flush=True)
    heads, group, dim, page = 1, 4, 64, 32
    rng = np.random.default_rng(large)
    pages = 70
    k = np.zeros((pages, heads, page, dim), np.int64)
    k[..., 0] = 1
    v = rng.integers(1, 8, k.shape)
    ks = np.ones((pages, heads, page), np.float32)
    q = np.zeros((3 * n, group * dim), np.float32)
    q[:, ::dim] = 0.25
    start = np.arange(4) * n
    lengths = [700, 333, 64]
    tables, rest = tables_of(pages, lengths, page, rng)
    order = np.concatenate([t[t >= 0] for t in tables])
    for small in (0.0, 2.0 ** -60, 2.0 ** -100):
        for where in ("front", "waves", "end", "prefix"):
            vs = np.full(ks.shape, np.float32(2.0 ** large))
            if where == "front":
                vs[order[:11]] = small                          # the first half of sequence 0
                vs[tables[1, :5]] = small
                vs[tables[2, 0]] = small
            elif where == "waves":
                vs[order[::4]] = small                          # steps that one wave takes
            elif where == "end":
                vs[order[11:22]] = small
                vs[tables[1, 5:11]] = small
            else:
                vs[rest] = small
            kw = dict(q_start=start, max_q=n, causal=False)
            if where == "prefix":
                kw.update(prefix_table=rest[:20], prefix_length=601)
            got, ref, tol = run((k, v), ks, vs, bits, tables, lengths, q, **kw)
            assert np.all(np.abs(got - ref) <= tol), (small, where, float(np.max(np.abs(got - ref) / tol)))


@pytest.mark.parametrize("size", [90, 100, 112])
@pytest.mark.parametrize("n", [1, 6, 40])
def test_scores_far_below_zero(n, size):
    # All scores are -2^size: weights alike, as at any other score.
    print("attention low scores", n, size, flush=True)
    heads, group, dim, page = 1, 4, 64, 32
    rng = np.random.default_rng(size)
    k = np.zeros((70, heads, page, dim), np.int64)
    k[..., 0] = 1
    v = rng.integers(-7, 8, k.shape)
    ks = np.ones((70, heads, page), np.float32)
    vs = (2.0 ** rng.integers(-4, 5, ks.shape)).astype(np.float32)
    q = np.zeros((3 * n, group * dim), np.float32)
    q[:, ::dim] = -(2.0 ** size)
    lengths = [700, 333, 64]
    tables, rest = tables_of(70, lengths, page, rng)
    for kw in ({}, dict(prefix_table=rest[:20], prefix_length=601)):
        got, ref, tol = run((k, v), ks, vs, 4, tables, lengths, q, q_start=np.arange(4) * n, max_q=n, scale=1.0, **kw)
        assert np.all(np.abs(got - ref) <= tol), float(np.max(np.abs(got - ref) / tol))
