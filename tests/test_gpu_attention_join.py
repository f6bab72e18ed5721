"""cache_attention where many rows are joined from many parts, on the GPU.

Bar: that of test_gpu_attention.py."""
import numpy as np
import pytest
import torch

from bit_gemm_block_amd import decode as D
from oracle import decode_oracle as O
from test_gpu_attention import DEV, bar, check, dev, host, make_cache, queries, tables_of

pytestmark = pytest.mark.gpu


def counts(ws, seqs):
    """How many parts every sequence had: the last words of a workspace that a
    call has used, (first, number) for each sequence and the prefix."""
    return ws[-8 * (seqs + 1):].view(torch.int32).view(seqs + 1, 2)[:seqs, 1].tolist()


def whole(q, cache, table, length, causal):
    """One sequence and head of the cache, all its queries at once, as oracle's
    attention returns them."""
    kc, vc, ks, vs, bits = cache
    (k, _), (v, _) = (O.tokens(c, s, table, length, bits) for c, s in ((kc, ks), (vc, vs)))
    k, v, q = k[0], v[0], q.astype(np.float64)
    hidden = np.zeros((len(q), length), bool)
    if causal:
        hidden = np.arange(length) > length - len(q) + np.arange(len(q))[:, None]
    t = np.where(hidden, -np.inf, q @ k.T * k.shape[1] ** -0.5)
    p = np.exp(t - t.max(axis=1, keepdims=True))
    p /= p.sum(axis=1, keepdims=True)
    reach = np.where(hidden, 0, np.abs(q) @ np.abs(k).T * k.shape[1] ** -0.5).max(axis=1, keepdims=True)
    return p @ v, p @ np.abs(v), reach


# Part counts on both sides of what the join takes at once, and those that leave
# its lanes a part too many.
@pytest.mark.parametrize("parts", [16, 17, 18, 21, 33, 34, 35, 37, 48, 63, 64, 65, 81])
@pytest.mark.parametrize("dim", [64, 128, 256])
def test_one_long_sequence_among_short_ones(dim, parts):
    print("attention join runs", dim, parts, flush=True)
    S, heads, group, page = 64, 2, 4, 64
    lengths = [100] * S
    lengths[40] = 256 * (parts - 1) + 5
    pages = sum(-(-n // page) for n in lengths) + 1
    cache = make_cache(pages, heads, page, dim, 4, parts)
    tables, _ = tables_of(pages, lengths, page, np.random.default_rng(parts))
    q = queries(S, heads * group, dim, "f32", parts)
    got = check(q, cache, tables, lengths)
    ws = D.cache_attention_workspace(cache[1], S, heads * group, S, tables.shape[1])
    again = D.cache_attention(dev(q), cache[1], dev(tables), dev(np.array(lengths, np.int32)), out_dtype=torch.float32,
                              workspace=ws)
    assert np.array_equal(host(again), got)
    assert S * heads * group >= 512 and counts(ws, S) == [parts if s == 40 else 1 for s in range(S)]


@pytest.mark.parametrize("parts", [17, 21, 33, 35, 48, 63, 65, 70])
@pytest.mark.parametrize("dim", [64, 128])
def test_one_prompt_in_many_parts(dim, parts):
    print("attention join prompt", dim, parts, flush=True)
    n, page, L = 520, 64, 256 * parts + 10
    pages = -(-L // page) + 1
    cache = make_cache(pages, 1, page, dim, 4, parts)
    tables, _ = tables_of(pages, [L], page, np.random.default_rng(parts))
    q = queries(n, 1, dim, "f32", parts)
    ws = D.cache_attention_workspace(cache[1], n, 1, 1, tables.shape[1], n)
    for causal in (True, False):
        got = host(D.cache_attention(dev(q), cache[1], dev(tables), dev(np.array([L], np.int32)),
                                     q_start=dev(np.array([0, n], np.int32)), max_q=n, causal=causal,
                                     out_dtype=torch.float32, workspace=ws))
        assert counts(ws, 1) == [parts]
        ref, size, reach = whole(q, cache[0], tables[0], L, causal)
        tol = bar(ref, size, reach, tables.shape[1] * page, "f32")
        assert np.all(np.abs(got - ref) <= tol), float(np.max(np.abs(got - ref) / tol))
