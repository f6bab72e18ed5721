"""cache_attention of steps that mix long runs of queries with single ones: sizes
that count the queries there are, not the longest run times the sequences.

Bar: that of test_gpu_attention.py."""
import ctypes

import numpy as np
import pytest
import torch

from bit_gemm_block_amd import decode as D
from bit_gemm_block_amd import w4a4 as W
from test_gpu_attention import check, make_cache, queries, tables_of

P = 0x10000


def size_and_status(T, q_heads, S, width, max_q, heads=8, page=64, dim=128):
    """Bytes of workspace, and what a call with a byte less says.  Fake addresses: a
    prefix needs a workspace at any size, so that a call whose sizes are taken
    ends at the missing byte."""
    c = ctypes.byref(D.CacheStruct(P, P, P, P, 1 << 20, heads, page, dim, 4))
    n = D.lib().w4a4_cache_attention_workspace_size(c, T, q_heads, S, width, max_q, 1)
    st = D.lib().w4a4_cache_attention(c, P, W.F32, q_heads * dim, T, q_heads, P, S, width, P, P, max_q, 1, P, 1, P, 0.1, P,
                                      W.F32, q_heads * dim, P, max(n, 1) - 1, None)
    return n, st


@pytest.mark.parametrize("T,q_heads,S,width,max_q", [
    (4096 + 127, 32, 128, 128, 4096),        # 128 sequences, one of 4096 queries, the others of one
    (2048 + 255, 32, 256, 128, 2048),
    (8192 + 63, 32, 64, 256, 8192),
    (32768 + 1023, 64, 1024, 512, 32768),
    (512 + 1023, 32, 1024, 64, 1 << 30),     # no more queries than there are rows
    ((1 << 19) - 1, 32, 1, 128, 1 << 19),    # just under 2^24 heads' rows: by the rows of q,
    (1 << 20, 32, 64, 128, 8191),            # and by the sequences' most
])
def test_sizes_that_are_taken(T, q_heads, S, width, max_q):
    n, st = size_and_status(T, q_heads, S, width, max_q)
    assert n > 0 and st == W.ERR_WORKSPACE


@pytest.mark.parametrize("T,q_heads,S,width,max_q", [
    (128 * 4096, 32, 128, 128, 4096),
    (1 << 19, 32, 1, 128, 1 << 19),
    (1 << 20, 32, 64, 128, 8192),
])
def test_sizes_that_are_refused(T, q_heads, S, width, max_q):
    assert size_and_status(T, q_heads, S, width, max_q) == (0, W.ERR_UNSUPPORTED)


@pytest.mark.parametrize("dim", [64, 128, 256])
@pytest.mark.parametrize("S", [1, 3, 64])
def test_workspace_is_bounded_by_the_chip(dim, S):
    # Many rows: partial results of eight rounds of 768 workgroups of 64 rows, at
    # most, however long the prompts.
    largest = 8 * 768 * 64 * (dim + 2) * 4 + (S + 1) * 8
    for q_heads in (8, 32, 56):
        for n in (17, 100, 1000, 2048, 4096, 5000, 8192, 16384):
            if n * S * q_heads < 1 << 24:
                c = ctypes.byref(D.CacheStruct(P, P, P, P, 1 << 20, 8, 64, dim, 4))
                for T in {n * S, n + S - 1}:     # all as long, or one
                    need = D.lib().w4a4_cache_attention_workspace_size(c, T, q_heads, S, 512, n, 0)
                    assert need <= largest, (q_heads, n, T, need)


def mixed(counts, lengths, heads, group, dim, bits, dt, width, seed, spare=3, **kw):
    start = np.concatenate(([0], np.cumsum(counts)))
    page = 32
    pages = sum(-(-n // page) for n in lengths) + 1
    cache = make_cache(pages, heads, page, dim, bits, seed)
    tables, rest = tables_of(pages, lengths, page, np.random.default_rng(seed), width=width)
    if kw.pop("prefix", False):
        kw.update(prefix_table=tables[0, :4].copy(), prefix_length=101)
    q = queries(int(start[-1]) + spare, heads * group, dim, dt, seed)
    check(q, cache, tables, lengths, q_start=start, **kw)


# Sequences to look through for a row's: one, up to 64 at once, in two rounds and in
# three; none, one or several queries of each; tables for parts and for none.
@pytest.mark.gpu
@pytest.mark.parametrize("S", [1, 2, 3, 63, 64, 65, 130, 1000, 4100])
@pytest.mark.parametrize("width", [12, 130])
def test_one_prompt_among_decoding_sequences(S, width):
    print("attention mixed", S, width, flush=True)
    rng = np.random.default_rng(S)
    for at in sorted({0, S // 2, S - 1}):
        counts, lengths = rng.integers(0, 2, S), rng.integers(0, 40, S)
        counts[at], lengths[at] = 41, 350 if width == 12 else 4100
        mixed(counts, lengths.tolist(), 2, 4, 64, 4, "f32", width, S, max_q=41, prefix=S in (3, 130) and at == 0)


@pytest.mark.gpu
@pytest.mark.parametrize("group", [1, 3, 7, 16, 40, 64, 65, 130])
@pytest.mark.parametrize("dim,bits,dt", [(64, 4, "f16"), (128, 8, "f32"), (256, 4, "f32")])
def test_runs_of_every_length(group, dim, bits, dt):
    # Runs of queries that begin and end anywhere in 64 rows; empty ones side by
    # side, at the front and at the end.
    print("attention runs", group, dim, bits, dt, flush=True)
    counts = [0, 0, 5, 1, 0, 64, 63, 0, 0, 2, 17, 1, 1, 33, 0]
    lengths = [9, 0, 5, 70, 3, 64, 100, 1, 0, 1, 200, 0, 33, 30, 2]
    for kw in (dict(max_q=64), dict(max_q=64, causal=False), dict(max_q=40)):
        mixed(counts, lengths, 1, group, dim, bits, dt, 40, group, **kw)


# A tile of rows that waves share, its sequences with none to three queries: joined
# by the rows of q where there are fewer than three of each.
@pytest.mark.gpu
@pytest.mark.parametrize("counts", [[0, 3, 0, 1, 0], [3, 1, 0, 0, 2, 1, 1], [1, 0] * 40 + [3], [0] * 70 + [2, 3]])
@pytest.mark.parametrize("group", [1, 4, 5])
@pytest.mark.parametrize("width", [4, 130])
@pytest.mark.parametrize("prefix", [False, True])
def test_drafts_of_several_lengths(counts, group, width, prefix):
    print("attention drafts", len(counts), group, width, prefix, flush=True)
    rng = np.random.default_rng(len(counts))
    lengths = rng.integers(1, 60, len(counts))
    lengths[[1, -1]] = 128 if width == 4 else 2900, 100
    mixed(counts, lengths.tolist(), 2, group, 128, 4, "f32", width, group, spare=1, max_q=3, prefix=prefix)


@pytest.mark.gpu
def test_more_places_than_a_grid():
    # 1024 sequences of which one has 512 queries, of 32 heads: 2^24 places of rows,
    # of which 1535 are there.
    print("attention many places", flush=True)
    counts, lengths = [1] * 1024, [1 + s % 30 for s in range(1024)]
    counts[700], lengths[700] = 512, 600
    mixed(counts, lengths, 2, 16, 64, 4, "f16", 40, 1, max_q=512)


@pytest.mark.gpu
def test_a_captured_step_follows_the_runs():
    # One graph whose replays have their queries in other sequences.
    print("attention mixed graph", flush=True)
    S, heads, group, dim, page, T = 70, 2, 4, 64, 32, 200
    dev = "cuda:0"
    _, c = make_cache(300, heads, page, dim, 4, 3)
    rng = np.random.default_rng(3)
    tables = torch.from_numpy(rng.integers(0, 300, (S, 80)).astype(np.int32)).to(dev)
    q = torch.from_numpy(queries(T, heads * group, dim, "f32", 3)).to(dev)
    lengths, start = (torch.zeros(n, dtype=torch.int32, device=dev) for n in (S, S + 1))
    ws = D.cache_attention_workspace(c, T, heads * group, S, 80, 130)
    out = torch.zeros((T, heads * group * dim), device=dev)
    args = dict(q_start=start, max_q=130, out=out)
    D.cache_attention(q, c, tables, lengths, workspace=ws, **args)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        D.cache_attention(q, c, tables, lengths, workspace=ws, **args)
    for k in range(4):
        counts = rng.integers(0, 2, S)
        counts[(17 * k) % S] = 100 + 10 * k
        start.copy_(torch.from_numpy(np.concatenate(([0], np.cumsum(counts))).astype(np.int32)))
        lengths.copy_(torch.from_numpy(rng.integers(0, 2500, S).astype(np.int32)))
        out.fill_(5.0)
        D.cache_attention(q, c, tables, lengths, **args)
        torch.cuda.synchronize()
        want = out.clone()
        out.fill_(5.0)
        ws.random_(0, 255)
        g.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, want), k
        assert bool((out[int(start[-1]):] == 5).all())
