"""cache_attention against the float64 reference, on the GPU.

Bar, u = 2^-24.  A score t = scale q . k is off by the query's pair (2^-22 of the
products' absolute sum; fp16 queries exactly nothing) and float32 sums of its
matrix instructions (at most 16 in a chain, 2 u a step and addend), its factors
(4 u) and its difference to the reference, at most 64 u of the largest absolute
sum of products ("reach") in all; exp2 adds 4 u.  So p and its sum are off by
e = reach (2^-22 + 96 u) + 8 u of themselves, the quotient by twice that.  The
weights' pair adds 2^-20, their cut-off 2^-33 of the row's largest for each
token; sums over n steps of 32 tokens, parts and waves 8 u a step.  Of
sum p |v|: 2 e + 2^-20 + 8 u (n + 64); of its largest in the row: 2^-33 tokens.
An fp16 result is rounded once more (2^-11 of the value, at least 2^-25).
"""
import numpy as np
import pytest
import torch

from bit_gemm_block_amd import decode as D
from bit_gemm_block_amd import w4a4 as W
from oracle import decode_oracle as O

pytestmark = pytest.mark.gpu

DEV = "cuda:0"
U = 2.0 ** -24
NP = {"f16": np.float16, "f32": np.float32}
TORCH = {"f16": torch.float16, "f32": torch.float32}


def dev(a):
    return None if a is None else torch.from_numpy(np.ascontiguousarray(a)).to(DEV)


def host(t):
    torch.cuda.synchronize()
    return t.cpu().numpy()


def make_cache(pages, heads, page, dim, bits, seed):
    """Codes of quantized normal rows (two channels of the keys larger) and
    scales that differ from row to row; as numpy and on the GPU."""
    rng = np.random.default_rng(seed)
    out = []
    for gain in (4.0, 1.0):
        x = rng.standard_normal((pages, heads, page, dim)).astype(np.float32)
        x[..., 7::dim // 2] *= gain
        x *= 2.0 ** rng.uniform(-1, 1, (pages, heads, page, 1)).astype(np.float32)
        q, s = O.quantize(x, bits)
        out.append((O.pack(q, bits), s))
    a = (out[0][0], out[1][0], out[0][1], out[1][1])
    return a + (bits,), D.KVCache(*(dev(t) for t in a), bits)


def tables_of(pages, lengths, page, rng, width=None):
    """Pages of every sequence, drawn without repetition; -1 behind them."""
    need = [-(-max(L, 0) // page) for L in lengths]
    order = rng.permutation(pages)
    assert sum(need) <= pages
    t = np.full((len(lengths), max(need + [1]) if width is None else width), -1, np.int32)
    at = 0
    for i, n in enumerate(need):
        t[i, :n] = order[at:at + n]
        at += n
    return t, order[at:].astype(np.int32)


def bar(ref, size, reach, tokens, out):
    e = np.repeat(reach, ref.shape[1] // reach.shape[1], axis=1) * (2.0 ** -22 + 96 * U) + 8 * U
    tol = size * (2 * e + 2.0 ** -20 + 8 * U * (tokens / 32 + 64)) + 2.0 ** -33 * tokens * size.max(axis=1, keepdims=True)
    return tol + np.maximum(2.0 ** -11 * np.abs(ref), 2.0 ** -25) if out == "f16" else tol


def check(q, cache, tables, lengths, out="f32", dt=None, keep=None, **kw):
    """The call against the reference; the rows that belong to no sequence are
    checked to be left as they were."""
    arrays, c = cache
    lengths = np.asarray(lengths, np.int32)
    o = dict(kw)
    if o.get("prefix_length") is not None:
        o["prefix_length"] = int(o["prefix_length"])
    ref, size, reach = O.attention(q, arrays, tables, lengths, **o)
    g = dict(kw)
    for name in ("q_start", "prefix_table"):
        if g.get(name) is not None:
            g[name] = dev(np.asarray(g[name], np.int32))
    if g.get("prefix_length") is not None:
        g["prefix_length"] = dev(np.array([g["prefix_length"]], np.int32))
    buf = torch.full((q.shape[0], q.shape[1]), 77.0, dtype=TORCH[out], device=DEV)
    got = host(D.cache_attention(dev(q), c, dev(tables), dev(lengths), out=buf, **g))
    none = np.isnan(ref[:, 0])
    assert np.all(got[none] == 77.0)
    cap = max(1, tables.shape[1] * c.k.shape[2] + (0 if kw.get("prefix_table") is None else len(kw["prefix_table"]) * c.k.shape[2]))
    tol = bar(ref, size, reach, cap, out)[~none]
    e = np.abs(got - ref)[~none]
    assert np.all(e <= tol), (float(np.nanmax(e / np.maximum(tol, 1e-300))), np.argwhere(~(e <= tol))[:4].tolist())
    return got


def queries(T, heads, dim, dt, seed):
    rng = np.random.default_rng(seed)
    return (1.5 * rng.standard_normal((T, heads * dim))).astype(NP[dt])


LENGTHS = [0, 1, 2, 15, 16, 17, 31, 32, 33, 63, 64, 65, 127, 128, 129, 200, 257, 1000]


@pytest.mark.parametrize("dim,bits", [(64, 4), (64, 8), (128, 4), (128, 8), (256, 4), (256, 8)])
@pytest.mark.parametrize("dt", ["f16", "f32"])
def test_decode_lengths(dim, bits, dt):
    print("attention lengths", dim, bits, dt, flush=True)
    for heads, group, page in ((2, 4, 16), (1, 1, 64)):
        cache = make_cache(sum(-(-n // page) for n in LENGTHS) + 2, heads, page, dim, bits, dim + bits)
        tables, _ = tables_of(cache[0][0].shape[0], LENGTHS, page, np.random.default_rng(1))
        check(queries(len(LENGTHS), heads * group, dim, dt, 3), cache, tables, LENGTHS)
        check(queries(len(LENGTHS), heads * group, dim, dt, 4), cache, tables, LENGTHS, out="f16")


@pytest.mark.parametrize("group", [1, 2, 3, 7, 8, 15, 16, 17, 32, 33, 40, 64, 65, 130])
@pytest.mark.parametrize("dim", [64, 128, 256])
def test_groups(group, dim):
    print("attention groups", group, dim, flush=True)
    lengths = [100, 1, 333]
    for bits, dt in ((4, "f32"), (8, "f16")):
        cache = make_cache(20, 3, 32, dim, bits, group)
        tables, _ = tables_of(20, lengths, 32, np.random.default_rng(2))
        check(queries(3, 3 * group, dim, dt, group), cache, tables, lengths)


@pytest.mark.parametrize("page", [16, 32, 64, 256])
@pytest.mark.parametrize("n", [2, 5, 9, 40, 150])
@pytest.mark.parametrize("causal", [True, False])
def test_several_queries(page, n, causal):
    # From one query to n, sequences shorter than their queries among them.
    print("attention queries", page, n, causal, flush=True)
    counts = [n, 1, 0, 2, n, n // 2 + 1]
    lengths = [n + 70, 1, 50, 1, n - 1, 300]
    start = np.concatenate(([0], np.cumsum(counts)))
    T = int(start[-1]) + 3                                   # rows of no sequence behind them
    pages = sum(-(-L // page) for L in lengths) + 1
    for dim, bits, heads, group, dt in ((64, 4, 2, 4, "f32"), (128, 8, 1, 7, "f16"), (128, 4, 2, 1, "f32"), (256, 4, 1, 2, "f16")):
        cache = make_cache(pages, heads, page, dim, bits, n)
        tables, _ = tables_of(pages, lengths, page, np.random.default_rng(n))
        check(queries(T, heads * group, dim, dt, n), cache, tables, lengths, q_start=start, max_q=n, causal=causal)


def test_queries_past_max_q_are_left():
    print("attention max_q", flush=True)
    cache = make_cache(10, 2, 16, 64, 4, 1)
    tables, _ = tables_of(10, [60, 70], 16, np.random.default_rng(1))
    check(queries(12, 4, 64, "f32", 1), cache, tables, [60, 70], q_start=[0, 7, 12], max_q=4)


@pytest.mark.parametrize("prefix", [0, 1, 16, 33, 100, 700])
@pytest.mark.parametrize("dim,bits", [(64, 4), (128, 8), (128, 4), (256, 4)])
def test_shared_prefix(prefix, dim, bits):
    print("attention prefix", prefix, dim, bits, flush=True)
    page = 32
    lengths = [0, 1, 40, 31, 300, 5, 64]
    pages = sum(-(-n // page) for n in lengths) + -(-prefix // page) + 1
    for heads, group, dt, out in ((2, 4, "f32", "f32"), (1, 7, "f16", "f16")):
        cache = make_cache(pages, heads, page, dim, bits, prefix)
        tables, rest = tables_of(pages, lengths, page, np.random.default_rng(prefix))
        S = len(lengths)
        check(queries(S + 2, heads * group, dim, dt, 5), cache, tables, lengths, out=out, prefix_table=rest,
              prefix_length=prefix)
        start = np.array([0, 0, 1, 4, 9, 20, 25, 26])        # none to eleven queries
        check(queries(28, heads * group, dim, dt, 6), cache, tables, lengths, out=out, q_start=start, max_q=11,
              prefix_table=rest, prefix_length=prefix)


def test_prefix_is_the_same_as_pages_in_front():
    # A prefix that ends with a page, and the same pages in every table.
    print("attention prefix in tables", flush=True)
    heads, group, dim, page = 2, 4, 128, 16
    cache = make_cache(40, heads, page, dim, 4, 8)
    lengths = np.array([20, 3, 64, 17, 1], np.int32)
    tables, rest = tables_of(40, lengths, page, np.random.default_rng(8))
    q = queries(5, heads * group, dim, "f32", 8)
    ref, size, reach = O.attention(q, cache[0], np.concatenate((np.tile(rest[:6], (5, 1)), tables), 1), lengths + 96)
    got = host(D.cache_attention(dev(q), cache[1], dev(tables), dev(lengths), prefix_table=dev(rest[:6]),
                                 prefix_length=dev(np.array([96], np.int32)), out_dtype=torch.float32))
    assert np.all(np.abs(got - ref) <= bar(ref, size, reach, 200, "f32"))


@pytest.mark.parametrize("prefix", [False, True])
def test_pages_that_do_not_exist(prefix):
    # Absent pages hold nothing, wherever they are; lengths beyond the table end with it.
    print("attention bad pages", prefix, flush=True)
    heads, group, dim, page = 2, 2, 64, 16
    cache = make_cache(30, heads, page, dim, 4, 3)
    lengths = [100, 90, 16, 40, 4000, -5, 2 ** 31 - 1]
    tables = np.random.default_rng(4).permutation(30)[np.arange(7 * 7) % 30].reshape(7, 7).astype(np.int32)
    tables[0, 0], tables[0, 3], tables[1, 5] = -1, 30, -2 ** 31
    tables[2, :] = 2 ** 31 - 1
    tables[3, 1] = 99
    kw = dict(prefix_table=np.array([3, -1, 5, 30, 8], np.int32), prefix_length=75) if prefix else {}
    check(queries(7, heads * group, dim, "f32", 1), cache, tables, lengths, **kw)
    start = np.array([0, 3, 20, 21, 25, 60, 61, 64])
    check(queries(64, heads * group, dim, "f32", 2), cache, tables, lengths, q_start=start, max_q=40, **kw)
    if prefix:
        for n in (-1, 1000, 2 ** 31 - 1):
            check(queries(7, heads * group, dim, "f16", 3), cache, tables, lengths, prefix_table=kw["prefix_table"],
                  prefix_length=n)


@pytest.mark.parametrize("bits", [4, 8])
@pytest.mark.parametrize("dt", ["f16", "f32"])
def test_what_masked_positions_hold(bits, dt):
    # Slots behind a sequence's end and, for earlier queries, later tokens hold
    # NaN, infinities and huge values.
    print("attention masked", bits, dt, flush=True)
    heads, group, dim, page = 1, 4, 128, 32
    rng = np.random.default_rng(6)
    lengths = [45, 64, 1, 70]
    for trouble in (np.nan, np.inf, -np.inf, 3e38):
        (kc, vc, ks, vs, _), _ = make_cache(12, heads, page, dim, bits, 5)
        tables, _ = tables_of(12, lengths, page, rng)
        clean = ks.copy(), vs.copy()
        for s, L in enumerate(lengths):
            for at in range(L, -(-L // page) * page):
                ks[tables[s, at // page], :, at % page] = trouble
                vs[tables[s, at // page], :, at % page] = trouble
        cache = lambda a, b: ((kc, vc, a, b, bits), D.KVCache(dev(kc), dev(vc), dev(a), dev(b), bits))  # noqa: E731
        q = queries(4, group, dim, dt, 9)
        a = check(q, cache(ks, vs), tables, lengths)
        b = check(q, cache(*clean), tables, lengths)
        assert np.array_equal(a, b)
        # Sequence 0's last token is seen by the last of its nine queries only.
        start = np.array([0, 9, 13, 13, 14])
        q = queries(14, group, dim, dt, 10)
        b = check(q, cache(ks, vs), tables, lengths, q_start=start, max_q=9)
        ks[tables[0, 1], :, 12] = trouble
        vs[tables[0, 1], :, 12] = trouble
        _, c = cache(ks, vs)
        a = host(D.cache_attention(dev(q), c, dev(tables), dev(np.asarray(lengths, np.int32)), q_start=dev(start.astype(np.int32)),
                                   max_q=9, out_dtype=torch.float32))
        rest = [t for t in range(14) if t != 8]
        tol = bar(*O.attention(q, (kc, vc, *clean, bits), tables, lengths, q_start=start, max_q=9), 96, "f32")
        assert np.all(np.abs(a - b)[rest] <= 2 * tol[rest])
        if trouble != 3e38:
            assert not np.isfinite(a[8]).any()


@pytest.mark.parametrize("dt", ["f16", "f32"])
@pytest.mark.parametrize("n", [1, 30])
def test_scales_far_apart(dt, n):
    # Values of very different sizes, zero rows, keys that make one token win,
    # queries of very different sizes.
    print("attention far scales", dt, n, flush=True)
    heads, group, dim, page = 2, 4, 64, 16
    (kc, vc, ks, vs, bits), _ = make_cache(40, heads, page, dim, 4, 11)
    rng = np.random.default_rng(12)
    vs *= 2.0 ** rng.integers(-30, 31, vs.shape).astype(np.float32)
    vs[rng.random(vs.shape) < 0.2] = 0
    ks *= 2.0 ** rng.integers(-6, 3, ks.shape).astype(np.float32)
    cache = ((kc, vc, ks, vs, bits), D.KVCache(dev(kc), dev(vc), dev(ks), dev(vs), bits))
    lengths = [300, 40, 17, 200]
    tables, _ = tables_of(40, lengths, page, rng)
    q = queries(4 * n, heads * group, dim, dt, 13).reshape(4 * n * heads * group, dim)
    q *= (2.0 ** rng.integers(-12, 3, (len(q), 1))).astype(q.dtype)
    q[3] = 0
    q = q.reshape(4 * n, -1)
    start = np.arange(5) * n
    check(q, cache, tables, lengths, q_start=start, max_q=n)
    if dt == "f32":                                         # beyond fp16's range, scores as before
        big = q * np.float32(2.0 ** 40)
        check(big, cache, tables, lengths, q_start=start, max_q=n, scale=2.0 ** -40 / 8)
    check(q, cache, tables, lengths, q_start=start, max_q=n, scale=-0.3)
    check(q, cache, tables, lengths, q_start=start, max_q=n, scale=0.0)


def test_rising_scores():
    # Each token's score above all before it: the reference moves again and again.
    print("attention rising", flush=True)
    page, dim = 16, 64
    k = np.zeros((40, 1, page, dim), np.int64)
    k[..., 0] = 7
    ks = (np.arange(40 * page, dtype=np.float32).reshape(40, 1, page) + 1) / 7
    v = np.random.default_rng(1).integers(-7, 8, k.shape)
    vs = np.ones_like(ks)
    for step in (0.01, 0.5, 20.0, -0.5, -20.0):
        a = (O.pack(k, 4), O.pack(v, 4), ks * abs(step), vs, 4)
        cache = (a, D.KVCache(*(dev(t) for t in a[:4]), 4))
        q = np.zeros((2, dim), np.float32)
        q[:, 0] = np.sign(step)
        check(q, cache, np.tile(np.arange(40, dtype=np.int32), (2, 1)), [640, 333], scale=1.0)


def test_strides():
    # q as columns of one projection and at odd addresses, out likewise.
    print("attention strides", flush=True)
    heads, group, dim, page = 2, 2, 64, 16
    cache = make_cache(20, heads, page, dim, 4, 2)
    lengths = [50, 100, 7]
    tables, _ = tables_of(20, lengths, page, np.random.default_rng(2))
    C = heads * group * dim
    for dt in ("f16", "f32"):
        for out in ("f16", "f32"):
            q = queries(3, heads * group, dim, dt, 2)
            wide = torch.full((3, C + 9), float("nan"), dtype=TORCH[dt], device=DEV)
            wide[:, 3:3 + C] = dev(q)
            buf = torch.full((5, C + 5), 5.0, dtype=TORCH[out], device=DEV)
            args = (cache[1], dev(tables), dev(np.asarray(lengths, np.int32)))
            want = D.cache_attention(dev(q), *args, out_dtype=TORCH[out])
            got = D.cache_attention(wide[:, 3:3 + C], *args, out=buf[1:4, 1:1 + C])
            assert torch.equal(got, want)
            buf[1:4, 1:1 + C] = 5
            assert bool((buf == 5).all())


def test_long_sequence_and_offsets():
    # 40000 tokens of one sequence, its pages beyond 2^32 bytes of codes.
    print("attention long", flush=True)
    heads, dim, page, L = 1, 256, 128, 40001
    pages = (1 << 32) // (page * dim) + 400
    c = D.KVCache.empty(pages, heads, page, dim, 8, DEV)
    n = -(-L // page)
    (kc, vc, ks, vs, _), small = make_cache(n, heads, page, dim, 8, 4)
    order = np.arange(pages - n, pages)[::-1].astype(np.int64)
    at = dev(order)
    for name in ("k", "v", "k_scale", "v_scale"):
        getattr(c, name)[at] = getattr(small, name)
    q = queries(1, 2, dim, "f32", 4)
    ref, size, reach = O.attention(q, (kc, vc, ks, vs, 8), np.arange(n)[None], [L])
    got = host(D.cache_attention(dev(q), c, dev(order[None].astype(np.int32)), dev(np.array([L], np.int32)),
                                 out_dtype=torch.float32))
    assert np.all(np.abs(got - ref) <= bar(ref, size, reach, L, "f32"))


def test_sequences_do_not_depend_on_each_other():
    print("attention alone", flush=True)
    heads, group, dim, page = 2, 4, 128, 16
    cache = make_cache(60, heads, page, dim, 4, 6)
    lengths = np.array([300, 20, 100, 1], np.int32)
    tables, _ = tables_of(60, lengths, page, np.random.default_rng(6))
    q = queries(4, heads * group, dim, "f32", 6)
    f = lambda q, t, n: host(D.cache_attention(dev(q), cache[1], dev(t), dev(n), out_dtype=torch.float32))  # noqa: E731
    want = f(q, tables, lengths)
    assert np.array_equal(f(q, tables, lengths), want)
    q2, n2 = q.copy(), lengths.copy()
    q2[0], n2[0] = np.nan, 5
    assert np.array_equal(f(q2, tables, n2)[1:], want[1:])


def test_empty_and_refused():
    cache = make_cache(8, 2, 16, 64, 4, 1)[1]
    q = torch.zeros((3, 256), device=DEV)
    t, n = torch.zeros((3, 2), dtype=torch.int32, device=DEV), torch.ones(3, dtype=torch.int32, device=DEV)
    s = torch.tensor([0, 1, 2, 3], dtype=torch.int32, device=DEV)
    assert D.cache_attention(q[:0], cache, t[:0], n[:0]).shape == (0, 256)
    assert bool((D.cache_attention(q, cache, t[:, :0].contiguous(), n) == 0).all())     # tables without pages
    bad = [dict(q=q[:, :100]), dict(q=q[0]), dict(q=q.t()), dict(q=q.cpu()), dict(tables=t[0]), dict(tables=t[:2]),
           dict(lengths=n[:2]), dict(q=q[:2]), dict(max_q=2), dict(q_start=s[:3]), dict(prefix_table=s), dict(prefix_length=n[:1]),
           dict(prefix_table=s, prefix_length=n), dict(tables=t.t().contiguous().t()), dict(out=q[:, :128].half()),
           dict(lengths=n.cpu())]
    for kw in bad:
        a = dict(q=q, cache=cache, tables=t, lengths=n, **{k: v for k, v in kw.items() if k not in ("q", "tables", "lengths")})
        a.update({k: v for k, v in kw.items() if k in ("q", "tables", "lengths")})
        with pytest.raises(ValueError):
            D.cache_attention(a.pop("q"), a.pop("cache"), a.pop("tables"), a.pop("lengths"), **a)
    for kw in (dict(tables=t.long()), dict(lengths=n.long()), dict(q=q.double())):
        a = dict(q=q, tables=t, lengths=n)
        a.update(kw)
        with pytest.raises(TypeError):
            D.cache_attention(a["q"], cache, a["tables"], a["lengths"])
    for kw in (dict(scale=float("nan")), dict(q_start=s, max_q=0)):
        with pytest.raises(W.W4A4Error):
            D.cache_attention(q, cache, t, n, **kw)
    with pytest.raises(W.W4A4Error):                        # 4 heads of the cache, 3 of q
        D.cache_attention(q[:, :192], cache, t, n)
    with pytest.raises(W.W4A4Error):
        D.cache_attention(q, cache, torch.zeros((3, 64), dtype=torch.int32, device=DEV), n,
                          workspace=torch.empty(16, dtype=torch.uint8, device=DEV))


@pytest.mark.parametrize("prefix", [False, True])
def test_graph_and_streams(prefix):
    # A captured step follows the tables, lengths and the cache's contents.
    print("attention graph", prefix, flush=True)
    heads, group, dim, page = 2, 4, 128, 16
    _, c = make_cache(80, heads, page, dim, 4, 7)
    rng = np.random.default_rng(7)
    tables = dev(rng.permutation(80)[:60].reshape(4, 15).astype(np.int32))
    lengths = dev(np.array([200, 3, 50, 0], np.int32))
    q = dev(queries(4, heads * group, dim, "f32", 7))
    kw = dict(prefix_table=dev(np.arange(20, dtype=np.int32)), prefix_length=dev(np.array([310], np.int32))) if prefix else {}
    ws = D.cache_attention_workspace(c, 4, heads * group, 4, 15, prefix_width=20 if prefix else 0)
    out = torch.zeros((4, heads * group * dim), device=DEV)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        got = D.cache_attention(q, c, tables, lengths, out_dtype=torch.float32, **kw)
    side.synchronize()
    assert torch.equal(got, D.cache_attention(q, c, tables, lengths, out_dtype=torch.float32, **kw))
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        D.cache_attention(q, c, tables, lengths, out=out, workspace=ws, **kw)
    for k in range(4):
        q.mul_(-1.1)
        lengths.add_(7)
        tables.copy_(tables.flip(0))
        if prefix:
            kw["prefix_length"].sub_(90)
        want = D.cache_attention(q, c, tables, lengths, out_dtype=torch.float32, **kw)
        out.zero_()
        ws.random_(0, 255)
        g.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, want), k


@pytest.mark.parametrize("dim,bits,dt", [(64, 4, "f32"), (64, 8, "f16"), (128, 8, "f32"), (128, 4, "f16")])
def test_long_parts_of_many_rows(dim, bits, dt):
    # So many sequences that one of 9000 tokens is cut into eight parts of 36 steps
    # of 32 only, more than whose pages are looked up at once; some of them absent.
    print("attention long parts", dim, bits, dt, flush=True)
    S, heads, group, page = 96, 8, 20, 64
    lengths = [9000] + [1] * (S - 1)
    cache = make_cache(240, heads, page, dim, bits, 21)
    tables, _ = tables_of(240, lengths, page, np.random.default_rng(3), width=144)
    tables[0, [5, 18, 70, 71, 140]] = [-1, 240, -7, 1 << 30, -1]
    check(queries(S, heads * group, dim, dt, 9), cache, tables, lengths)


@pytest.mark.parametrize("dt", ["f16", "f32"])
def test_long_runs_of_few_rows(dt):
    # So many heads that one workgroup takes all tokens of a head, its waves 36
    # steps each.  The reference takes three of the heads.
    print("attention long runs", dt, flush=True)
    heads, dim, page, lengths = 768, 64, 64, [4500, 300]
    g = np.random.default_rng(4)
    kc, vc = (g.integers(0, 256, (78, heads, page, dim // 2), dtype=np.uint8) for _ in range(2))
    ks, vs = (g.uniform(0.01, 0.05, (78, heads, page)).astype(np.float32) for _ in range(2))
    tables, _ = tables_of(78, lengths, page, g)
    tables[0, [3, 66]] = -1
    q = queries(2, heads, dim, dt, 5)
    got = host(D.cache_attention(dev(q), D.KVCache(dev(kc), dev(vc), dev(ks), dev(vs), 4), dev(tables),
                                 dev(np.array(lengths, np.int32)), out_dtype=torch.float32)).reshape(2, heads, dim)
    at = [0, 400, 767]
    few = tuple(np.ascontiguousarray(t[:, at]) for t in (kc, vc, ks, vs))
    ref, size, reach = O.attention(q.reshape(2, heads, dim)[:, at].reshape(2, -1), few + (4,), tables, lengths)
    assert np.all(np.abs(got[:, at].reshape(2, -1) - ref) <= bar(ref, size, reach, tables.shape[1] * page, "f32"))


@pytest.mark.parametrize("n", [1, 30])
def test_scales_of_either_sign(n):
    # A cache that a caller filled: values are codes times scales, whatever their signs.
    print("attention signs", n, flush=True)
    heads, group, dim, page = 2, 4, 64, 16
    (kc, vc, ks, vs, bits), _ = make_cache(40, heads, page, dim, 8, 14)
    rng = np.random.default_rng(15)
    vs *= (rng.choice([-1.0, 1.0], vs.shape) * 2.0 ** rng.integers(-30, 31, vs.shape)).astype(np.float32)
    ks *= rng.choice([-1.0, 1.0], ks.shape).astype(np.float32)
    cache = ((kc, vc, ks, vs, bits), D.KVCache(dev(kc), dev(vc), dev(ks), dev(vs), bits))
    lengths = [300, 40, 17, 200]
    tables, _ = tables_of(40, lengths, page, rng)
    check(queries(4 * n, heads * group, dim, "f32", 16), cache, tables, lengths, q_start=np.arange(5) * n, max_q=n)
    vs[:] = -np.float32(2.0 ** 40)
    cache = ((kc, vc, ks, vs, bits), D.KVCache(dev(kc), dev(vc), dev(ks), dev(vs), bits))
    check(queries(4 * n, heads * group, dim, "f32", 17), cache, tables, lengths, q_start=np.arange(5) * n, max_q=n)


@pytest.mark.parametrize("dim,bits", [(64, 4), (64, 8), (128, 4), (128, 8), (256, 4), (256, 8)])
@pytest.mark.parametrize("dt", ["f16", "f32"])
@pytest.mark.parametrize("n", [1, 40])
def test_precision_over_a_whole_output(dim, bits, dt, n):
    # Norm over norm.  A score of normal queries and keys is a few units, a sum of
    # `dim` products the largest of which is about a fifth of the sum of their
    # sizes; the matrix instructions cut each product at 2^-22 of the largest with
    # it (24 bits, two of them lost to subnormal codes), of random sign, so that a
    # score is off by 2^-22 times a few units times the chain of up to 16: below
    # 2^-18, as is, to first order, an average of values under such weights.
    print("attention precision", dim, bits, dt, n, flush=True)
    heads, group, page, lengths = 2, 4, 32, [700, 64, 333]
    cache = make_cache(36, heads, page, dim, bits, dim + n)
    tables, _ = tables_of(36, lengths, page, np.random.default_rng(n))
    q = queries(3 * n, heads * group, dim, dt, n)
    got = check(q, cache, tables, lengths, q_start=np.arange(4) * n, max_q=n)
    ref, _, _ = O.attention(q, cache[0], tables, lengths, q_start=np.arange(4) * n, max_q=n)
    off = float(np.linalg.norm(got - ref) / np.linalg.norm(ref))
    print("  off by", off, flush=True)
    assert off <= 2.0 ** -18
