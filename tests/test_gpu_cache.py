"""cache_write and cache_read against the quantizer's definition, on the GPU:
codes, scales and values are equal to it, bit for bit."""
import numpy as np
import pytest
import torch

from bit_gemm_block_amd import decode as D
from bit_gemm_block_amd import w4a4 as W
from oracle import decode_oracle as O

pytestmark = pytest.mark.gpu

DEV = "cuda:0"
NP = {"f16": np.float16, "f32": np.float32}
TORCH = {"f16": torch.float16, "f32": torch.float32}


def dev(a):
    return torch.from_numpy(np.ascontiguousarray(a)).to(DEV)


def host(t):
    torch.cuda.synchronize()
    return t.cpu().numpy()


def values(T, heads, dim, dt, seed):
    """Rows of every size; borders of the quantizer among them."""
    rng = np.random.default_rng(seed)
    x = rng.standard_normal((T, heads, dim)) * 10.0 ** rng.uniform(-3, 3, (T, heads, 1))
    x[:, :, 3] *= 20
    if T > 2:
        x[1] = 0
        x[2] = rng.integers(-14, 15, (heads, dim)) * 0.5   # halves: codes on a border
        x[2, :, 0] = 7
    return np.clip(x, -60000, 60000).astype(NP[dt])


def filled(pages, heads, page, dim, bits, seed=0):
    """A cache with known rubbish in it."""
    g = torch.Generator(device=DEV).manual_seed(seed)
    c = D.KVCache.empty(pages, heads, page, dim, bits, DEV)
    for t in (c.k, c.v):
        t.copy_(torch.randint(0, 256, t.shape, generator=g, device=DEV, dtype=torch.uint8))
    for t in (c.k_scale, c.v_scale):
        t.copy_(torch.rand(t.shape, generator=g, device=DEV))
    return c


def parts(c):
    return [host(t) for t in (c.k, c.v, c.k_scale, c.v_scale)]


def written(before, c, k, v, slots, heads, dim, bits, page):
    """What the cache must hold after the write."""
    out = [a.copy() for a in before]
    for codes, scale, x in ((out[0], out[2], k), (out[1], out[3], v)):
        q, s = O.quantize(x.reshape(-1, heads, dim), bits)
        for t, slot in enumerate(slots):
            if 0 <= slot < codes.shape[0] * page:
                codes[slot // page, :, slot % page] = O.pack(q[t], bits)
                scale[slot // page, :, slot % page] = s[t]
    return out


@pytest.mark.parametrize("bits", [4, 8])
@pytest.mark.parametrize("dim", [64, 128, 256])
@pytest.mark.parametrize("T,heads,page,dt", [(1, 1, 16, "f32"), (3, 2, 32, "f16"), (37, 3, 16, "f32"), (100, 8, 64, "f16"),
                                             (513, 5, 128, "f32")])
def test_write_and_read(T, heads, page, dt, dim, bits):
    print("cache", T, heads, page, dt, dim, bits, flush=True)
    rng = np.random.default_rng(T)
    pages = -(-T // page) + 2
    slots = rng.permutation(pages * page)[:T].astype(np.int32)
    if T > 3:
        slots[3] = -1
    if T > 8:
        slots[[5, 8]] = pages * page, 2 ** 31 - 1
    k, v = values(T, heads, dim, dt, 1).reshape(T, -1), values(T, heads, dim, dt, 2).reshape(T, -1)
    c = filled(pages, heads, page, dim, bits)
    before = parts(c)
    D.cache_write(c, dev(k), dev(v), dev(slots))
    want = written(before, c, k, v, slots, heads, dim, bits, page)
    for got, ref in zip(parts(c), want):
        assert np.array_equal(got, ref)

    at = np.concatenate((slots, slots[:1], np.array([-7, pages * page], np.int32)))   # repeated and absent ones
    for out in ("f16", "f32"):
        rk, rv = D.cache_read(c, dev(at), out_dtype=TORCH[out])
        for got, codes, scale in ((host(rk), want[0], want[2]), (host(rv), want[1], want[3])):
            have = (at >= 0) & (at < pages * page)
            p = np.where(have, at, 0)
            x = O.unpack(codes[p // page, :, p % page], bits).astype(np.float32) * scale[p // page, :, p % page][..., None]
            x[~have] = 0
            with np.errstate(over="ignore"):
                ref = x.reshape(len(at), -1).astype(NP[out])
            assert got.dtype == NP[out] and np.array_equal(got, ref)


def test_strides_and_halves():
    # Columns of one projection, at odd addresses; only keys, only values; given outputs.
    print("cache strides", flush=True)
    T, heads, dim, page = 21, 2, 64, 16
    C = heads * dim
    for dt in ("f16", "f32"):
        k, v = values(T, heads, dim, dt, 3).reshape(T, C), values(T, heads, dim, dt, 4).reshape(T, C)
        both = torch.full((T, 2 * C + 5), float("nan"), dtype=TORCH[dt], device=DEV)
        both[:, 1:1 + C], both[:, 3 + C:3 + 2 * C] = dev(k), dev(v)
        slots = np.arange(T, dtype=np.int32) + 5
        a, b = filled(3, heads, page, dim, 4), filled(3, heads, page, dim, 4)
        D.cache_write(a, dev(k), dev(v), dev(slots))
        D.cache_write(b, both[:, 1:1 + C], both[:, 3 + C:3 + 2 * C], dev(slots))
        for x, y in zip(parts(a), parts(b)):
            assert np.array_equal(x, y)
        rk, rv = D.cache_read(a, dev(slots), out_dtype=TORCH[dt])
        buf = torch.full((T + 2, 2 * C + 7), 3.0, dtype=TORCH[dt], device=DEV)
        gk, none = D.cache_read(a, dev(slots), k=buf[1:-1, 1:1 + C], want_v=False)
        assert none is None and torch.equal(gk, rk) and bool((buf[:, 1 + C:] == 3).all())
        none, gv = D.cache_read(a, dev(slots), v=buf[1:-1, 3 + C:3 + 2 * C], want_k=False)
        assert none is None and torch.equal(gv, rv)
        buf[1:-1, 1:1 + C] = 3
        buf[1:-1, 3 + C:3 + 2 * C] = 3
        assert bool((buf == 3).all())


def test_far_values():
    # Subnormal rows (the scale is zero or has few bits), the largest numbers.
    print("cache far values", flush=True)
    x = np.zeros((6, 64), np.float32)
    x[0, :3] = 1e-45, -1e-45, 0
    x[1, :3] = 1.4e-44, -1e-45, 7e-45
    x[2, :2] = 3.4e38, -3.4e38
    x[3, :] = np.linspace(-1e-38, 1e-38, 64)
    x[4, 5] = -65504
    x[5, :] = -0.0
    for bits in (4, 8):
        c = filled(1, 1, 16, 64, bits)
        slots = np.arange(6, dtype=np.int32)
        before = parts(c)
        D.cache_write(c, dev(x), dev(-x), dev(slots))
        for got, ref in zip(parts(c), written(before, c, x, -x, slots, 1, 64, bits, 16)):
            assert np.array_equal(got, ref)


def test_long_offsets():
    # More than 2^32 bytes of codes: the last slot of the cache.
    print("cache long offsets", flush=True)
    page, heads, dim = 128, 16, 256
    pages = (1 << 32) // (page * heads * dim) + 3
    c = D.KVCache.empty(pages, heads, page, dim, 8, DEV)
    c.k[-1].zero_()
    c.k[0].zero_()
    k, v = values(2, heads, dim, "f32", 7).reshape(2, -1), values(2, heads, dim, "f32", 8).reshape(2, -1)
    slots = np.array([pages * page - 1, 3], np.int32)
    D.cache_write(c, dev(k), dev(v), dev(slots))
    rk, rv = D.cache_read(c, dev(slots), out_dtype=torch.float32)
    for got, x in ((host(rk), k), (host(rv), v)):
        q, s = O.quantize(x.reshape(2, heads, dim), 8)
        assert np.array_equal(got, (q.astype(np.float32) * s[..., None]).reshape(2, -1))
    assert bool((c.k[-1, :, :-1] == 0).all()) and bool((c.k[0, :, 4:] == 0).all()) and bool((c.k[0, :, :3] == 0).all())


def test_refused():
    c = filled(2, 2, 16, 64, 4)
    x, i = torch.zeros((4, 128), device=DEV), torch.zeros(4, dtype=torch.int32, device=DEV)
    for k, v, s in ((x[:, :64], x, i), (x, x[:3], i), (x, x, i[:3]), (x, x.cpu(), i), (x, x, i.cpu()), (x[0], x, i),
                    (x.t(), x, i)):
        with pytest.raises(ValueError):
            D.cache_write(c, k, v, s)
    for k, v, s in ((x.half(), x, i), (x.double(), x.double(), i), (x, x, i.long())):
        with pytest.raises(TypeError):
            D.cache_write(c, k, v, s)
    with pytest.raises(ValueError):
        D.cache_read(c, i[None])
    with pytest.raises(TypeError):
        D.cache_read(c, i, out_dtype=torch.float64)
    with pytest.raises(W.W4A4Error):
        D.cache_read(c, i, want_k=False, want_v=False)
    with pytest.raises(ValueError):
        D.cache_read(D.KVCache(c.k, c.v, c.k_scale[:1], c.v_scale), i)
    with pytest.raises(ValueError):
        D.cache_read(D.KVCache(c.k[:, :, ::2], c.v[:, :, ::2], c.k_scale[:, :, ::2], c.v_scale[:, :, ::2]), i)
    with pytest.raises(W.W4A4Error):
        D.cache_read(D.KVCache.empty(2, 2, 16, 32, 4, DEV), i)
    D.cache_write(c, x[:0], x[:0], i[:0])
    assert D.cache_read(c, i[:0])[0].shape == (0, 128)


def test_graph():
    print("cache graph", flush=True)
    T, heads, dim, page = 12, 2, 128, 16
    c = filled(4, heads, page, dim, 4)
    k = dev(values(T, heads, dim, "f32", 5).reshape(T, -1))
    v = dev(values(T, heads, dim, "f32", 6).reshape(T, -1))
    slots = torch.arange(T, dtype=torch.int32, device=DEV)
    ok, ov = torch.zeros((T, heads * dim), device=DEV), torch.zeros((T, heads * dim), device=DEV)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        D.cache_write(c, k, v, slots)
        D.cache_read(c, slots, k=ok, v=ov)
    for n in range(4):
        k.mul_(1.25)
        v.neg_()
        slots.add_(12).remainder_(64)
        slots[n] = -1
        g.replay()
        d = filled(4, heads, page, dim, 4, seed=n)
        D.cache_write(d, k, v, slots)
        wk, wv = D.cache_read(d, slots, out_dtype=torch.float32)
        torch.cuda.synchronize()
        assert torch.equal(ok, wk) and torch.equal(ov, wv), n
