"""qlinear_w4a16 against the float64 reference, on the GPU.

Bar: products are exact, and a result is a float32 sum in a chain of matrix
instructions (four to a tile of 128, a wave's tiles; three times as many for
float32 x), whose 32 products and addend each may be cut rather than rounded
(2 u each, u = 2^-24): with n tiles in a row at most 4 n * 3 chain links of a
few roundings, then the waves' and parts' sums and the scale.  Together below
(32 n + 64) u of the sum of absolute products; an fp16 result is rounded once
more (2^-11 of the value, at least 2^-25).
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
    return torch.from_numpy(np.ascontiguousarray(a)).to(DEV)


def host(t):
    torch.cuda.synchronize()
    return t.cpu().numpy()


def inputs(M, K, N, group, x_dt, s_dt, seed):
    rng = np.random.default_rng(seed)
    x = rng.standard_normal((M, K))
    x[:, 5 % K] *= 50
    q = rng.integers(-8, 8, (N, K))
    s = (rng.uniform(0.5, 1.5, (N, K // group) if group else (N,)) * K ** -0.5).astype(NP[s_dt])
    return x.astype(NP[x_dt]), O.pack(q, 4), s


def bar(size, ref, K, out):
    tol = (32 * (K // 128 + 1) + 64) * U * size
    return tol + np.maximum(2.0 ** -11 * np.abs(ref), 2.0 ** -25) if out == "f16" else tol


def check(x, wq, s, group, layout, out, **kw):
    ref, size = O.qlinear_w4a16(x, wq, s, group)
    w = dev(O.tile(wq) if layout == "tiled" else wq)
    got = host(D.qlinear_w4a16(dev(x), w, dev(s), group, w_layout=layout, out_dtype=TORCH[out], **kw))
    assert got.dtype == NP[out]
    e = np.abs(got - ref)
    assert np.all(e <= bar(size, ref, x.shape[1], out)), float(np.max(e / bar(size, ref, x.shape[1], out)))
    return got


ROWS = [1, 2, 3, 7, 8, 9, 15, 16, 17, 31, 32, 33, 48, 63, 64, 65, 129]


@pytest.mark.parametrize("M", ROWS)
@pytest.mark.parametrize("x_dt", ["f16", "f32"])
def test_rows(M, x_dt):
    print("w4a16 rows", M, x_dt, flush=True)
    for K, N, group in ((512, 200, 128), (2304, 48, 0)):
        x, wq, s = inputs(M, K, N, group, x_dt, "f16", M)
        check(x, wq, s, group, "tiled", "f32")


@pytest.mark.parametrize("K,group,layout", [(64, 0, "rowmajor"), (64, 64, "rowmajor"), (128, 0, "tiled"), (128, 128, "tiled"),
                                            (192, 64, "rowmajor"), (192, 192, "rowmajor"), (320, 64, "rowmajor"),
                                            (384, 192, "rowmajor"), (640, 320, "rowmajor"), (1088, 64, "rowmajor"),
                                            (1024, 256, "tiled"), (1536, 512, "rowmajor"), (4096, 128, "tiled"),
                                            (14336, 0, "tiled"), (14336, 128, "tiled"), (16384, 64, "rowmajor")])
@pytest.mark.parametrize("x_dt", ["f16", "f32"])
def test_channels_and_groups(K, group, layout, x_dt):
    print("w4a16 channels", K, group, layout, x_dt, flush=True)
    for M, N in ((1, 33), (20, 16)):
        x, wq, s = inputs(M, K, N, group, x_dt, "f32", K)
        check(x, wq, s, group, layout, "f32")


@pytest.mark.parametrize("N", [1, 15, 16, 17, 63, 64, 65, 127, 1007, 4096, 28672])
@pytest.mark.parametrize("out", ["f16", "f32"])
def test_outputs(N, out):
    print("w4a16 outputs", N, out, flush=True)
    for M, layout, group in ((1, "tiled", 128), (5, "rowmajor", 64), (40, "tiled", 0)):
        x, wq, s = inputs(M, 256, N, group, "f16", "f16", N)
        check(x, wq, s, group, layout, out)


def test_the_layers_weights():
    # The layer's own quantized weights, rotated by a Hadamard block: the product
    # with rotated rows is the float product within the weights' rounding.
    print("w4a16 layer's weights", flush=True)
    rng = np.random.default_rng(5)
    w, x = rng.standard_normal((96, 512)).astype(np.float32), rng.standard_normal((3, 512)).astype(np.float32)
    rot = W.hadamard_rotate(dev(x), 128)
    for layout, group in (("tiled", 0), ("tiled", 128), ("rowmajor", 64)):
        wq, ws = W.quantize_weight_int4(dev(w), 128, group, torch.float16, layout=layout)
        got = host(D.qlinear_w4a16(rot, wq, ws, group, w_layout=layout))
        plain = wq if layout == "rowmajor" else W.quantize_weight_int4(dev(w), 128, group, torch.float16)[0]
        ref, size = O.qlinear_w4a16(host(rot), host(plain), host(ws), group)
        assert np.all(np.abs(got - ref) <= bar(size, ref, 512, "f32"))
        # half a step of a weight is max|w| / 14, some 3.3 / 14 of the deviation, uniform: 0.14 of the product
        exact = x.astype(np.float64) @ w.astype(np.float64).T
        assert np.linalg.norm(got - exact) <= 0.25 * np.linalg.norm(exact)


@pytest.mark.parametrize("x_dt", ["f16", "f32"])
def test_strides_and_neighbours(x_dt):
    print("w4a16 strides", x_dt, flush=True)
    x, wq, s = inputs(19, 256, 37, 128, x_dt, "f16", 3)
    wide = torch.full((19, 256 + 64), float("nan"), dtype=TORCH[x_dt], device=DEV)
    wide[:, 32:288] = dev(x)
    w, sc = dev(O.tile(wq)), dev(s)
    want = D.qlinear_w4a16(dev(x), w, sc, 128)
    for out_dt in (torch.float32, torch.float16):
        buf = torch.full((21, 50), 7.0, dtype=out_dt, device=DEV)
        got = D.qlinear_w4a16(wide[:, 32:288], w, sc, 128, out=buf[1:20, 5:42])
        assert got.data_ptr() == buf[1:20, 5:42].data_ptr()
        assert torch.equal(got, want.to(out_dt))
        buf[1:20, 5:42] = 7.0
        assert bool((buf == 7.0).all())
    assert torch.equal(D.qlinear_w4a16(wide[4:5, 32:288], w, sc, 128).isnan(), torch.zeros((1, 37), device=DEV, dtype=torch.bool))


@pytest.mark.parametrize("x_dt", ["f16", "f32"])
def test_far_values(x_dt):
    # The type's range; an infinity or a NaN stays in its row.
    print("w4a16 far values", x_dt, flush=True)
    x, wq, s = inputs(18, 384, 40, 128, "f32", "f32", 9)
    big = 60000.0 if x_dt == "f16" else 1e33
    small = 2.0 ** -20 if x_dt == "f16" else 1e-30   # fp16: subnormal numbers
    x = np.clip(x, -4, 4)
    x[2] *= big / 4
    x[3] *= small
    x[4, ::2] = 0
    x = x.astype(NP[x_dt])
    ref = check(x, wq, s, 128, "tiled", "f32")
    x[7, 100], x[8, 5], x[9, 9] = np.inf, np.nan, -np.inf
    got = host(D.qlinear_w4a16(dev(x), dev(O.tile(wq)), dev(s), 128))
    assert np.all(~np.isfinite(got[7:10]))
    keep = [m for m in range(18) if m not in (7, 8, 9)]
    assert np.array_equal(got[keep], ref[keep])


def test_rows_do_not_depend_on_each_other():
    print("w4a16 rows alone", flush=True)
    x, wq, s = inputs(40, 1024, 70, 128, "f16", "f16", 11)
    w, sc = dev(O.tile(wq)), dev(s)
    want = D.qlinear_w4a16(dev(x), w, sc, 128)
    x[1:] = x[:1]
    got = D.qlinear_w4a16(dev(x), w, sc, 128)
    assert torch.equal(got[0], want[0]) and torch.equal(got, got[:1].expand_as(got))
    assert torch.equal(D.qlinear_w4a16(dev(x), w, sc, 128), got)


def test_empty_and_refused():
    x, wq, s = inputs(4, 256, 32, 128, "f16", "f16", 1)
    w, sc, xt = dev(O.tile(wq)), dev(s), dev(x)
    assert D.qlinear_w4a16(xt[:0], w, sc, 128).shape == (0, 32)
    assert D.qlinear_w4a16(xt, w[:0], sc[:0], 128).shape == (4, 0)
    for args in ((xt[0], w, sc, 128), (xt, w[:16], sc, 128), (xt, w, sc[:, 0], 128), (xt, w, sc, 0), (xt, w, sc, 100),
                 (xt, w, sc[:, :1].contiguous(), 128), (xt.t(), w, sc, 128), (xt.cpu(), w, sc, 128), (xt, w.cpu(), sc, 128)):
        with pytest.raises(ValueError):
            D.qlinear_w4a16(*args)
    with pytest.raises(ValueError):
        D.qlinear_w4a16(xt, w, sc, 128, out=torch.empty((4, 31), device=DEV))
    for args in ((xt.double(), w, sc, 128), (xt, w.int(), sc, 128), (xt, w, sc.double(), 128)):
        with pytest.raises(TypeError):
            D.qlinear_w4a16(*args)
    with pytest.raises(W.W4A4Error):
        D.qlinear_w4a16(xt, w, sc.repeat_interleave(2, 1).contiguous(), 64)
    with pytest.raises(W.W4A4Error):
        D.qlinear_w4a16(dev(np.zeros((2, 260), np.float16))[:, 2:258], w, sc, 128)


def test_graph_and_streams():
    print("w4a16 graph", flush=True)
    x, wq, s = inputs(24, 2048, 512, 128, "f16", "f16", 21)
    w, sc, xt = dev(O.tile(wq)), dev(s), dev(x)
    out = torch.zeros((24, 512), device=DEV)
    ws = D.qlinear_w4a16_workspace(24, 512, 2048, DEV)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        got = D.qlinear_w4a16(xt, w, sc, 128)
    side.synchronize()
    assert torch.equal(got, D.qlinear_w4a16(xt, w, sc, 128))
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        D.qlinear_w4a16(xt, w, sc, 128, out=out, workspace=ws)
    for k in range(4):
        xt.mul_(0.75)
        want = D.qlinear_w4a16(xt, w, sc, 128)
        out.zero_()
        g.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, want), k


@pytest.mark.parametrize("K,group", [(64, 64), (192, 64), (192, 192), (1088, 64)])
@pytest.mark.parametrize("x_dt", ["f16", "f32"])
def test_nothing_behind_the_scales_counts(K, group, x_dt):
    # K ends in the middle of a tile: that tile's second half has no scale.
    print("w4a16 scales' end", K, group, x_dt, flush=True)
    for M in (1, 5, 20, 40):
        x, wq, s = inputs(M, K, 33, group, x_dt, "f32", K + M)
        room = torch.full((s.size + 64,), float("nan"), device=DEV)
        room[:s.size] = dev(s).reshape(-1)
        ref, size = O.qlinear_w4a16(x, wq, s, group)
        got = host(D.qlinear_w4a16(dev(x), dev(wq), room[:s.size].view(s.shape), group, w_layout="rowmajor"))
        assert np.all(np.abs(got - ref) <= bar(size, ref, K, "f32"))
