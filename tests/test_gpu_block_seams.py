"""norm_residual and gated_activation against the float64 reference, on the GPU.

Bars, u = 2^-24 (a row's sum is formed in at most 16 + 6 + 16 float32 steps):
* a norm: relative 64 u of the value plus 64 u of |r w| times the mean of |v|
  (the centring of a layer norm), carried along linearly; the result of the
  first step, h', has an error dh, which the second norm multiplies by |r w|
  and, through its statistics, adds relative to |x| by dh's root mean square
  over that of h';
* a rounding to fp16: 2^-11 of the value, at least 2^-25;
* activations: 16 u of the value (the library's exp and erfc, a quotient, two
  products) plus, for the exponent's rounding, 4 u |g| of the value.
"""
import numpy as np
import pytest
import torch

from bit_gemm_block_amd import block as B
from bit_gemm_block_amd import w4a4 as W
from oracle import block_oracle as O

pytestmark = pytest.mark.gpu

DEV = "cuda:0"
U = 2.0 ** -24
F16, F32 = torch.float16, torch.float32
NP = {"f16": np.float16, "f32": np.float32}


def dev(a):
    return None if a is None else torch.from_numpy(np.ascontiguousarray(a)).to(DEV)


def host(t):
    torch.cuda.synchronize()
    return t.cpu().numpy()


def rounding(v, dt):
    return np.maximum(2.0 ** -11 * np.abs(v), 2.0 ** -25) if dt == np.float16 else 2 * U * np.abs(v)


def norm_error(v, dv, kind, w, b, offset, eps):
    """Bound on the error of norm(v) where v is off by at most dv."""
    if kind == "none":
        return dv
    c = v - v.mean(axis=1, keepdims=True) if kind == "layer" else v
    r = 1.0 / np.sqrt(np.mean(c * c, axis=1, keepdims=True) + eps)
    f = np.abs(r * (1.0 if w is None else offset + w.astype(np.float64)))
    if kind == "layer":
        dv = dv + 64 * U * np.mean(np.abs(v), axis=1, keepdims=True) + np.mean(dv, axis=1, keepdims=True)
    rel = 64 * U + np.sqrt(np.mean(dv * dv, axis=1, keepdims=True)) * r
    x = np.abs(c) * f
    return f * dv + rel * x + 4 * U * (x + (0.0 if b is None else np.abs(b.astype(np.float64))))


def check(h, y, kw, h_dt, x_dt, got):
    o = dict(kw)
    ref_h, ref_x = O.norm_residual(h, y, **o)
    d = np.zeros(ref_h.shape)
    if y is not None:
        v = O.norm(y, o.get("post", "none"), o.get("post_w"), o.get("post_b"), o.get("offset", 0.0), o["eps"])
        d = norm_error(y.astype(np.float64), d, o.get("post", "none"), o.get("post_w"), o.get("post_b"),
                       o.get("offset", 0.0), o["eps"])
        if o.get("gate") is not None:
            g = o["gate"].astype(np.float64)[np.arange(y.shape[0]) // o["gate_rows"]]
            v, d = v * g, np.abs(g) * d
        rs = abs(o.get("rs", 1.0))
        d = rs * d + 4 * U * (rs * np.abs(v) + np.abs(ref_h))
    gh, gx = got
    if gh is not None:
        assert np.all(np.abs(gh - ref_h) <= d + rounding(ref_h, h_dt)), "h'"
    if gx is not None:
        d = norm_error(ref_h, d, o.get("pre", "none"), o.get("pre_w"), o.get("pre_b"), o.get("offset", 0.0),
                       o["eps"])
        assert np.all(np.abs(gx - ref_x) <= d + rounding(ref_x, x_dt)), "x"


def run(h, y, kw, x_dt="f16", **more):
    names = {"post": "post_norm", "post_w": "post_weight", "post_b": "post_bias", "rs": "residual_scale",
             "pre": "pre_norm", "pre_w": "pre_weight", "pre_b": "pre_bias", "offset": "weight_offset"}
    args = {names.get(k, k): dev(v) if isinstance(v, np.ndarray) else v for k, v in kw.items()}
    out = B.norm_residual(dev(h), dev(y), x_dtype=None if x_dt is None else F16 if x_dt == "f16" else F32,
                          **args, **more)
    return tuple(None if t is None else host(t) for t in out)


def inputs(M, C, h_dt, y_dt, p_dt, seed, gate_rows=0, bias=True):
    rng = np.random.default_rng(seed)
    h = rng.standard_normal((M, C))
    h[:, 5 % C] *= 60
    y = 3 * rng.standard_normal((M, C)) + 0.5
    p = {k: (rng.uniform(0.5, 1.5, C) if k[-1] == "w" else 0.3 * rng.standard_normal(C)).astype(NP[p_dt])
         for k in (("post_w", "pre_w", "post_b", "pre_b") if bias else ("post_w", "pre_w"))}
    if gate_rows:
        p["gate"] = rng.standard_normal((-(-M // gate_rows), C)).astype(np.float32)
        p["gate_rows"] = gate_rows
    return h.astype(NP[h_dt]), y.astype(NP[y_dt]), p


WIDTHS = [(3, 1), (5, 7), (9, 32), (6, 64), (7, 100), (4, 512), (5, 513), (3, 1000), (6, 2048), (5, 2049),
          (4, 2056), (3, 4096), (5, 4100), (2, 5003), (3, 8192), (2, 8200), (2, 14336), (2, 16384), (1, 16383),
          (300, 96), (70, 4096)]


@pytest.mark.parametrize("M,C", WIDTHS)
@pytest.mark.parametrize("kind", ["rms", "layer"])
def test_norm_residual_widths(M, C, kind):
    print("norms", M, C, kind, flush=True)
    h, y, p = inputs(M, C, "f32", "f32", "f16", M + C, gate_rows=3)
    kw = dict(p, post=kind, pre=kind, rs=0.7, eps=1e-5)
    check(h, y, kw, np.float32, np.float16, run(h, y, kw))
    check(h, y, kw, np.float32, np.float32, run(h, y, kw, "f32"))


@pytest.mark.parametrize("h_dt,y_dt,p_dt,x_dt", [(a, b, c, d) for a in ("f16", "f32") for b in ("f16", "f32")
                                                 for c in ("f16", "f32") for d in ("f16", "f32")])
@pytest.mark.parametrize("C", [200, 203, 4096])
def test_norm_residual_types(C, h_dt, y_dt, p_dt, x_dt):
    print("norm types", C, h_dt, y_dt, p_dt, x_dt, flush=True)
    h, y, p = inputs(6, C, h_dt, y_dt, p_dt, C, gate_rows=4)
    p["gate"] = p["gate"].astype(NP[p_dt])
    kw = dict(p, post="rms", pre="layer", rs=-1.5, eps=1e-6, offset=1.0)
    check(h, y, kw, NP[h_dt], NP[x_dt], run(h, y, kw, x_dt))


@pytest.mark.parametrize("C", [72, 1001, 4096])
def test_norm_residual_parts(C):
    # every part alone: only the norm, only the sum, no x, no h', no weights
    print("norm parts", C, flush=True)
    h, y, p = inputs(10, C, "f32", "f32", "f32", C, gate_rows=1)
    one = {"eps": 1e-6}
    for kind in ("rms", "layer"):
        got = run(h, None, {**one, "pre": kind, "pre_w": p["pre_w"]})
        assert got[0] is None
        check(h, None, {**one, "pre": kind, "pre_w": p["pre_w"]}, np.float32, np.float16, got)
        kw = {**one, "post": kind, "post_b": p["post_b"]}
        got = run(h, y, kw, None)
        assert got[1] is None
        check(h, y, kw, np.float32, np.float32, got)
        kw = {**one, "post": kind, "pre": kind}
        check(None, y, kw, np.float32, np.float16, run(None, y, kw))
    kw = {**one, "gate": p["gate"], "gate_rows": 1, "rs": 0.25}
    check(h, y, kw, np.float32, np.float32, run(h, y, kw, "f32"))
    got = run(h, y, {**one, "pre": "rms"}, want_h=False)
    assert got[0] is None
    check(h, y, {**one, "pre": "rms"}, np.float32, np.float16, got)
    got = run(h, y, one, "f32")
    assert np.array_equal(got[0], h + y) and np.array_equal(got[1], h + y)


def test_norm_residual_special_rows():
    print("norm special rows", flush=True)
    M, C = 9, 2048
    h, y, p = inputs(M, C, "f32", "f32", "f32", 3, bias=False)
    h[1], y[1] = 0, 0                                  # an empty row: 0 / sqrt(eps)
    h[2], y[2] = 5, 0                                  # equal values: no variance
    kw = dict(p, post="layer", pre="layer", eps=1e-5)
    clean = run(h, y, kw, "f32")
    check(h, y, kw, np.float32, np.float32, clean)
    assert np.all(clean[1][1] == 0) and np.all(clean[1][2] == 0)
    h2, y2 = h.copy(), y.copy()
    y2[4, 7], h2[5, 8], y2[6, 2047] = np.inf, np.nan, -np.inf
    got = run(h2, y2, kw, "f32")
    keep = [0, 1, 2, 3, 7, 8]
    assert np.array_equal(got[0][keep], clean[0][keep]) and np.array_equal(got[1][keep], clean[1][keep])
    assert np.isnan(got[1][4:7]).all()
    # a row of large values whose squares pass fp16 but not float32, and one
    # whose values are far below eps
    h[3], y[3] = 0, 1e15 * np.sign(y[3])
    h[4], y[4] = 0, 1e-20
    kw = dict(p, post="rms", pre="none", eps=1e-5)
    kw.pop("pre_w")
    check(h, y, kw, np.float32, np.float32, run(h, y, kw, "f32"))
    # a variance far below the mean
    h[:], y[:] = 0, 1000 + np.random.default_rng(0).standard_normal((M, C))
    kw = dict(post="layer", eps=1e-5)
    check(h, y, kw, np.float32, np.float32, run(h, y, kw, None))


@pytest.mark.parametrize("C", [64, 70, 4096, 9000])
def test_norm_residual_slices_and_in_place(C):
    print("norm slices", C, flush=True)
    M = 20
    h, y, p = inputs(M, C, "f16", "f32", "f32", 8, gate_rows=7)
    kw = dict(p, post="rms", pre="rms", rs=0.5, eps=1e-6)
    ref = run(h, y, kw)
    check(h, y, kw, np.float16, np.float16, ref)
    args = dict(post_norm="rms", pre_norm="rms", residual_scale=0.5, eps=1e-6, gate_rows=7,
                **{n: dev(p[k]) for n, k in (("post_weight", "post_w"), ("post_bias", "post_b"),
                                             ("pre_weight", "pre_w"), ("pre_bias", "pre_b"))})
    for first in (0, 8, 3):
        def slot(a, dt):
            w = torch.full((a.shape[0], C + 24), 9.0, dtype=dt, device=DEV)
            w[:, first:first + C] = dev(a)
            return w
        wh, wy, wg = slot(h, F16), slot(y, F32), slot(p["gate"], F32)
        wx = torch.full((M, C + 24), 9.0, dtype=F16, device=DEV)
        part = wh[:, first:first + C]
        B.norm_residual(part, wy[:, first:first + C], gate=wg[:, first:first + C], h_out=part,
                        x_out=wx[:, first:first + C], **args)
        wh, wx = host(wh), host(wx)
        check(h, y, kw, np.float16, np.float16, (wh[:, first:first + C], wx[:, first:first + C]))
        for w in (wh, wx):
            assert np.all(w[:, :first] == 9.0) and np.all(w[:, first + C:] == 9.0)


def test_norm_residual_empty_same_bits_and_stream():
    print("norm streams", flush=True)
    e = torch.zeros((0, 64), device=DEV)
    a, b = B.norm_residual(e, e, pre_norm="rms")
    assert tuple(a.shape) == (0, 64) and tuple(b.shape) == (0, 64)
    h, y, p = inputs(50, 4096, "f32", "f32", "f32", 1, bias=False)
    kw = dict(p, post="rms", pre="rms", eps=1e-6)
    first = run(h, y, kw)
    again = run(h, y, kw)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        other = run(h, y, kw)
    for g in (again, other):
        assert np.array_equal(g[0], first[0]) and np.array_equal(g[1], first[1])


def test_norm_residual_refusals():
    print("norm refusals", flush=True)
    h, y = torch.zeros((4, 64), device=DEV), torch.zeros((4, 64), device=DEV)
    w = torch.ones(64, device=DEV)
    for kw, err in [(dict(pre_norm="rms", pre_weight=w[:63]), ValueError),
                    (dict(pre_norm="rms", pre_weight=w, pre_bias=w.half()), TypeError),
                    (dict(pre_norm="rms", pre_weight=w.bfloat16()), W.W4A4Error),
                    (dict(gate=torch.ones((3, 64), device=DEV), gate_rows=1), ValueError),
                    (dict(gate=torch.ones((4, 64), device=DEV), gate_rows=0), ValueError),
                    (dict(pre_weight=w), W.W4A4Error), (dict(post_norm="rms", eps=-1.0), W.W4A4Error),
                    (dict(x_dtype=torch.bfloat16), TypeError), (dict(h_out=h.half()), TypeError),
                    (dict(pre_norm="rms", x_dtype=None), W.W4A4Error)]:
        with pytest.raises(err):
            B.norm_residual(h, y, **kw)
    with pytest.raises(ValueError):
        B.norm_residual(h, y[:3])
    with pytest.raises(TypeError):
        B.norm_residual(h, y.bfloat16())
    with pytest.raises(ValueError):
        B.norm_residual(h.t(), y.t())
    with pytest.raises(W.W4A4Error):
        B.norm_residual(torch.zeros((2, 16392), device=DEV), pre_norm="rms")


# --------------------------------------------------------------------------
# Gated activation
# --------------------------------------------------------------------------
def act_bound(g, ref, dt, u):
    u = 1.0 if u is None else np.abs(u.astype(np.float64))
    return (16 + 4 * np.abs(g.astype(np.float64))) * U * np.abs(ref) + 2.0 ** -140 * u + rounding(ref, dt)


def act_case(M, F, act, src, dst, up, seed):
    rng = np.random.default_rng(seed)
    g = (3 * rng.standard_normal((M, F))).astype(NP[src])
    u = (2 * rng.standard_normal((M, F))).astype(NP[src]) if up else None
    ref = O.activation(g, act) * (1.0 if u is None else u.astype(np.float64))
    return g, u, ref


@pytest.mark.parametrize("act", ["silu", "gelu", "gelu_tanh", "relu"])
@pytest.mark.parametrize("src", ["f16", "f32"])
@pytest.mark.parametrize("dst", ["f16", "f32"])
@pytest.mark.parametrize("M,F", [(1, 1), (3, 7), (8, 2048), (5, 2056), (33, 1407), (2, 14336), (100, 64)])
def test_gated_activation(M, F, act, src, dst):
    print("gated", M, F, act, src, dst, flush=True)
    for up in (True, False):
        g, u, ref = act_case(M, F, act, src, dst, up, M + F)
        out = torch.float16 if dst == "f16" else torch.float32
        got = host(B.gated_activation(dev(g), dev(u), act, out))
        assert np.all(np.abs(got - ref) <= act_bound(g, ref, NP[dst], u))
        for first in (0, 8, 1):                                  # halves of one projection, slices
            wide = torch.full((M, 2 * F + 16), 4.0, dtype=F16 if src == "f16" else F32, device=DEV)
            wide[:, first:first + F] = dev(g)
            if up:
                wide[:, first + F:first + 2 * F] = dev(u)
            o = torch.full((M, F + 9), 4.0, dtype=out, device=DEV)
            B.gated_activation(wide[:, first:first + F], wide[:, first + F:first + 2 * F] if up else None, act,
                               out=o[:, first:first + F])
            w = host(o)
            assert np.array_equal(w[:, first:first + F], got)
            assert np.all(w[:, :first] == 4.0) and np.all(w[:, first + F:] == 4.0)


@pytest.mark.parametrize("act", ["silu", "gelu", "gelu_tanh", "relu"])
def test_gated_activation_extremes(act):
    print("gated extremes", act, flush=True)
    g = np.array([[0.0, -0.0, 1e-30, -1e-30, 20, -20, 80, -80, 1e4, -1e4, 3e38, 700, -5.5, np.inf, np.nan]], np.float32)
    got = host(B.gated_activation(dev(g), None, act, F32))[0]
    with np.errstate(all="ignore"):
        ref = O.activation(g[:, :13], act)
    # cubes past float32 leave exp(-inf) = 0 and exp(inf) = inf: the limits themselves
    ref = np.where(g[:, :13] <= -1e4, 0.0, ref)
    ref = np.where(g[:, :13] == 3e38, g[:, :13], ref)
    assert np.all(np.abs(got[:13] - ref) <= act_bound(g[:, :13], ref, np.float32, None))
    assert got[13] == np.inf and np.isnan(got[14])
    up = host(B.gated_activation(dev(np.full((1, 3), 2.0, np.float32)),
                                 dev(np.array([[np.inf, np.nan, 1e6]], np.float32)), act))[0]
    assert up[0] == np.inf and np.isnan(up[1]) and up[2] == np.inf   # past fp16's range: infinity


def test_gated_activation_empty_refusals_and_stream():
    print("gated refusals", flush=True)
    z = torch.zeros((0, 8), device=DEV)
    assert tuple(B.gated_activation(z, z).shape) == (0, 8)
    assert tuple(B.gated_activation(z.t(), None).shape) == (8, 0)
    g = torch.zeros((4, 8), device=DEV)
    for args, kw, err in [((g, g.half()), {}, TypeError), ((g, g[:, :7]), {}, ValueError),
                          ((g.bfloat16(), None), {}, TypeError), ((g, None), {"act": "tanh"}, ValueError),
                          ((g, None), {"out_dtype": torch.bfloat16}, TypeError),
                          ((g, None), {"out": g[:3]}, ValueError), ((g.t(), None), {}, ValueError)]:
        with pytest.raises(err):
            B.gated_activation(*args, **kw)
    x = torch.randn((64, 4096), device=DEV)
    want = host(B.gated_activation(x, x))
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        got = B.gated_activation(x, x)
    s.synchronize()
    assert np.array_equal(got.cpu().numpy(), want)
