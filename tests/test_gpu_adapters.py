"""adapter_add against the float64 reference, on the GPU.

Bars:
* small whole numbers: every sum is exact in float32 (and in the fp16 pair), so
  the output equals the reference bit for bit;
* random values, u = 2^-24: t is a float32 sum in at most K / 4 + 32 steps (the
  matrix instruction takes four channels or more a step), carried through
  |B|; with fp16 factors t keeps at least 21 bits of the row's largest |t|;
  t B is a float32 sum of at most r + 8 steps; scaling, unscaling and the sum
  with y round the result three times:
    |out - ref| <= u ((K / 4 + 32) |x||A||B| + (8 + r + 8) max|t| sum|B| + 3 (|ref| + |y|)).
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


def dev(a):
    return torch.from_numpy(np.ascontiguousarray(a)).to(DEV)


def host(t):
    torch.cuda.synchronize()
    return t.cpu().numpy()


def runs(rng, M, L, none=0.15):
    """An adapter (or -1) for every row, in runs of random length."""
    out = np.empty(M, np.int32)
    m = 0
    while m < M:
        n = int(rng.integers(1, 40))
        out[m:m + n] = -1 if rng.random() < none else rng.integers(0, L)
        m += n
    return out


SHAPES = [  # M, K, N, adapters, rank, dtype, order
    (1, 64, 1, 1, 8, "f16", "runs"), (1, 4096, 4096, 3, 16, "f16", "runs"),
    (2, 14336, 67, 2, 24, "f16", "mixed"), (5, 64, 3, 2, 1, "f32", "mixed"),
    (8, 4096, 300, 8, 64, "f16", "mixed"), (15, 128, 255, 15, 8, "f16", "mixed"),
    (16, 320, 256, 16, 40, "f16", "mixed"), (17, 192, 257, 3, 32, "f16", "runs"),
    (33, 1088, 1007, 5, 20, "f32", "mixed"), (40, 16384, 64, 2, 3, "f32", "runs"),
    (64, 512, 260, 64, 128, "f16", "mixed"), (100, 448, 130, 7, 256, "f16", "runs"),
    (70, 256, 96, 4, 256, "f32", "runs"), (300, 64, 1030, 9, 17, "f32", "mixed"),
    (257, 576, 515, 6, 48, "f16", "runs"), (1009, 128, 70, 4, 16, "f16", "mixed"),
    (1040, 640, 260, 5, 72, "f16", "runs"), (2100, 192, 129, 3, 8, "f32", "runs"),
    (1500, 1024, 516, 6, 32, "f16", "runs"), (2049, 64, 33, 2, 200, "f16", "mixed"),
    (2900, 320, 70, 3, 32, "f16", "runs"), (2833, 192, 65, 5, 40, "f16", "mixed"),
    (2848, 64, 33, 2, 24, "f32", "runs"), (3001, 128, 40, 4, 64, "f32", "mixed"),
    (130, 2112, 36, 2, 128, "f16", "runs"), (128, 64, 300, 40, 16, "f32", "mixed"),
]


def case(M, K, N, L, R, dt, order, seed, whole):
    rng = np.random.default_rng(seed)
    t = np.float16 if dt == "f16" else np.float32
    if whole:
        x = rng.integers(-2, 3, (M, K)).astype(t)
        At = rng.integers(-1, 2, (L, R, K)).astype(t)
        Bt = rng.integers(-3, 4, (L, N, R)).astype(t)
        y = rng.integers(-100, 101, (M, N)).astype(np.float32)
        scales = (2.0 ** rng.integers(-1, 3, L)).astype(np.float32)
    else:
        x = rng.standard_normal((M, K)).astype(np.float32)
        x[:, 7 % K] *= 100
        x[0] *= 30
        x = x.astype(t)
        At = (0.05 * rng.standard_normal((L, R, K))).astype(t)
        Bt = (0.2 * rng.standard_normal((L, N, R))).astype(t)
        y = rng.standard_normal((M, N)).astype(np.float32)
        scales = rng.uniform(0.2, 2.0, L).astype(np.float32)
    index = runs(rng, M, L)
    if order == "mixed":
        index = rng.permutation(np.where(rng.random(M) < 0.1, -1, rng.integers(0, L, M))).astype(np.int32)
    ranks = rng.integers(0, R + 1, L).astype(np.int32)
    ranks[rng.integers(0, L)] = R
    return y, x, At, Bt, index, ranks, scales


@pytest.mark.parametrize("M,K,N,L,R,dt,order", SHAPES)
def test_whole_numbers_exact(M, K, N, L, R, dt, order):
    print("adapters, whole numbers", M, K, N, L, R, dt, order, flush=True)
    c = case(M, K, N, L, R, dt, order, M + K + N, True)
    got = host(B.adapter_add(*[dev(a) for a in c]))
    assert np.array_equal(got, O.adapter_add(*c).astype(np.float32))
    got = host(B.adapter_add(dev(c[0]), *[dev(a) for a in c[1:5]]))      # no ranks, no scales
    assert np.array_equal(got, O.adapter_add(*c[:5]).astype(np.float32))


def bound(c):
    R, K = c[2].shape[1:]
    first, second = O.adapter_add_scale(*c)
    ref = O.adapter_add(*c)
    y = 0.0 if c[0] is None else np.abs(c[0])
    return ref, U * ((K / 4 + 32) * first + (16 + R) * second + 3 * (np.abs(ref) + y))


@pytest.mark.parametrize("M,K,N,L,R,dt,order", SHAPES)
def test_random_values(M, K, N, L, R, dt, order):
    print("adapters, random", M, K, N, L, R, dt, order, flush=True)
    c = case(M, K, N, L, R, dt, order, M + K + N + 1, False)
    ref, tol = bound(c)
    got = host(B.adapter_add(*[dev(a) for a in c]))
    assert np.all(np.abs(got - ref) <= tol), float(np.max(np.abs(got - ref) / tol))


@pytest.mark.parametrize("xmag,amag,bmag", [(6e4, 0.5, 0.1), (6e4, 6e4, 1e-3), (1e-3, 1e-3, 1.0),
                                            (6e-8, 6e-8, 6e4)])
def test_magnitudes_of_t_outside_fp16(xmag, amag, bmag):
    # t up to 1e12 and down to 1e-14: the pair follows the row.
    print("adapters, magnitudes", xmag, amag, bmag, flush=True)
    rng = np.random.default_rng(5)
    M, K, N, L, R = 20, 256, 48, 2, 16
    x = (xmag * rng.uniform(-1, 1, (M, K))).astype(np.float16)
    At = (amag * rng.uniform(-1, 1, (L, R, K))).astype(np.float16)
    Bt = (bmag * rng.uniform(-1, 1, (L, N, R))).astype(np.float16)
    c = (None, x, At, Bt, (np.arange(M) % L).astype(np.int32))
    ref, tol = bound(c)
    got = host(B.adapter_add(None, *[dev(a) for a in c[1:]]))
    assert np.all(np.abs(got - ref) <= tol)


@pytest.mark.parametrize("dt", ["f16", "f32"])
@pytest.mark.parametrize("M", [24, 1100])
def test_values_that_must_not_matter(M, dt):
    # NaN and infinities in rows past the ranks, in unused adapters, in other
    # rows of x and y, and in the workspace leave every other row's bits alone.
    print("adapters, garbage", M, dt, flush=True)
    K, N, L, R = 192, 100, 6, 24
    y, x, At, Bt, index, ranks, scales = case(M, K, N, L, R, dt, "mixed", 11, False)
    index[index == 4] = 3                                        # adapter 4: unused
    ranks[:] = [5, 24, 17, 8, 24, 0]
    clean = host(B.adapter_add(*[dev(a) for a in (y, x, At, Bt, index, ranks, scales)]))
    x2, y2, At2, Bt2 = x.copy(), y.copy(), At.copy(), Bt.copy()
    for a in range(L):
        At2[a, ranks[a]:] = np.nan
        Bt2[a][:, ranks[a]:] = np.inf
    At2[4], Bt2[4], At2[5], Bt2[5] = np.inf, np.nan, np.nan, np.nan
    x2[index < 0] = np.nan                                       # rows without an adapter
    bad = int(np.nonzero(index == 1)[0][0])
    x2[bad, 3] = np.inf
    y2[int(np.nonzero(index == 3)[0][0]), 7] = np.nan
    ws = torch.full((B.adapter_workspace_size(M, K, R) // 4,), float("nan"), device=DEV)
    got = host(B.adapter_add(*[dev(a) for a in (y2, x2, At2, Bt2, index, ranks, scales)], workspace=ws))
    keep = np.ones((M, N), bool)
    keep[bad] = False
    keep[np.isnan(y2)] = False
    assert np.array_equal(got[keep], clean[keep])
    assert not np.isfinite(got[bad]).any()
    assert np.isnan(got[np.isnan(y2)]).all()


def test_one_adapter_with_infinite_factors_keeps_to_its_rows():
    print("adapters, infinite factors", flush=True)
    y, x, At, Bt, index, ranks, scales = case(40, 128, 72, 3, 16, "f16", "mixed", 3, False)
    clean = host(B.adapter_add(*[dev(a) for a in (y, x, At, Bt, index, None, None) if a is not None]))
    Bt[1], At[1, 2] = np.inf, np.nan
    got = host(B.adapter_add(*[dev(a) for a in (y, x, At, Bt, index)]))
    assert np.array_equal(got[index != 1], clean[index != 1])
    assert not np.isfinite(got[index == 1]).any()


@pytest.mark.parametrize("M", [7, 1030])
def test_index_and_ranks_out_of_range(M):
    print("adapters, out of range", M, flush=True)
    y, x, At, Bt, index, ranks, scales = case(M, 128, 60, 4, 16, "f16", "mixed", 9, True)
    index[:] = np.array([-1, 4, 2 ** 31 - 1, -2 ** 31, 0, 1, 3], np.int32)[np.arange(M) % 7]
    ranks[:] = [-5, 17, 2 ** 31 - 1, 16]
    c = (y, x, At, Bt, index, ranks, scales)
    got = host(B.adapter_add(*[dev(a) for a in c]))
    assert np.array_equal(got, O.adapter_add(*c).astype(np.float32))
    index[:] = -1                                                # nothing for any row
    got = host(B.adapter_add(*[dev(a) for a in c]))
    assert np.array_equal(got, y)
    none = torch.zeros((0, 16, 128), dtype=F16, device=DEV)      # no adapter loaded at all
    got = host(B.adapter_add(dev(y), dev(x), none, torch.zeros((0, 60, 16), dtype=F16, device=DEV),
                             dev(index)))
    assert np.array_equal(got, y)


@pytest.mark.parametrize("M,dt", [(5, "f16"), (50, "f32"), (1200, "f16")])
def test_slices_in_place_and_without_y(M, dt):
    print("adapters, slices", M, dt, flush=True)
    K, N, L, R = 192, 132, 4, 16
    c = case(M, K, N, L, R, dt, "runs", 21, True)
    y, x, At, Bt, index, ranks, scales = c
    ref = O.adapter_add(*c).astype(np.float32)
    rest = [dev(a) for a in (At, Bt, index, ranks, scales)]
    wide_x = torch.zeros((M, K + 64), dtype=F16 if dt == "f16" else F32, device=DEV)
    wide_x[:, 32:32 + K] = dev(x)
    for first in (0, 4, 3):                                      # aligned and odd columns
        wide = torch.full((M, N + 9), 5.0, device=DEV)
        part = wide[:, first:first + N]
        part.copy_(dev(y))
        got = B.adapter_add(part, wide_x[:, 32:32 + K], *rest, out=part)
        assert got is part
        w = host(wide)
        assert np.array_equal(w[:, first:first + N], ref)
        assert np.all(w[:, :first] == 5.0) and np.all(w[:, first + N:] == 5.0)
    out = torch.full((M, N + 4), 5.0, device=DEV)
    B.adapter_add(dev(y), dev(x), *rest, out=out[:, :N])         # y and out of different distances
    assert np.array_equal(host(out)[:, :N], ref) and bool((out[:, N:] == 5.0).all())
    got = host(B.adapter_add(None, dev(x), *rest))
    assert np.array_equal(got, O.adapter_add(None, *c[1:]).astype(np.float32))
    same = dev(y)
    B.adapter_add(same, dev(x), *rest, out=same)
    assert np.array_equal(host(same), ref)


def test_empty_sizes():
    print("adapters, empty", flush=True)
    At, Bt = torch.zeros((2, 8, 64), dtype=F16, device=DEV), torch.zeros((2, 10, 8), dtype=F16, device=DEV)
    ix = torch.zeros((0,), dtype=torch.int32, device=DEV)
    out = B.adapter_add(None, torch.zeros((0, 64), dtype=F16, device=DEV), At, Bt, ix)
    assert tuple(out.shape) == (0, 10)
    out = B.adapter_add(None, torch.zeros((3, 64), dtype=F16, device=DEV), At, Bt[:, :0],
                        torch.zeros((3,), dtype=torch.int32, device=DEV))
    assert tuple(out.shape) == (3, 0)


def test_same_bits_again_and_on_another_stream():
    print("adapters, streams", flush=True)
    c = [dev(a) for a in case(130, 4096, 600, 12, 32, "f16", "mixed", 2, False)]
    first = host(B.adapter_add(*c))
    assert np.array_equal(host(B.adapter_add(*c)), first)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        got = B.adapter_add(*c)
    s.synchronize()
    assert np.array_equal(got.cpu().numpy(), first)


def test_graph_replays():
    print("adapters, graph", flush=True)
    c = [dev(a) for a in case(9, 1024, 256, 4, 16, "f16", "mixed", 4, False)]
    out = torch.zeros((9, 256), device=DEV)
    ws = B.adapter_workspace(9, 1024, 16, DEV)
    B.adapter_add(*c, out=out, workspace=ws)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        B.adapter_add(*c, out=out, workspace=ws)
    for k in range(3):
        c[0].add_(1.0)
        want = host(B.adapter_add(*c))
        out.zero_()
        g.replay()
        assert np.array_equal(host(out), want), k


def test_offsets_past_32_bits():
    # out holds 2^31 + elements; the rows on both sides of 2^31 and the last.
    M, K, N, L, R = 75000, 64, 28700, 3, 8
    print("adapters, offsets", M, N, flush=True)
    rng = np.random.default_rng(1)
    x = rng.integers(-2, 3, (M, K)).astype(np.float16)
    At = rng.integers(-1, 2, (L, R, K)).astype(np.float16)
    Bt = rng.integers(-3, 4, (L, N, R)).astype(np.float16)
    index = (np.arange(M) // 1000 % (L + 1) - 1).astype(np.int32)
    out = B.adapter_add(None, dev(x), dev(At), dev(Bt), dev(index))
    at = np.array([0, 1, 999, 74823, 74824, 74825, 74826, 74827, 74828, 74990, 74999])
    got = host(out[torch.from_numpy(at).to(DEV)])
    assert np.array_equal(got, O.adapter_add(None, x[at], At, Bt, index[at]).astype(np.float32))


def test_binding_refusals():
    print("adapters, refusals", flush=True)
    M, K, N, L, R = 4, 128, 32, 2, 16
    good = dict(y=torch.zeros((M, N), device=DEV), x=torch.zeros((M, K), dtype=F16, device=DEV),
                At=torch.zeros((L, R, K), dtype=F16, device=DEV),
                Bt=torch.zeros((L, N, R), dtype=F16, device=DEV),
                index=torch.zeros(M, dtype=torch.int32, device=DEV))
    B.adapter_add(**good)
    for name, value, err in [
            ("At", good["At"].float(), TypeError), ("Bt", good["Bt"].float(), TypeError),
            ("x", good["x"].bfloat16(), TypeError), ("index", good["index"].long(), TypeError),
            ("y", good["y"].half(), TypeError), ("ranks", torch.zeros(L, device=DEV), TypeError),
            ("scales", torch.zeros(L, dtype=F16, device=DEV), TypeError),
            ("x", torch.zeros((M, 64), dtype=F16, device=DEV), ValueError),
            ("index", good["index"][:3], ValueError), ("y", good["y"][:, :31], ValueError),
            ("Bt", torch.zeros((L, N, 8), dtype=F16, device=DEV), ValueError),
            ("ranks", torch.zeros(3, dtype=torch.int32, device=DEV), ValueError),
            ("y", torch.zeros((N, M), device=DEV).t(), ValueError),
            ("out", torch.zeros((1, N), device=DEV).expand(M, N), ValueError),
            ("index", good["index"].cpu(), ValueError), ("At", good["At"].cpu(), ValueError),
            ("workspace", torch.zeros(8, dtype=torch.uint8, device=DEV), W.W4A4Error)]:
        with pytest.raises(err):
            B.adapter_add(**{**good, name: value})
    with pytest.raises(W.W4A4Error) as e:                        # fp16 rank not a multiple of 8
        B.adapter_add(good["y"], good["x"], good["At"][:, :12].contiguous(),
                      good["Bt"][:, :, :12].contiguous(), good["index"])
    assert e.value.status == W.ERR_UNSUPPORTED
    with pytest.raises(W.W4A4Error) as e:                        # rows of x off 16 bytes
        B.adapter_add(good["y"], torch.zeros((M, K + 4), dtype=F16, device=DEV)[:, :K], good["At"],
                      good["Bt"], good["index"])
    assert e.value.status == W.ERR_MISALIGNED


PARTS = [  # M, K, N, adapters, rank, dtype, order: few rows, K taken whole or in parts
    (3, 8192, 70, 1, 8, "f16", "runs"), (4, 8128, 70, 1, 16, "f16", "runs"),
    (4, 8192, 33, 1, 24, "f16", "runs"), (16, 16384, 1030, 2, 64, "f16", "runs"),
    (16, 960, 2060, 1, 8, "f16", "runs"), (16, 1024, 2060, 1, 8, "f16", "runs"),
    (31, 8192, 515, 40, 40, "f16", "mixed"), (100, 8256, 300, 4, 256, "f16", "runs"),
    (127, 9664, 130, 3, 128, "f16", "mixed"), (4, 448, 5, 1, 3, "f32", "runs"),
    (4, 512, 1100, 1, 12, "f32", "runs"), (19, 4032, 65, 2, 33, "f32", "runs"),
    (19, 4096, 65, 5, 33, "f32", "mixed"), (127, 4160, 40, 3, 200, "f32", "runs"),
]


@pytest.mark.parametrize("M,K,N,L,R,dt,order", PARTS)
def test_few_rows_with_long_rows(M, K, N, L, R, dt, order):
    print("adapters, parts of K", M, K, N, L, R, dt, order, flush=True)
    c = case(M, K, N, L, R, dt, order, M + K + N + 2, True)
    assert np.array_equal(host(B.adapter_add(*[dev(a) for a in c])), O.adapter_add(*c).astype(np.float32))
    c = case(M, K, N, L, R, dt, order, M + K + N + 3, False)
    ref, tol = bound(c)
    ws = B.adapter_workspace(M, K, R, DEV)
    ws.view(torch.float32).fill_(float("nan"))           # what no part writes is not read
    got = host(B.adapter_add(*[dev(a) for a in c], workspace=ws))
    assert np.all(np.abs(got - ref) <= tol), float(np.max(np.abs(got - ref) / tol))


def test_a_workspace_for_more_rows_serves_fewer():
    for R in (8, 24, 256):
        sizes = [B.adapter_workspace_size(M, 16384, R) for M in (1, 3, 64, 127, 128, 400, 600, 4096)]
        assert sizes == sorted(sizes)


MANY = [  # M, K, N, adapters, rank, dtype, order: many rows at every width of the ranks
    (128, 2112, 257, 2, 16, "f16", "runs"), (300, 64, 1000, 9, 8, "f16", "mixed"),
    (300, 576, 67, 3, 24, "f16", "mixed"), (300, 128, 1031, 4, 64, "f16", "mixed"),
    (300, 2112, 36, 2, 128, "f16", "runs"), (270, 192, 300, 5, 104, "f16", "mixed"),
    (257, 1088, 130, 3, 256, "f16", "runs"), (300, 64, 515, 40, 12, "f32", "mixed"),
    (300, 576, 261, 3, 13, "f32", "runs"), (140, 192, 1031, 4, 52, "f32", "mixed"),
    (300, 320, 65, 2, 128, "f32", "runs"), (130, 128, 300, 3, 253, "f32", "mixed"),
    (1500, 128, 2100, 4, 16, "f16", "mixed"), (1500, 64, 2100, 4, 40, "f16", "runs"),
]


@pytest.mark.parametrize("M,K,N,L,R,dt,order", MANY)
def test_many_rows_at_every_width(M, K, N, L, R, dt, order):
    print("adapters, many rows", M, K, N, L, R, dt, order, flush=True)
    c = case(M, K, N, L, R, dt, order, M + K + N + 4, True)
    assert np.array_equal(host(B.adapter_add(*[dev(a) for a in c])), O.adapter_add(*c).astype(np.float32))
    c = case(M, K, N, L, R, dt, order, M + K + N + 5, False)
    ref, tol = bound(c)
    got = host(B.adapter_add(*[dev(a) for a in c]))
    assert np.all(np.abs(got - ref) <= tol), float(np.max(np.abs(got - ref) / tol))
