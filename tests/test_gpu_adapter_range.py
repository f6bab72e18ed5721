"""adapter_add where a row's low-rank values lie far apart, on the GPU, with a
bar that follows every rank by itself.

Bars, u = 2^-24, t = the float64 x At^T of a row, s its scale:
* t is a sum of floats in at most K / 4 + 32 steps, or exact where the inputs
  are whole numbers (times one power of two per rank) that stay below 2^24;
* s t B is a float32 sum of at most r + 8 steps after one rounding of s t;
* from 128 rows on with fp16 factors s t is a pair of fp16 values: off by 2^-22
  of itself, or 2^-49 of the largest of the row's ranks, whichever is more;
* scaling, unscaling and the sum with y round the result three times; results
  that pass into float32's subnormal numbers add 2^-149 a step:
    |out - ref| <= u (steps |x||A||B| + (r + 16 + 4) sum |s t||B| + 3 (|ref| + |y|))
                   + 2^-49 max|s t| sum|B| + 2^-149 (r + 16) (1 + sum|B|).
"""
import numpy as np
import pytest
import torch

from bit_gemm_block_amd import block as B

pytestmark = pytest.mark.gpu

DEV = "cuda:0"
U = 2.0 ** -24


def dev(a):
    return None if a is None else torch.from_numpy(np.ascontiguousarray(a)).to(DEV)


def host(t):
    torch.cuda.synchronize()
    return t.cpu().numpy()


def reference(y, x, At, Bt, index, scales, t_exact):
    """The float64 result and its bar."""
    M, N, (L, R, K) = x.shape[0], Bt.shape[1], At.shape
    ref = np.zeros((M, N)) if y is None else y.astype(np.float64)
    tol = np.zeros((M, N))
    for a in range(L):
        rows = np.nonzero(index == a)[0]
        if rows.size == 0:
            continue
        xa, A, Ba = x[rows].astype(np.float64), At[a].astype(np.float64), Bt[a].astype(np.float64)
        s = 1.0 if scales is None else float(scales[a])
        t = s * (xa @ A.T)
        ref[rows] += t @ Ba.T
        b = np.abs(Ba).T
        if not t_exact:
            tol[rows] += U * (K / 4 + 32) * abs(s) * ((np.abs(xa) @ np.abs(A).T) @ b)
        tol[rows] += U * (R + 20) * (np.abs(t) @ b)
        tol[rows] += 2.0 ** -49 * np.abs(t).max(axis=1)[:, None] * b.sum(axis=0) + 2.0 ** -149 * (R + 16) * (1 + b.sum(axis=0))
    return ref, tol + 3 * U * (np.abs(ref) + (0.0 if y is None else np.abs(y)))


FORMS = [(M, R, dt) for M in (20, 130, 1100, 2900) for R in (16, 64, 200) for dt in ("f16", "f32")]


@pytest.mark.parametrize("M,R,dt", FORMS)
@pytest.mark.parametrize("apart", [12, 21, 25])
def test_one_rank_far_above_the_others(M, R, dt, apart):
    # One rank of t is about 2^apart above the others, and half of the columns
    # of Bt do not take it: what they get is the others' alone.
    print("adapters, ranks apart", M, R, dt, apart, flush=True)
    K, N, L = 64, 48, 2
    rng = np.random.default_rng(M + R + apart)
    t = np.float16 if dt == "f16" else np.float32
    x = rng.integers(-2047, 2048, (M, K)).astype(t)
    At = rng.integers(-15, 16, (L, R, K)).astype(np.float32)
    At[:, :, 0] = 15                                     # no empty rank
    big = rng.integers(0, R, L)
    At *= 2.0 ** -(apart // 2 + 1)
    At[np.arange(L), big] *= 2.0 ** apart                # at most 15 * 2^12
    At = At.astype(t)
    Bt = rng.integers(-7, 8, (L, N, R)).astype(t)
    for a in range(L):
        Bt[a, ::2, big[a]] = 0
    index = rng.integers(-1, L, M).astype(np.int32)
    scales = np.array([1.0, -0.25], np.float32)
    ref, tol = reference(None, x, At, Bt, index, scales, True)
    got = host(B.adapter_add(None, *[dev(a) for a in (x, At, Bt, index)], scales=dev(scales)))
    assert np.all(np.abs(got - ref) <= tol), float(np.max(np.abs(got - ref) / np.maximum(tol, 1e-300)))


@pytest.mark.parametrize("M,R,dt", FORMS)
def test_neighbouring_rows_of_other_magnitudes(M, R, dt):
    # Rows of one tile at 1e-6, 1, 1e4 and 0, adapters with scales of 1e-30 and
    # 1e30: every row's power of two is its own.
    print("adapters, rows' magnitudes", M, R, dt, flush=True)
    K, N, L = 256, 48, 3
    rng = np.random.default_rng(M + R)
    t = np.float16 if dt == "f16" else np.float32
    x = (np.array([1e-6, 1.0, 1e4, 0.0])[np.arange(M) % 4][:, None] * rng.uniform(-1, 1, (M, K))).astype(t)
    At = rng.uniform(-0.05, 0.05, (L, R, K)).astype(t)
    Bt = rng.uniform(-0.2, 0.2, (L, N, R)).astype(t)
    index = rng.integers(-1, L, M).astype(np.int32)
    for scales in (None, np.array([1e-30, 1.0, 1e30], np.float32), np.array([0.0, -1e-12, 1e12], np.float32)):
        ref, tol = reference(None, x, At, Bt, index, scales, False)
        got = host(B.adapter_add(None, *[dev(a) for a in (x, At, Bt, index)], scales=dev(scales)))
        assert np.all(np.abs(got - ref) <= tol), float(np.max(np.abs(got - ref) / np.maximum(tol, 1e-300)))
        assert np.all(got[3::4] == 0)
