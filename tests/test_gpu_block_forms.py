"""Forms of the operators beside the layer that ordinary sizes do not reach, on
the GPU: a single row cut from a wider matrix, more adapters than a wave has
lanes, more rows than a launch has workgroups, and more than 2^31 elements.
Bars as in the operators' own tests."""
import numpy as np
import pytest
import torch

import test_gpu_block_seams as seams
from bit_gemm_block_amd import block as B
from bit_gemm_block_amd import mlp as MLP
from oracle import block_oracle as O

pytestmark = pytest.mark.gpu

DEV = "cuda:0"
F16, F32 = torch.float16, torch.float32


def dev(a):
    return None if a is None else torch.from_numpy(np.ascontiguousarray(a)).to(DEV)


def host(t):
    torch.cuda.synchronize()
    return t.cpu().numpy()


def whole_numbers(M, K, N, L, R, dt, seed, index=None):
    """Inputs whose sums are exact."""
    rng = np.random.default_rng(seed)
    t = np.float16 if dt == "f16" else np.float32
    return (rng.integers(-100, 101, (M, N)).astype(np.float32), rng.integers(-2, 3, (M, K)).astype(t),
            rng.integers(-1, 2, (L, R, K)).astype(t), rng.integers(-3, 4, (L, N, R)).astype(t),
            rng.integers(-1, L, M).astype(np.int32) if index is None else index,
            rng.integers(0, R + 1, L).astype(np.int32), (2.0 ** rng.integers(-1, 3, L)).astype(np.float32))


@pytest.mark.parametrize("dt", ["f16", "f32"])
def test_one_row_of_a_wider_matrix(dt):
    # The distance to a next row that there is not does not matter.
    print("one row", dt, flush=True)
    c = whole_numbers(1, 192, 100, 2, 16, dt, 3, np.array([1], np.int32))
    wide = torch.zeros((3, 192 + 4 + (dt == "f32")), dtype=F16 if dt == "f16" else F32, device=DEV)[:, :192]
    wide[:1] = dev(c[1])
    y = torch.zeros((3, 103), device=DEV)[:, :100]
    y[:1] = dev(c[0])
    got = B.adapter_add(y[:1], wide[:1], *[dev(a) for a in c[2:]], out=y[:1])
    assert np.array_equal(host(got), O.adapter_add(*c).astype(np.float32))
    again = B.adapter_add(dev(c[0]), wide[:1], *[dev(a) for a in c[2:5]])     # every rank
    assert np.array_equal(host(again), O.adapter_add(*c[:5]).astype(np.float32))
    h, out = y[:1], torch.empty((1, 100), device=DEV)
    want = host(B.norm_residual(h.contiguous(), pre_norm="rms", x_dtype=F32)[1])
    B.norm_residual(h, pre_norm="rms", h_out=torch.as_strided(y, (1, 100), (100, 1)), x_out=out)
    assert np.array_equal(host(out), want)


@pytest.mark.parametrize("M,K,N,L,R,dt", [(1, 64, 40, 65, 8, "f16"), (40, 128, 100, 100, 16, "f16"),
                                          (100, 64, 70, 300, 5, "f32"), (300, 128, 70, 200, 24, "f16"),
                                          (200, 64, 300, 130, 16, "f32"), (130, 192, 40, 4000, 8, "f16")])
def test_more_than_64_adapters(M, K, N, L, R, dt):
    print("many adapters", M, K, N, L, R, dt, flush=True)
    c = whole_numbers(M, K, N, L, R, dt, M + L)
    c[4][-1] = L - 1
    c[4][0] = L - 1 if M == 1 else 64
    c[5][[64, L - 1]] = R, max(R // 2, 1)
    assert np.array_equal(host(B.adapter_add(*[dev(a) for a in c])), O.adapter_add(*c).astype(np.float32))
    assert np.array_equal(host(B.adapter_add(*[dev(a) for a in c[:5]])), O.adapter_add(*c[:5]).astype(np.float32))


@pytest.mark.parametrize("M,C", [(4 * 2 ** 20 + 9, 16), (2 ** 20 + 5, 520)])
def test_norms_of_more_rows_than_workgroups(M, C):
    # Three sums a row: a workgroup's second row starts on the other slot.
    print("norms, long loop", M, C, flush=True)
    step = 2 ** 20 if C > 512 else 4 * 2 ** 20
    h = torch.randn((M, C), dtype=F16, device=DEV)
    y = torch.randn((M, C), dtype=F16, device=DEV)
    rows = np.array([0, 1, 2, 3, 4, 1000, step - 2, step - 1, step, step + 1, step + 2, step + 3, step + 4, M - 1])
    at = torch.from_numpy(rows).to(DEV)
    size = torch.tensor([1, 300, 0.01, 40, 2, 1, 7, 500, 300, 0.01, 200, 0, 100, 3], device=DEV)[:, None]
    h[at] = (h[at].float() * size).half()
    y[at] = (y[at].float() * size.flip(0) + size).half()
    rng = np.random.default_rng(2)
    p = {k: rng.uniform(0.5, 1.5, C).astype(np.float32) for k in ("post_w", "pre_w")}
    kw = dict(p, post="layer", pre="rms", rs=0.5, eps=1e-5)
    h0, y0 = host(h[at]), host(y[at])
    gh, gx = B.norm_residual(h, y, post_norm="layer", pre_norm="rms", residual_scale=0.5, eps=1e-5,
                             post_weight=dev(p["post_w"]), pre_weight=dev(p["pre_w"]), x_dtype=F32)
    seams.check(h0, y0, kw, np.float16, np.float32, (host(gh[at]), host(gx[at])))


def test_norms_past_2_31_elements():
    M, C = 131080, 16384
    print("norms, offsets", M, C, flush=True)
    h = torch.empty((M, C), dtype=F16, device=DEV).normal_()
    rows = np.array([0, 1, 65535, 65536, 131071, 131072, 131073, M - 1])
    at = torch.from_numpy(rows).to(DEV)
    gx = B.norm_residual(h, pre_norm="rms", eps=1e-5)[1]
    seams.check(host(h[at]), None, dict(pre="rms", eps=1e-5), np.float16, np.float16, (None, host(gx[at])))


@pytest.mark.parametrize("M,F,gap", [(40000, 24, 8), (40000, 23, 5), (70000, 30700, 0), (131080, 16390, 10)])
def test_gated_rows_and_offsets(M, F, gap):
    # More rows than the grid has, and both forms past 2^31 elements.
    print("gated, rows", M, F, gap, flush=True)
    g = torch.empty((M, F + gap), dtype=F16, device=DEV).normal_()[:, :F]
    at = {0, 1, 32767, 32768, 32769, M - 2, M - 1} | {min(2 ** 31 // (F + gap) + i, M - 1) for i in (-1, 0, 1)}
    at = torch.tensor(sorted(at), device=DEV)
    out = torch.full((M, F + gap), 7.0, dtype=F16, device=DEV)
    B.gated_activation(g, None, "silu", out=out[:, :F])
    gr, got = host(g[at]), host(out[at])
    ref = O.activation(gr, "silu")
    assert np.all(np.abs(got[:, :F] - ref) <= seams.act_bound(gr, ref, np.float16, None))
    assert np.all(got[:, F:] == 7.0)


def test_a_step_with_buffers_and_h_out_allocates_nothing():
    print("mlp allocations", flush=True)
    mlp, _ = MLP.random_block(256, 512, 3, 8)
    h = torch.randn((9, 256), device=DEV)
    index = torch.randint(-1, 3, (9,), dtype=torch.int32, device=DEV)
    x, buf, out = mlp.enter(h, mlp.pre_weight), mlp.buffers(9), torch.empty_like(h)
    want, want_x = mlp(h, x, index)
    count = lambda: torch.cuda.memory_stats()["allocation.all.allocated"]  # noqa: E731
    before = count()
    got, got_x = mlp(h, x, index, buf, out)
    assert count() == before
    assert got is out and torch.equal(got, want) and torch.equal(got_x, want_x)
    got, got_x = mlp(h, x, index, buf, h)                # in place
    assert got is h and torch.equal(h, want)
