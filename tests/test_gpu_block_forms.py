"""Forms of the operators beside the layer that ordinary sizes do not reach, on
the GPU: a single row cut from a wider matrix."""
import numpy as np
import pytest
import torch

from bit_gemm_block_amd import block as B
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
