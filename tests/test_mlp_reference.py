"""mlp.reference, the block without quantization that the example measures itself
against, for every field of a block, next to the oracle's formulas.  Runs
without a GPU; both are float64."""
import numpy as np
import pytest
import torch

from bit_gemm_block_amd import mlp as MLP
from oracle import block_oracle as O


def adapters(rng, L, R, K, N, ranks, scales):
    n = lambda a: torch.from_numpy(a)  # noqa: E731
    return MLP.Adapters(n(rng.standard_normal((L, R, K))), n(rng.standard_normal((L, N, R))),
                        n(np.array([R, 3, 0], np.int32)) if ranks else None,
                        n(np.array([0.5, -2.0, 1.0], np.float32)) if scales else None)


@pytest.mark.parametrize("norm", ["rms", "layer"])
@pytest.mark.parametrize("act", ["silu", "gelu", "gelu_tanh", "relu"])
@pytest.mark.parametrize("ranks,scales,post,gate_rows", [(True, True, True, 0), (False, False, False, 1),
                                                         (True, False, True, 3), (False, True, False, 4)])
def test_reference_follows_every_field(norm, act, ranks, scales, post, gate_rows):
    rng = np.random.default_rng(gate_rows + 1)
    M, C, F, L, R = 7, 24, 16, 3, 8
    w = {"gate_up": rng.standard_normal((2 * F, C)) * C ** -0.5, "down": rng.standard_normal((C, F)) * F ** -0.5}
    a1, a2 = adapters(rng, L, R, C, 2 * F, ranks, scales), adapters(rng, L, R, F, C, ranks, scales)
    post_w, pre_w = rng.uniform(0.5, 1.5, C), rng.uniform(0.5, 1.5, C)
    gate = rng.standard_normal((-(-M // gate_rows), C)) if gate_rows else None
    h, x = rng.standard_normal((M, C)), rng.standard_normal((M, C))
    index = np.array([0, 1, 2, -1, 3, 1, 0], np.int32)
    t = lambda a: None if a is None else torch.from_numpy(a)  # noqa: E731
    mlp = MLP.GatedMLP(MLP.Projection(None, None, 8, "tiled", a1), MLP.Projection(None, None, 8, "tiled", a2),
                       t(post_w) if post else None, t(pre_w), norm=norm, act=act, gate=t(gate),
                       gate_rows=max(gate_rows, 1), residual_scale=0.7, eps=1e-4)

    def project(v, name, a):
        n = lambda b: None if b is None else b.numpy()  # noqa: E731
        return O.adapter_add(v @ w[name].T, v, n(a.At), n(a.Bt), index, n(a.ranks), n(a.scales))
    y = project(x, "gate_up", a1)
    y = project(O.activation(y[:, :F], act) * y[:, F:], "down", a2)
    want = O.norm_residual(h, y, norm if post else "none", post_w if post else None, gate=gate,
                           gate_rows=max(gate_rows, 1), rs=0.7, pre=norm, pre_w=pre_w, eps=1e-4)
    got = MLP.reference(mlp, {k: t(v) for k, v in w.items()}, t(h), t(x), t(index))
    for a, b in zip(got, want):
        assert np.allclose(a.numpy(), b, rtol=1e-11, atol=1e-11)


def test_reference_without_adapters_or_index():
    rng = np.random.default_rng(0)
    t = lambda *s: torch.from_numpy(rng.standard_normal(s))  # noqa: E731
    w = {"gate_up": t(32, 24), "down": t(24, 16)}
    h, x, one = t(4, 24), t(4, 24), torch.ones(24, dtype=torch.float64)
    plain = MLP.Projection(None, None, 8, "tiled")
    own = MLP.Projection(None, None, 8, "tiled", adapters(rng, 3, 8, 24, 32, True, True))
    a = MLP.reference(MLP.GatedMLP(plain, plain, one, one), w, h, x, None)
    b = MLP.reference(MLP.GatedMLP(own, plain, one, one), w, h, x, None)
    assert all(torch.equal(p, q) for p, q in zip(a, b))
