"""attention.reference, the block without quantization that the command measures
itself against, next to the oracle's formulas.  Runs without a GPU; both are
float64."""
import numpy as np
import pytest
import torch

from bit_gemm_block_amd import attention as A
from bit_gemm_block_amd import mlp as M
from oracle import block_oracle as BO


def attend(q, k, v, H, E, D):
    """q [n, H D] of the last n of the tokens k, v [L, E, D], causal."""
    n, L = q.shape[0], k.shape[0]
    o = np.zeros_like(q)
    for i in range(n):
        end = L - n + i + 1
        for h in range(H):
            t = k[:end, h * E // H] @ q[i, h * D:(h + 1) * D] / np.sqrt(D)
            p = np.exp(t - t.max())
            o[i, h * D:(h + 1) * D] = (p / p.sum()) @ v[:end, h * E // H]
    return o


@pytest.mark.parametrize("norm,post,encoded", [("rms", True, False), ("layer", False, True), ("rms", False, True)])
@pytest.mark.parametrize("H,E,D,counts", [(4, 2, 8, (1, 1, 1)), (6, 2, 4, (3, 0, 5)), (2, 2, 8, (4,))])
def test_reference_is_its_formula(norm, post, encoded, H, E, D, counts):
    rng = np.random.default_rng(len(counts) + H)
    C, T = 12, sum(counts)
    n = lambda *s: rng.standard_normal(s)  # noqa: E731
    t = torch.from_numpy
    w1, w2 = n((H + 2 * E) * D, C), n(C, H * D)
    past = [(n(L, E, D), n(L, E, D)) for L in (5, 0, 3)[:len(counts)]]
    post_w, pre_w = rng.uniform(0.5, 1.5, C), rng.uniform(0.5, 1.5, C)
    gate, h, x = n(-(-T // 2), C), n(T, C), n(T, C)

    def encode(q, k):
        q.mul_(0.5)
        k.add_(1.0)
    R = 3
    adapter = M.Adapters(t(n(2, R, C)), t(n(2, (H + 2 * E) * D, R)))
    index = (np.arange(T) % 3 - 1).astype(np.int32)
    block = A.CachedAttention(M.Projection(None, None, 8, "tiled", adapter), M.Projection(None, None, 8, "tiled"), H, E,
                              D, t(post_w) if post else None, t(pre_w), encode if encoded else None, norm, t(gate), 2,
                              0.7, 1e-4)
    y = BO.adapter_add(x @ w1.T, x, adapter.At.numpy(), adapter.Bt.numpy(), index)
    q, k, v = y[:, :H * D], y[:, H * D:(H + E) * D], y[:, (H + E) * D:]
    if encoded:
        q, k = q * 0.5, k + 1.0
    o, at, grown = np.zeros_like(q), 0, []
    for (pk, pv), c in zip(past, counts):
        kk = np.concatenate((pk, k[at:at + c].reshape(c, E, D)))
        vv = np.concatenate((pv, v[at:at + c].reshape(c, E, D)))
        o[at:at + c] = attend(q[at:at + c], kk, vv, H, E, D)
        grown.append((kk, vv))
        at += c
    want = BO.norm_residual(h, o @ w2.T, norm if post else "none", post_w if post else None, gate=gate, gate_rows=2,
                            rs=0.7, pre=norm, pre_w=pre_w, eps=1e-4)
    got_h, got_x, got_past = A.reference(block, {"qkv": t(w1), "out": t(w2)}, t(h), t(x),
                                         [(t(a), t(b)) for a, b in past], counts, t(index))
    assert np.allclose(got_h.numpy(), want[0], rtol=1e-10, atol=1e-10)
    assert np.allclose(got_x.numpy(), want[1], rtol=1e-10, atol=1e-10)
    for (a, b), (c, d) in zip(got_past, grown):
        assert np.allclose(a.numpy(), c, atol=1e-12) and np.allclose(b.numpy(), d, atol=1e-12)


def test_slots_follow_the_tables():
    tables = torch.tensor([[4, 1], [0, 3]], dtype=torch.int32)
    got = A.slots_of(tables, torch.tensor([0, 0, 1, 1]), torch.tensor([0, 17, 15, 31]), 16)
    assert got.dtype == torch.int32 and got.tolist() == [64, 17, 15, 63]
