"""The gated MLP block (W4A4 projections, adapters, gated activation, seam norm)
as a whole: its steps are each checked against float64 references elsewhere;
here that the block wires them as its formula says.

* adapters and norms carry the result: with every projection's W4A4 output taken
  from the layer itself, the block equals the float64 formula of the remaining
  steps to float32 and fp16 rounding;
* against the block without quantization: 4-bit weights and activations of
  normal data carry an error of about 7/64 of a step's range each; the block's
  update stays within 0.45 of it in norm, which any misplaced step exceeds (an
  update without adapters, for instance, is checked to be further off than the
  block's own).
"""
import numpy as np
import pytest
import torch

from bit_gemm_block_amd import block as B
from bit_gemm_block_amd import mlp as MLP
from bit_gemm_block_amd import w4a4 as W
from oracle import block_oracle as O

pytestmark = pytest.mark.gpu

DEV = "cuda:0"


def host(t):
    torch.cuda.synchronize()
    return t.cpu().numpy()


def inputs(M, C, L, seed=3):
    g = torch.Generator().manual_seed(seed)
    h = torch.randn((M, C), generator=g).to(DEV)
    index = torch.randint(-1, L, (M,), generator=g, dtype=torch.int32).to(DEV)
    return h, index


@pytest.mark.parametrize("M,C,F,L,rank,layout", [(1, 256, 512, 2, 8, "tiled"), (9, 512, 384, 4, 16, "tiled"),
                                                 (70, 256, 640, 3, 8, "tiled_f6"),
                                                 (200, 512, 512, 5, 32, "tiled")])
def test_block_is_its_steps(M, C, F, L, rank, layout):
    print("mlp", M, C, F, L, rank, layout, flush=True)
    mlp, w = MLP.random_block(C, F, L, rank, w_layout=layout)
    h, index = inputs(M, C, L)
    x = mlp.enter(h, mlp.pre_weight)
    buf = mlp.buffers(M)
    h0 = h.clone()
    got_h, got_x = mlp(h, x, index, buf)
    assert torch.equal(h, h0)
    plain_h, plain_x = mlp(h, x, index)                       # without buffers: the same bits
    assert torch.equal(plain_h, got_h) and torch.equal(plain_x, got_x)

    ix = host(index)

    def project(p, v):
        y = host(W.qlinear_forward(v, p.wq, p.w_scale, p.had_block, 0, w_layout=p.w_layout))
        a = p.adapters
        return O.adapter_add(y, host(v), host(a.At), host(a.Bt), ix, host(a.ranks), host(a.scales))
    y1 = project(mlp.gate_up, x)
    act = O.activation(y1[:, :F], "silu") * y1[:, F:]
    y1_gpu = W.qlinear_forward(x, mlp.gate_up.wq, mlp.gate_up.w_scale, mlp.gate_up.had_block, 0,
                               w_layout=layout)
    a = mlp.gate_up.adapters
    B.adapter_add(y1_gpu, x, a.At, a.Bt, index, a.ranks, a.scales, out=y1_gpu)
    act_gpu = B.gated_activation(y1_gpu[:, :F], y1_gpu[:, F:])
    # one rounding to fp16 beside float32 sums of some hundred terms
    assert np.all(np.abs(host(act_gpu) - act) <= 2.0 ** -10 * np.abs(act) + 1e-4 * np.sqrt(np.mean(act ** 2)))
    y2 = project(mlp.down, act_gpu)                           # from the codes of the block's own activations
    ref_h, ref_x = O.norm_residual(host(h), y2, "rms", host(mlp.post_weight), rs=mlp.residual_scale, pre="rms",
                                   pre_w=host(mlp.pre_weight), eps=mlp.eps)
    rms = lambda v: np.sqrt(np.mean(v ** 2))  # noqa: E731
    assert np.max(np.abs(host(got_h) - ref_h)) <= 1e-4 * rms(ref_h)
    assert np.all(np.abs(host(got_x) - ref_x) <= 2.0 ** -10 * np.abs(ref_x) + 1e-4 * rms(ref_x))

    full, _ = MLP.reference(mlp, w, h, x, index)
    update = full - h.double()
    off = float(((got_h.double() - h.double()) - update).norm() / update.norm())
    bare, _ = mlp(h, x, None)
    without = float(((bare.double() - h.double()) - update).norm() / update.norm())
    print("  off by", off, "without adapters", without, flush=True)
    assert off <= 0.45
    if (ix >= 0).mean() > 0.5:
        assert without > off


def test_block_replays_as_graph():
    print("mlp graph", flush=True)
    M, C, F, L = 12, 512, 512, 4
    mlp, _ = MLP.random_block(C, F, L, 16)
    h, index = inputs(M, C, L)
    x = mlp.enter(h, mlp.pre_weight)
    buf, out = mlp.buffers(M), torch.empty_like(h)
    mlp(h, x, index, buf, out)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        mlp(h, x, index, buf, out)
    for k in range(3):
        h.mul_(1.25)
        x.copy_(mlp.enter(h, mlp.pre_weight))
        index.copy_(torch.roll(index, 1))
        want_h, want_x = mlp(h, x, index)
        want_h, want_x = host(want_h), host(want_x)
        out.zero_()
        buf["x"].zero_()
        g.replay()
        assert np.array_equal(host(out), want_h) and np.array_equal(host(buf["x"]), want_x), k
