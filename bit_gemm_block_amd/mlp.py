"""A gated MLP block on the W4A4 layer, for requests with adapters of their own.

    x  [M, C]                       the previous seam's normed stream (fp16)
    y  = W4A4(x; gate|up)           one shared projection, [M, 2F] float32
    y += adapters of each row's request                       (adapter_add)
    a  = act(y[:, :F]) * y[:, F:]   [M, F] fp16               (gated_activation)
    y  = W4A4(a; down)              [M, C] float32
    y += adapters of each row's request                       (adapter_add)
    h' = h + scale * gate * norm(y),  x' = norm(h')           (norm_residual)

Every step enqueues on the current stream and can be captured into a HIP graph;
with buffers() made once and h_out given, a step allocates nothing.

    python -m bit_gemm_block_amd.mlp [--tokens M] [--hidden C] [--ffn F] ...

builds a block with random weights, runs it eagerly and as a graph, and prints
the time of a step and its distance from the block without quantization.
"""
from __future__ import annotations

import argparse
from dataclasses import dataclass, field
from typing import Dict, Optional, Tuple

import torch

from . import block as B
from . import w4a4 as W


@dataclass
class Adapters:
    """The stacked adapters of one projection (see block.adapter_add)."""
    At: torch.Tensor
    Bt: torch.Tensor
    ranks: Optional[torch.Tensor] = None
    scales: Optional[torch.Tensor] = None


@dataclass
class Projection:
    """Quantized weights of one projection, and its requests' adapters."""
    wq: torch.Tensor
    w_scale: torch.Tensor
    had_block: int
    w_layout: str
    adapters: Optional[Adapters] = None

    @classmethod
    def quantize(cls, w: torch.Tensor, had_block: int, w_layout: str = "tiled",
                 adapters: Optional[Adapters] = None) -> "Projection":
        """From float weights [N, K] (rotated by the Hadamard block and quantized
        per output channel)."""
        wq, ws = W.quantize_weight_int4(w, had_block, 0, torch.float16, layout=w_layout)
        return cls(wq, ws, had_block, w_layout, adapters)

    def __call__(self, x: torch.Tensor, index: Optional[torch.Tensor],
                 buf: Dict[str, torch.Tensor], name: str) -> torch.Tensor:
        y = W.qlinear_forward(x, self.wq, self.w_scale, self.had_block, 0, y=buf.get(name),
                              workspace=buf.get("layer"), w_layout=self.w_layout)
        if self.adapters is not None and index is not None:
            a = self.adapters
            B.adapter_add(y, x, a.At, a.Bt, index, a.ranks, a.scales, out=y,
                          workspace=buf.get("adapters"))
        return y


@dataclass
class GatedMLP:
    gate_up: Projection
    down: Projection
    post_weight: Optional[torch.Tensor]  # of the norm after the block (None: no norm)
    pre_weight: torch.Tensor             # of the norm before the next block
    norm: str = "rms"
    act: str = "silu"
    gate: Optional[torch.Tensor] = None
    gate_rows: int = 1
    residual_scale: float = 1.0
    eps: float = 1e-5
    _none: Dict[str, torch.Tensor] = field(default_factory=dict, repr=False)

    def buffers(self, M: int) -> Dict[str, torch.Tensor]:
        """Buffers of a step of M tokens (calls that share them must not overlap
        in time)."""
        dev = self.gate_up.w_scale.device
        N1, C = self.gate_up.w_scale.shape[0], self.down.w_scale.shape[0]
        F = N1 // 2
        layer = max(W.qlinear_workspace_size(M, N1, C, 0), W.qlinear_workspace_size(M, C, F, 0))
        adapters = max([B.adapter_workspace_size(M, K, p.adapters.At.shape[1])
                        for p, K in ((self.gate_up, C), (self.down, F)) if p.adapters is not None] + [1])
        empty = lambda n, t: torch.empty(n, dtype=t, device=dev)  # noqa: E731
        return {"layer": empty(layer, torch.uint8), "adapters": empty(adapters, torch.uint8),
                "gate_up": empty((M, N1), torch.float32), "act": empty((M, F), torch.float16),
                "down": empty((M, C), torch.float32), "x": empty((M, C), torch.float16)}

    def enter(self, h: torch.Tensor, pre_weight: torch.Tensor) -> torch.Tensor:
        """The normed stream x of the first block."""
        return B.norm_residual(h, pre_norm=self.norm, pre_weight=pre_weight, eps=self.eps)[1]

    def __call__(self, h: torch.Tensor, x: torch.Tensor, index: Optional[torch.Tensor] = None,
                 buf: Optional[Dict[str, torch.Tensor]] = None,
                 h_out: Optional[torch.Tensor] = None) -> Tuple[torch.Tensor, torch.Tensor]:
        """(h', x') from the residual stream h, the normed stream x (fp16) and the
        adapter of every row (int32, outside the adapters: none).  With buffers,
        x' is theirs; h' is h_out (which may be h), a new tensor without one."""
        buf = self._none if buf is None else buf
        y = self.gate_up(x, index, buf, "gate_up")
        F = y.shape[1] // 2
        a = B.gated_activation(y[:, :F], y[:, F:], self.act, out=buf.get("act"))
        y = self.down(a, index, buf, "down")
        post = self.post_weight
        return B.norm_residual(h, y, post_norm="none" if post is None else self.norm, post_weight=post,
                               gate=self.gate, gate_rows=self.gate_rows,
                               residual_scale=self.residual_scale, pre_norm=self.norm,
                               pre_weight=self.pre_weight, eps=self.eps, h_out=h_out, x_out=buf.get("x"))


def random_block(C: int, F: int, adapters: int, rank: int, seed: int = 0, w_layout: str = "tiled",
                 had_block: int = 128, device="cuda") -> Tuple[GatedMLP, Dict[str, torch.Tensor]]:
    """A block with random weights, and those weights before quantization."""
    gen = torch.Generator(device=device).manual_seed(seed)
    rnd = lambda *s: torch.randn(s, generator=gen, device=device)  # noqa: E731
    w1, w2 = rnd(2 * F, C) * C ** -0.5, rnd(C, F) * F ** -0.5

    def lora(K, N):
        if adapters == 0:
            return None
        return Adapters((rnd(adapters, rank, K) * K ** -0.5).half(),
                        (0.3 * rnd(adapters, N, rank) * rank ** -0.5).half(),
                        torch.full((adapters,), rank, dtype=torch.int32, device=device),
                        torch.linspace(0.5, 1.0, adapters, device=device))
    p1 = Projection.quantize(w1, had_block, w_layout, lora(C, 2 * F))
    p2 = Projection.quantize(w2, had_block, w_layout, lora(F, C))
    mlp = GatedMLP(p1, p2, 1.0 + 0.1 * rnd(C), 1.0 + 0.1 * rnd(C), residual_scale=0.5)
    return mlp, {"gate_up": w1, "down": w2}


def reference(mlp: GatedMLP, w: Dict[str, torch.Tensor], h: torch.Tensor, x: torch.Tensor,
              index: Optional[torch.Tensor]) -> Tuple[torch.Tensor, torch.Tensor]:
    """The block in float64 without quantization (the weights w)."""
    def project(v, weight, a):
        y = v @ weight.double().t()
        if a is not None and index is not None:
            for i in range(a.At.shape[0]):
                rows = index == i
                r = a.At.shape[1] if a.ranks is None else min(max(int(a.ranks[i]), 0), a.At.shape[1])
                s = 1.0 if a.scales is None else float(a.scales[i])
                y[rows] += s * ((v[rows] @ a.At[i, :r].double().t()) @ a.Bt[i, :, :r].double().t())
        return y

    def norm(v, weight):
        if mlp.norm == "layer":
            v = v - v.mean(1, keepdim=True)
        return v / (v.square().mean(1, keepdim=True) + mlp.eps).sqrt() * weight.double()

    def act(g):
        f = torch.nn.functional
        return {"silu": f.silu, "gelu": f.gelu, "relu": f.relu,
                "gelu_tanh": lambda v: f.gelu(v, approximate="tanh")}[mlp.act](g)
    y = project(x.double(), w["gate_up"], mlp.gate_up.adapters)
    F = y.shape[1] // 2
    y = project(act(y[:, :F]) * y[:, F:], w["down"], mlp.down.adapters)
    if mlp.post_weight is not None:
        y = norm(y, mlp.post_weight)
    if mlp.gate is not None:
        y = y * mlp.gate.double()[torch.arange(y.shape[0], device=y.device) // mlp.gate_rows]
    out = h.double() + mlp.residual_scale * y
    return out, norm(out, mlp.pre_weight)


def main() -> None:
    ap = argparse.ArgumentParser(description="A gated MLP block with W4A4 projections and adapters")
    for name, value in (("tokens", 64), ("hidden", 4096), ("ffn", 14336), ("adapters", 16), ("rank", 16)):
        ap.add_argument(f"--{name}", type=int, default=value)
    ap.add_argument("--layout", default="tiled", choices=["tiled", "tiled_f6"])
    a = ap.parse_args()
    mlp, w = random_block(a.hidden, a.ffn, a.adapters, a.rank, w_layout=a.layout)
    h = torch.randn((a.tokens, a.hidden), device="cuda")
    index = (torch.arange(a.tokens) * (a.adapters + 1) // a.tokens - 1).int().cuda()
    x = mlp.enter(h, mlp.pre_weight)
    buf, out = mlp.buffers(a.tokens), torch.empty_like(h)
    got, x_next = mlp(h, x, index, buf, out)
    ref, _ = reference(mlp, w, h, x, index)
    d = (got.double() - h.double()) - (ref - h.double())
    print(f"{a.tokens} tokens, {a.hidden} -> 2 x {a.ffn} -> {a.hidden}, {a.adapters} adapters of rank {a.rank}")
    print(f"distance from the block without quantization: {float(d.norm() / (ref - h.double()).norm()):.3f} of it")

    def timed(f, n=50):
        f()
        torch.cuda.synchronize()
        e0, e1 = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
        e0.record()
        for _ in range(n):
            f()
        e1.record()
        e1.synchronize()
        return 1e3 * e0.elapsed_time(e1) / n
    print(f"eager: {timed(lambda: mlp(h, x, index, buf, out)):.1f} us a step")
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        mlp(h, x, index, buf, out)
    print(f"graph: {timed(g.replay):.1f} us a step")


if __name__ == "__main__":
    main()
