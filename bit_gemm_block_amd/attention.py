"""An attention block over the quantized cache, on the W4A4 layer's projections.

    x  [M, C]                       the previous seam's normed stream (fp16)
    y  = W4(x; q|k|v)               one projection, [M, (H + 2 Hk) D] float32
    encode(q, k)                    the caller's position encoding, in place (or none)
    cache[slots] = k, v             quantized per token and head       (cache_write)
    o  = softmax(q K^T / sqrt(D)) V over each sequence's pages         (cache_attention)
    y  = W4(o; out)                 [M, C] float32
    h' = h + scale * gate * norm(y),  x' = norm(h')                    (norm_residual)

The rows of a step are queries of a ragged batch: one new token of each sequence,
or a piece of a prompt of each.  The block chains with mlp.GatedMLP through
(h', x').  Projections are those of mlp.py, weight_only ones with activations
that are not quantized.  Every step enqueues on the current stream and can be
captured into a HIP graph, in which the batch's tensors may change between
replays; with buffers() made once and h_out given, a step allocates nothing.

    python -m bit_gemm_block_amd.attention [--seqs S] [--length L] [--hidden C] ...

builds a block with random weights and S sequences of L tokens, runs a decoding
step eagerly and as a graph, and prints the time of a step and its distance from
the block without quantization.
"""
from __future__ import annotations

import argparse
from dataclasses import dataclass, field
from typing import Callable, Dict, List, Optional, Sequence, Tuple

import torch

from . import block as B
from . import decode as D
from . import mlp as M
from .mlp import Projection


@dataclass
class Batch:
    """Which tokens a step holds: where they go (slots, int32 [M]) and what they
    see (see decode.cache_attention; lengths count the step's own tokens)."""
    slots: torch.Tensor
    tables: torch.Tensor
    lengths: torch.Tensor
    q_start: Optional[torch.Tensor] = None
    max_q: int = 1
    prefix_table: Optional[torch.Tensor] = None
    prefix_length: Optional[torch.Tensor] = None


def slots_of(tables: torch.Tensor, sequence: torch.Tensor, position: torch.Tensor, page_size: int) -> torch.Tensor:
    """The slots (int32) of tokens at positions of sequences."""
    page = tables[sequence.long(), (position // page_size).long()]
    return (page * page_size + position % page_size).int()


@dataclass
class CachedAttention:
    qkv: Projection                      # to the queries, keys and values, side by side
    out: Projection
    heads: int
    kv_heads: int
    head_dim: int
    post_weight: Optional[torch.Tensor]  # of the norm after the block (None: no norm)
    pre_weight: torch.Tensor             # of the norm before the next block
    encode: Optional[Callable[[torch.Tensor, torch.Tensor], None]] = None
    norm: str = "rms"
    gate: Optional[torch.Tensor] = None
    gate_rows: int = 1
    residual_scale: float = 1.0
    eps: float = 1e-5
    _none: Dict[str, torch.Tensor] = field(default_factory=dict, repr=False)

    def buffers(self, tokens: int, cache: D.KVCache, batch: Batch) -> Dict[str, torch.Tensor]:
        """Buffers of steps of so many tokens whose batches have the shapes of
        this one (calls that share them must not overlap in time)."""
        dev = self.qkv.w_scale.device
        C, A = self.out.w_scale.shape[0], self.heads * self.head_dim
        prefix = 0 if batch.prefix_table is None else batch.prefix_table.shape[0]
        empty = lambda n, t: torch.empty(n, dtype=t, device=dev)  # noqa: E731
        return {**M.projection_buffers(tokens, ((self.qkv, C), (self.out, A))),
                "qkv": empty((tokens, self.qkv.w_scale.shape[0]), torch.float32),
                "attention": D.cache_attention_workspace(cache, tokens, self.heads, batch.lengths.shape[0],
                                                         batch.tables.shape[1], batch.max_q, prefix),
                "o": torch.zeros((tokens, A), dtype=torch.float16, device=dev),
                "out": empty((tokens, C), torch.float32), "x": empty((tokens, C), torch.float16)}

    def enter(self, h: torch.Tensor, pre_weight: torch.Tensor) -> torch.Tensor:
        """The normed stream x of the first block."""
        return B.norm_residual(h, pre_norm=self.norm, pre_weight=pre_weight, eps=self.eps)[1]

    def __call__(self, h: torch.Tensor, x: torch.Tensor, cache: D.KVCache, batch: Batch,
                 index: Optional[torch.Tensor] = None, buf: Optional[Dict[str, torch.Tensor]] = None,
                 h_out: Optional[torch.Tensor] = None) -> Tuple[torch.Tensor, torch.Tensor]:
        """(h', x') from the residual stream h and the normed stream x (fp16) of
        the step's tokens, whose keys and values are written to the cache first;
        index is the adapter of every row.  Rows of no sequence get a result
        without meaning.  With buffers, x' is theirs; h' is h_out (which may be
        h), a new tensor without one."""
        buf = self._none if buf is None else buf
        y = self.qkv(x, index, buf, "qkv")
        A, E = self.heads * self.head_dim, self.kv_heads * self.head_dim
        q, k, v = y[:, :A], y[:, A:A + E], y[:, A + E:]
        if self.encode is not None:
            self.encode(q, k)
        D.cache_write(cache, k, v, batch.slots)
        o = buf.get("o")
        if o is None:
            o = torch.zeros((x.shape[0], A), dtype=torch.float16, device=x.device)
        D.cache_attention(q, cache, batch.tables, batch.lengths, q_start=batch.q_start, max_q=batch.max_q,
                          prefix_table=batch.prefix_table, prefix_length=batch.prefix_length, out=o,
                          workspace=buf.get("attention"))
        y = self.out(o, index, buf, "out")
        post = self.post_weight
        return B.norm_residual(h, y, post_norm="none" if post is None else self.norm, post_weight=post,
                               gate=self.gate, gate_rows=self.gate_rows, residual_scale=self.residual_scale,
                               pre_norm=self.norm, pre_weight=self.pre_weight, eps=self.eps, h_out=h_out,
                               x_out=buf.get("x"))


def random_block(C: int, heads: int, kv_heads: int, head_dim: int, seed: int = 0, had_block: int = 128,
                 weight_only: bool = False, device="cuda") -> Tuple[CachedAttention, Dict[str, torch.Tensor]]:
    """A block with random weights, and those weights before quantization."""
    gen = torch.Generator(device=device).manual_seed(seed)
    rnd = lambda *s: torch.randn(s, generator=gen, device=device)  # noqa: E731
    A, E = heads * head_dim, kv_heads * head_dim
    w1, w2 = rnd(A + 2 * E, C) * C ** -0.5, rnd(C, A) * A ** -0.5
    p1 = Projection.quantize(w1, had_block, weight_only=weight_only)
    p2 = Projection.quantize(w2, had_block, weight_only=weight_only)
    block = CachedAttention(p1, p2, heads, kv_heads, head_dim, 1.0 + 0.1 * rnd(C), 1.0 + 0.1 * rnd(C))
    return block, {"qkv": w1, "out": w2}


Past = List[Tuple[torch.Tensor, torch.Tensor]]


def reference(block: CachedAttention, w: Dict[str, torch.Tensor], h: torch.Tensor, x: torch.Tensor, past: Past,
              counts: Sequence[int], index: Optional[torch.Tensor] = None
              ) -> Tuple[torch.Tensor, torch.Tensor, Past]:
    """The block in float64 without quantization (the weights w): (h', x', past).
    past holds every sequence's keys and values in front of the step, [L, Hk, D]
    each, counts its rows of the step, which follow each other; the returned one
    holds the step's as well."""
    H, E, Dh = block.heads, block.kv_heads, block.head_dim
    y = M.project_reference(x.double(), w["qkv"], block.qkv.adapters, index)
    q, k, v = y.split([H * Dh, E * Dh, E * Dh], dim=1)
    if block.encode is not None:
        block.encode(q, k)
    o, grown, at = torch.zeros_like(q), [], 0
    for (pk, pv), n in zip(past, counts):
        rows = slice(at, at + n)
        at += n
        kk, vv = torch.cat((pk, k[rows].view(n, E, Dh))), torch.cat((pv, v[rows].view(n, E, Dh)))
        grown.append((kk, vv))
        if n == 0:
            continue
        hidden = torch.ones((n, kk.shape[0]), dtype=torch.bool, device=q.device).triu(kk.shape[0] - n + 1)
        for i in range(H):
            t = q[rows, i * Dh:(i + 1) * Dh] @ kk[:, i // (H // E)].t() * Dh ** -0.5
            o[rows, i * Dh:(i + 1) * Dh] = t.masked_fill(hidden, float("-inf")).softmax(1) @ vv[:, i // (H // E)]
    y = M.project_reference(o, w["out"], block.out.adapters, index)
    return (*M.seam_reference(block, h, y), grown)


def main() -> None:
    ap = argparse.ArgumentParser(description="A decoding step of an attention block over the quantized cache")
    for name, value in (("seqs", 32), ("length", 2048), ("hidden", 4096), ("heads", 32), ("kv-heads", 8),
                        ("head-dim", 128), ("page-size", 64), ("had-block", 128)):
        ap.add_argument(f"--{name}", type=int, default=value)
    ap.add_argument("--bits", type=int, default=4, choices=[4, 8])
    ap.add_argument("--weight-only", action="store_true", help="activations are not quantized")
    a = ap.parse_args()
    S, L, P = a.seqs, a.length, a.page_size
    block, w = random_block(a.hidden, a.heads, a.kv_heads, a.head_dim, had_block=a.had_block,
                            weight_only=a.weight_only)
    width = -(-L // P)
    cache = D.KVCache.empty(S * width, a.kv_heads, P, a.head_dim, a.bits)
    tables = torch.randperm(S * width, device="cuda").int().view(S, width)
    seq = torch.arange(S, device="cuda")
    past = []
    for s in range(S):
        k, v = (torch.randn((L - 1, a.kv_heads * a.head_dim), device="cuda") for _ in range(2))
        at = torch.arange(L - 1, device="cuda")
        D.cache_write(cache, k, v, slots_of(tables, torch.full_like(at, s), at, P))
        past.append(tuple(t.double().view(L - 1, a.kv_heads, a.head_dim) for t in (k, v)))
    batch = Batch(slots_of(tables, seq, torch.full_like(seq, L - 1), P), tables,
                  torch.full((S,), L, dtype=torch.int32, device="cuda"))
    h = torch.randn((S, a.hidden), device="cuda")
    x = block.enter(h, block.pre_weight)
    buf, out = block.buffers(S, cache, batch), torch.empty_like(h)
    got, _ = block(h, x, cache, batch, None, buf, out)
    ref, _, _ = reference(block, w, h, x, past, [1] * S)
    update = ref - h.double()
    print(f"{S} sequences of {L} tokens, {a.hidden} -> {a.heads} heads of {a.head_dim} on {a.kv_heads}, "
          f"{a.bits}-bit cache")
    off = float((got.double() - h.double() - update).norm() / update.norm())
    print(f"distance from the block without quantization: {off:.3f} of it")
    print(f"eager: {M.timed(lambda: block(h, x, cache, batch, None, buf, out)):.1f} us a step")
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        block(h, x, cache, batch, None, buf, out)
    print(f"graph: {M.timed(g.replay):.1f} us a step")


if __name__ == "__main__":
    main()
