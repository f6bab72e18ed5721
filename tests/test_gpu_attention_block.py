"""The attention block (projections, cache writes, attention over the cache, seam
norm) as a whole: its steps are each checked against float64 references
elsewhere; here that the block runs them as its formula says, over a prompt's
pieces and decoding steps, in a graph, and together with the gated MLP block.

* step by step from the GPU's own intermediate results: the cache holds the
  quantizer's codes and scales of the projection's columns, bit for bit, and
  nothing else changed; the attention output is within 2^-9 of the largest value
  a softmax average can have here (an fp16 rounding, 2^-11 of it, and the
  operator's own bound, below 2^-12 at these lengths); the seam as in the gated
  block's test;
* against the block without quantization: 4-bit weights of normal data carry an
  error of about 1/8 of themselves a projection (channel scales of max/7 with
  max near 3.2 sigma: a uniform error of 0.46 sigma / sqrt(12) = 0.13 sigma),
  W4A4 activations as much again, an 8-bit cache below 0.01, a 4-bit one the
  same 0.13.  Two projections in a row and the cache's keys and values, as
  independent errors: sqrt(2 + 1) 0.13 = 0.23 weight-only, sqrt(4 + 1) 0.13 =
  0.3 with W4A4, of each row's update, which the seam's norm keeps; the weights'
  share of an average over the values does not shrink, a score's error adds up
  to the same again: at most twice that, 0.45 and 0.6, which a misplaced head,
  page or step exceeds (independent rows are 1.41 apart).
"""
import numpy as np
import pytest
import torch

from bit_gemm_block_amd import attention as A
from bit_gemm_block_amd import decode as D
from bit_gemm_block_amd import mlp as MLP
from bit_gemm_block_amd import w4a4 as W
from oracle import block_oracle as BO
from oracle import decode_oracle as O

pytestmark = pytest.mark.gpu

DEV = "cuda:0"


def host(t):
    torch.cuda.synchronize()
    return t.cpu().numpy()


def rotate_halves(q, k):
    """A position encoding in place that is the same at every position (signs of
    a head's halves), so that the test can undo it."""
    for t in (q, k):
        t[:, ::3] *= -1.0


def setup(H, E, Dh, bits, weight_only, S=3, pages=24, page=16, C=256, seed=0, had_block=128):
    block, w = A.random_block(C, H, E, Dh, seed=seed, had_block=had_block, weight_only=weight_only)
    cache = D.KVCache.empty(pages, E, page, Dh, bits, DEV)
    for t in (cache.k, cache.v, cache.k_scale, cache.v_scale):
        t.zero_()
    g = torch.Generator().manual_seed(seed)
    tables = torch.randperm(pages, generator=g)[:S * (pages // S)].int().view(S, -1).to(DEV)
    return block, w, cache, tables, g


def step(tables, before, counts, page):
    """(batch, lengths after it): counts[s] tokens behind the before[s] that are there."""
    seq = torch.cat([torch.full((c,), s) for s, c in enumerate(counts)]).to(DEV)
    pos = torch.cat([torch.arange(b, b + c) for b, c in zip(before, counts)]).to(DEV)
    after = [b + c for b, c in zip(before, counts)]
    starts = torch.tensor(np.concatenate(([0], np.cumsum(counts))), dtype=torch.int32, device=DEV)
    return A.Batch(A.slots_of(tables, seq, pos, page), tables, torch.tensor(after, dtype=torch.int32, device=DEV),
                   starts, max(counts)), after


@pytest.mark.parametrize("H,E,Dh,bits,weight_only,had_block,encoded",
                         [(4, 2, 64, 4, True, 1, False), (4, 1, 128, 8, False, 128, True), (4, 4, 64, 8, True, 128, True),
                          (8, 2, 128, 4, False, 64, False)])
def test_a_prompt_and_decoding_steps(H, E, Dh, bits, weight_only, had_block, encoded):
    print("attention block", H, E, Dh, bits, weight_only, had_block, flush=True)
    S, C, page = 3, 256, 16
    block, w, cache, tables, g = setup(H, E, Dh, bits, weight_only, S, had_block=had_block)
    block.encode = rotate_halves if encoded else None
    past = [(torch.zeros((0, E, Dh), dtype=torch.float64, device=DEV),) * 2 for _ in range(S)]
    before = [0] * S
    for counts in ([37, 1, 20], [1, 1, 1], [3, 0, 17], [1, 1, 1]):   # pieces of prompts and decoding steps
        batch, after = step(tables, before, counts, page)
        T = sum(counts)
        h = torch.randn((T, C), generator=g).to(DEV)
        x = block.enter(h, block.pre_weight)
        buf = block.buffers(T, cache, batch)
        old = [t.clone() for t in (cache.k, cache.v, cache.k_scale, cache.v_scale)]
        got_h, got_x = block(h, x, cache, batch, None, buf)

        y = host(block.qkv(x, None, {}, "qkv")).copy()            # the same call: the same bits
        if encoded:
            y[:, :(H + E) * Dh] = np.where(np.concatenate((np.arange(H * Dh), np.arange(E * Dh))) % 3 == 0,
                                           -y[:, :(H + E) * Dh], y[:, :(H + E) * Dh])
        assert np.array_equal(host(buf["qkv"]), y)
        slots = host(batch.slots)
        for t, s, was_t, was_s, cols in ((cache.k, cache.k_scale, old[0], old[2], y[:, H * Dh:(H + E) * Dh]),
                                         (cache.v, cache.v_scale, old[1], old[3], y[:, (H + E) * Dh:])):
            q, sc = O.quantize(cols.reshape(T, E, Dh), bits)
            codes, scales = host(was_t).copy(), host(was_s).copy()
            for i, slot in enumerate(slots):
                codes[slot // page, :, slot % page] = O.pack(q[i], bits)
                scales[slot // page, :, slot % page] = sc[i]
            assert np.array_equal(host(t), codes) and np.array_equal(host(s), scales)
        arrays = tuple(host(t) for t in (cache.k, cache.v, cache.k_scale, cache.v_scale)) + (bits,)
        ref_o, size, _ = O.attention(y[:, :H * Dh], arrays, host(tables), host(batch.lengths), host(batch.q_start),
                                     batch.max_q)
        assert np.max(np.abs(host(buf["o"]) - ref_o)) <= 2.0 ** -9 * size.max()
        y2 = host(block.out(buf["o"], None, {}, "out")).astype(np.float64)
        assert np.array_equal(host(buf["out"]), y2)
        ref_h, ref_x = BO.norm_residual(host(h), y2, "rms", host(block.post_weight), pre="rms",
                                        pre_w=host(block.pre_weight), eps=block.eps)
        rms = lambda v: np.sqrt(np.mean(v ** 2))  # noqa: E731
        assert np.max(np.abs(host(got_h) - ref_h)) <= 1e-4 * rms(ref_h)
        assert np.all(np.abs(host(got_x) - ref_x) <= 2.0 ** -10 * np.abs(ref_x) + 1e-4 * rms(ref_x))

        full, _, past = A.reference(block, w, h, x, past, counts)
        update = full - h.double()
        off = float((got_h.double() - full).norm() / update.norm())
        print("  off by", off, flush=True)
        assert off <= (0.45 if weight_only else 0.6)
        before = after


def test_a_shared_prefix_is_the_same_tokens_in_front():
    """The prefix in pages of its own, or in front of every sequence's own table:
    one result, to the operator's two ways of summing."""
    print("attention block, prefix", flush=True)
    S, E, Dh, page = 3, 2, 64, 16
    block, _, cache, tables, g = setup(4, E, Dh, 4, True, S, pages=40)
    rows = torch.randn((64, E * Dh), generator=g).to(DEV)
    pages = torch.tensor([37, 39, 38], dtype=torch.int32, device=DEV)     # 48 tokens that all share
    seq = torch.zeros(48, dtype=torch.int64, device=DEV)
    D.cache_write(cache, rows[:48], rows[16:], A.slots_of(pages[None], seq, torch.arange(48, device=DEV), page))
    own = [0, 5, 30]
    tables = tables[:, :3].contiguous()
    for s, n in enumerate(own):
        at = torch.arange(n, device=DEV)
        D.cache_write(cache, rows[:n], rows[:n], A.slots_of(tables, torch.full_like(at, s), at, page))
    batch, after = step(tables, own, [1] * S, page)
    batch.prefix_table, batch.prefix_length = pages, torch.tensor([48], dtype=torch.int32, device=DEV)
    h = torch.randn((S, 256), generator=g).to(DEV)
    x = block.enter(h, block.pre_weight)
    o1 = block.buffers(S, cache, batch)
    got, _ = block(h, x, cache, batch, None, o1)
    joined = torch.cat((pages[None].expand(S, -1), tables), 1).contiguous()
    flat = A.Batch(batch.slots, joined, batch.lengths + 48, batch.q_start, 1)
    o2 = block.buffers(S, cache, flat)
    want, _ = block(h, x, cache, flat, None, o2)
    size = float(o2["o"].abs().max())
    assert float((o1["o"].float() - o2["o"].float()).abs().max()) <= 2.0 ** -9 * size
    assert float((got - want).abs().max()) <= 0.02 * float((want - h).abs().max())


@pytest.mark.parametrize("weight_only", [False, True])
def test_steps_replay_as_graph_with_the_gated_block(weight_only):
    """A layer of both blocks, captured once, decodes several tokens: every replay
    equals the eager step, while the batch's tensors move on."""
    print("attention and gated block, graph", weight_only, flush=True)
    S, C, page = 4, 256, 16
    block, _, cache, tables, g = setup(4, 2, 64, 8, weight_only, S, pages=16)
    mlp, _ = MLP.random_block(C, 512, 0, 8, weight_only=weight_only)
    before = [3, 16, 0, 31]
    batch, after = step(tables, before, [1] * S, page)
    batch.q_start = None
    h = torch.randn((S, C), generator=g).to(DEV)
    x = block.enter(h, block.pre_weight)
    h1, h2 = torch.empty_like(h), torch.empty_like(h)
    b1, b2 = block.buffers(S, cache, batch), mlp.buffers(S)

    def layer(out1, out2, u1, u2):
        a, ax = block(h, x, cache, batch, None, u1, out1)
        return mlp(a, ax, None, u2, out2)
    state = [t.clone() for t in (cache.k, cache.v, cache.k_scale, cache.v_scale)]
    layer(h1, h2, b1, b2)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        layer(h1, h2, b1, b2)
    for k in range(4):
        nb, after = step(tables, before, [1] * S, page)
        batch.slots.copy_(nb.slots)
        batch.lengths.copy_(nb.lengths)
        h.copy_(torch.randn((S, C), generator=g))
        x.copy_(block.enter(h, block.pre_weight))
        for t, s in zip((cache.k, cache.v, cache.k_scale, cache.v_scale), state):
            t.copy_(s)
        want, want_x = (host(t) for t in layer(None, None, None, None))
        held = [host(t) for t in (cache.k, cache.v, cache.k_scale, cache.v_scale)]
        for t, s in zip((cache.k, cache.v, cache.k_scale, cache.v_scale), state):
            t.copy_(s)
        h2.zero_()
        b2["x"].zero_()
        graph.replay()
        assert np.array_equal(host(h2), want) and np.array_equal(host(b2["x"]), want_x), k
        for t, e, s in zip((cache.k, cache.v, cache.k_scale, cache.v_scale), held, state):
            assert np.array_equal(host(t), e), k
            s.copy_(t)
        before = after


def test_a_step_with_buffers_and_h_out_allocates_nothing():
    print("attention block, allocations", flush=True)
    S, page = 3, 16
    for weight_only, had_block in ((False, 128), (True, 128), (True, 1)):
        block, _, cache, tables, g = setup(4, 2, 64, 4, weight_only, S, had_block=had_block)
        batch, _ = step(tables, [20, 0, 7], [1] * S, page)
        h = torch.randn((S, 256), generator=g).to(DEV)
        x, buf, out = block.enter(h, block.pre_weight), block.buffers(S, cache, batch), torch.empty_like(h)
        want, want_x = block(h, x, cache, batch)
        count = lambda: torch.cuda.memory_stats()["allocation.all.allocated"]  # noqa: E731
        before = count()
        got, got_x = block(h, x, cache, batch, None, buf, out)
        assert count() == before
        assert got is out and torch.equal(got, want) and torch.equal(got_x, want_x)
        got, _ = block(h, x, cache, batch, None, buf, h)      # in place
        assert got is h and torch.equal(h, want)


@pytest.mark.parametrize("M,layout,had_block", [(1, "tiled", 128), (9, "tiled", 1), (70, "tiled", 128)])
def test_weight_only_gated_block_is_its_steps(M, layout, had_block):
    print("weight-only gated block", M, layout, had_block, flush=True)
    C, F = 256, 640
    mlp, w = MLP.random_block(C, F, 2, 8, w_layout=layout, had_block=had_block, weight_only=True)
    g = torch.Generator().manual_seed(M)
    h = torch.randn((M, C), generator=g).to(DEV)
    index = torch.randint(-1, 2, (M,), generator=g, dtype=torch.int32).to(DEV)
    x = mlp.enter(h, mlp.pre_weight)
    buf, out = mlp.buffers(M), torch.empty_like(h)
    want, want_x = mlp(h, x, index)
    count = torch.cuda.memory_stats()["allocation.all.allocated"]
    got, got_x = mlp(h, x, index, buf, out)
    assert torch.cuda.memory_stats()["allocation.all.allocated"] == count
    assert torch.equal(got, want) and torch.equal(got_x, want_x)
    # the projection is the float64 product of the stored weights
    v = host(x if had_block == 1 else W.hadamard_rotate(x, had_block))
    wq, ws = (host(t) for t in W.quantize_weight_int4(w["gate_up"], had_block, 0, torch.float16, layout="rowmajor"))
    y, size = O.qlinear_w4a16(v, wq, ws, 0)
    got_y = host(MLP.Projection(mlp.gate_up.wq, mlp.gate_up.w_scale, had_block, layout, None, True)(x, None, {}, ""))
    assert np.all(np.abs(got_y - y) <= (32 * 2 + 64) * 2.0 ** -24 * size)      # two tiles of K
    # the weights' error alone: 0.13 of each of two projections (above), 0.26 and
    # as much again for the activation between them
    full, _ = MLP.reference(mlp, w, h, x, index)
    assert float((got.double() - full).norm() / (full - h.double()).norm()) <= 0.4


def test_layouts_of_quantized_activations_are_refused():
    mlp, _ = MLP.random_block(256, 256, 0, 8, w_layout="tiled_f6", weight_only=True)
    h = torch.zeros((2, 256), device=DEV)
    with pytest.raises(ValueError):
        mlp(h, h.half())
