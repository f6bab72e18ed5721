"""Measured cases of the operators that stand beside the W4A4 linear layer.

Three operators: low-rank adapters of many requests added to a shared
projection (`adapter_add`), the norms before and after a block joined with its
gate and residual (`norm_residual`), and the gated activation between two
projections (`gated_activation`).  Each case is one call on data that a serving
step has in hand.  `run` computes it in plain torch operations, or through the
package's entry points when `own` is set.
"""
import math

import torch

own = False

DEV = "cuda"


# --------------------------------------------------------------------------
# Cases
# --------------------------------------------------------------------------
def _adapter(name, M, K, N, adapters, rank, dtype, requests, mixed, none):
    """`requests` runs of tokens, one adapter (or none, in a share `none` of
    them) each; `mixed`: the tokens in random order instead of in runs."""
    return {"name": name, "op": "adapter_add", "M": M, "K": K, "N": N, "adapters": adapters, "rank": rank,
            "dtype": dtype, "requests": requests, "mixed": mixed, "none": none}


def _norm(name, M, C, kind, h, y, x, gate_rows, bias):
    """gate_rows: tokens that share a row of the gate (0: no gate)."""
    return {"name": name, "op": "norm_residual", "M": M, "C": C, "kind": kind, "h": h, "y": y, "x": x,
            "gate_rows": gate_rows, "bias": bias}


def _gated(name, M, F, act, src, dst, joined):
    """joined: gate and up are the two halves of one [M, 2F] projection."""
    return {"name": name, "op": "gated_activation", "M": M, "F": F, "act": act, "src": src, "dst": dst,
            "joined": joined}


def listed():
    return [
        # One token of one request on a 4096-wide projection: latency only.
        _adapter("adapters_token", 1, 4096, 4096, 8, 16, "float16", 1, False, 0.0),
        # A decoding batch: 64 requests, one token each, on the qkv projection,
        # ranks up to 64, an eighth of the requests on the base model.
        _adapter("adapters_decode", 64, 4096, 6144, 32, 64, "float16", 64, True, 0.125),
        # Odd sizes in float32, tokens of several requests interleaved.
        _adapter("adapters_odd_f32", 333, 1088, 1007, 5, 20, "float32", 12, True, 0.1),
        # Prompts of eight requests through the down projection.
        _adapter("adapters_prompt_down", 4096, 14336, 4096, 8, 32, "float16", 8, False, 0.1),
        # Prompts of sixteen requests through the gate and up projection: the
        # widest output.
        _adapter("adapters_prompt_gateup", 4096, 4096, 28672, 16, 16, "float16", 16, False, 0.1),
        # A decoding batch's eight tokens: latency only.
        _norm("norms_decode", 8, 4096, "rms", "float32", "float32", "float16", 0, False),
        # A prompt's tokens between two blocks of a 4096-wide model.
        _norm("norms_prompt", 4096, 4096, "rms", "float32", "float32", "float16", 0, False),
        # Layer norms with biases, an odd width, a gate row for each sequence
        # of 100 tokens, a half-precision residual stream.
        _norm("norms_odd_layer", 777, 5003, "layer", "float16", "float32", "float32", 100, True),
        # A long batch at the widest row, with a gate for every channel.
        _norm("norms_wide", 4096, 16384, "rms", "float16", "float32", "float16", 4096, False),
        # A decoding batch's eight tokens between gate-up and down.
        _gated("gated_decode", 8, 14336, "silu", "float32", "float16", True),
        # A prompt's tokens between gate-up and down.
        _gated("gated_prompt", 4096, 14336, "silu", "float32", "float16", True),
        # Odd sizes, gate and up from two projections, full-precision output.
        _gated("gated_odd_gelu", 1001, 1407, "gelu", "float32", "float32", False),
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 0.999)))))))


def draw(rng):
    """One more case: any operator, sizes over the logarithm of their range."""
    op = rng.choice(["adapter_add", "adapter_add", "norm_residual", "gated_activation"])
    M = _log(rng, 1, 4096)
    if op == "adapter_add":
        dtype = rng.choice(["float16", "float16", "float32"])
        rank = 8 * _log(rng, 1, 16) if dtype == "float16" else _log(rng, 1, 64)
        K = 64 * _log(rng, 1, 224)
        N = _log(rng, 1, 28672 if M * K <= 4096 * 4096 else 4096)
        adapters = _log(rng, 1, max(1, min(64, 512 // rank)))
        case = _adapter("", M, K, N, adapters, rank, dtype, min(M, _log(rng, 1, 64)), rng.random() < 0.4,
                        rng.choice([0.0, 0.1, 0.5]))
    elif op == "norm_residual":
        C = _log(rng, 32, 16384)
        C = C if rng.random() < 0.3 else (C + 7) // 8 * 8
        M = min(M, 48_000_000 // C)  # no more bytes than the largest listed case, whatever the types
        case = _norm("", M, C, rng.choice(["rms", "layer"]), rng.choice(["float32", "float16"]),
                     rng.choice(["float32", "float32", "float16"]), rng.choice(["float16", "float32"]),
                     rng.choice([0, 0, 1, 37, 4096]), rng.random() < 0.5)
    else:
        F = _log(rng, 64, 14336)
        F = F if rng.random() < 0.3 else (F + 7) // 8 * 8
        case = _gated("", M, F, rng.choice(["silu", "gelu", "gelu_tanh"]), rng.choice(["float32", "float32", "float16"]),
                      rng.choice(["float16", "float16", "float32"]), rng.random() < 0.7)
    del case["name"]
    return case


# --------------------------------------------------------------------------
# Inputs
# --------------------------------------------------------------------------
def _dt(name):
    return getattr(torch, name)


def _activation(gen, M, K, dtype):
    """Normal values, four massive channels, the first row like a BOS token's."""
    x = torch.randn((M, K), generator=gen, device=DEV)
    x[:, 7 % K::max(1, K // 4)] *= 30.0
    x[0] *= 8.0
    return x.to(dtype)


def _index(case, seed):
    """The adapter of every token (-1: none), on the host as a scheduler makes it."""
    g = torch.Generator().manual_seed(seed * 3 + 1)
    M, L, R = case["M"], case["adapters"], case["requests"]
    cuts = torch.randperm(M - 1, generator=g)[:R - 1] + 1 if M > 1 else torch.zeros(0, dtype=torch.int64)
    request = torch.bucketize(torch.arange(M), cuts.sort().values, right=True)
    of = torch.randint(0, L, (R,), generator=g, dtype=torch.int32)
    of[torch.rand(R, generator=g) < case["none"]] = -1
    index = of[request]
    return index[torch.randperm(M, generator=g)] if case["mixed"] else index


def prepare(case, seed):
    gen = torch.Generator(device=DEV).manual_seed(seed)
    s = dict(case)
    if case["op"] == "adapter_add":
        M, K, N, L, R, dt = case["M"], case["K"], case["N"], case["adapters"], case["rank"], _dt(case["dtype"])
        s["x"] = _activation(gen, M, K, dt)
        s["y"] = torch.randn((M, N), generator=gen, device=DEV)
        s["At"] = (torch.randn((L, R, K), generator=gen, device=DEV) * K ** -0.5).to(dt)
        s["Bt"] = (torch.randn((L, N, R), generator=gen, device=DEV) * R ** -0.5).to(dt)
        g = torch.Generator().manual_seed(seed * 5 + 2)
        s["ranks"] = torch.randint((R + 1) // 2, R + 1, (L,), generator=g, dtype=torch.int32).to(DEV)
        s["scales"] = (0.5 + torch.rand((L,), generator=g)).to(DEV)
        s["index"] = _index(case, seed).to(DEV)
    elif case["op"] == "norm_residual":
        M, C = case["M"], case["C"]
        s["h"] = _activation(gen, M, C, _dt(case["h"]))
        s["y"] = (2.0 * torch.randn((M, C), generator=gen, device=DEV)).to(_dt(case["y"]))
        for name, on in (("post_weight", True), ("post_bias", case["bias"]), ("pre_weight", True), ("pre_bias", case["bias"])):
            v = (1.0 if "weight" in name else 0.0) + 0.1 * torch.randn((C,), generator=gen, device=DEV)
            s[name] = v.to(torch.float16) if on else None
        rows = -(-M // case["gate_rows"]) if case["gate_rows"] else 0
        s["gate"] = torch.randn((rows, C), generator=gen, device=DEV) if rows else None
        s["residual_scale"], s["eps"] = 0.7, 1e-5
    else:
        M, F = case["M"], case["F"]
        if case["joined"]:
            both = (2.0 * torch.randn((M, 2 * F), generator=gen, device=DEV)).to(_dt(case["src"]))
            s["gate"], s["up"] = both[:, :F], both[:, F:]
        else:
            s["gate"] = (2.0 * torch.randn((M, F), generator=gen, device=DEV)).to(_dt(case["src"]))
            s["up"] = (2.0 * torch.randn((M, F), generator=gen, device=DEV)).to(_dt(case["src"]))
    return s


# --------------------------------------------------------------------------
# One pass
# --------------------------------------------------------------------------
def _plain_adapter_add(s):
    """All adapters' products, those of other adapters and past the rank set to zero."""
    L, R, K = s["At"].shape
    t = (s["x"].float() @ s["At"].float().reshape(L * R, K).t()).reshape(-1, L, R)
    a = torch.arange(L, device=t.device)
    mine = (s["index"][:, None] == a)[:, :, None] & (torch.arange(R, device=t.device) < s["ranks"][:, None])
    t = torch.where(mine, t * s["scales"][:, None], 0.0)
    return s["y"] + t.reshape(-1, L * R) @ s["Bt"].float().permute(0, 2, 1).reshape(L * R, -1)


def _plain_norm(v, kind, weight, bias, eps):
    if kind == "layer":
        v = v - v.mean(dim=1, keepdim=True)
    v = v / torch.sqrt((v * v).mean(dim=1, keepdim=True) + eps) * weight.float()
    return v if bias is None else v + bias.float()


def _plain_norm_residual(s):
    v = s["residual_scale"] * _plain_norm(s["y"].float(), s["kind"], s["post_weight"], s["post_bias"], s["eps"])
    if s["gate"] is not None:
        v = v * s["gate"][torch.arange(v.shape[0], device=v.device) // s["gate_rows"]]
    h = s["h"].float() + v
    x = _plain_norm(h, s["kind"], s["pre_weight"], s["pre_bias"], s["eps"])
    return {"h": h.to(s["h"].dtype), "x": x.to(_dt(s["x"]))}


def _plain_gated(s):
    g, u = s["gate"].float(), s["up"].float()
    if s["act"] == "silu":
        g = g / (1.0 + torch.exp(-g))
    elif s["act"] == "gelu":
        g = 0.5 * g * (1.0 + torch.erf(g * math.sqrt(0.5)))
    else:
        g = 0.5 * g * (1.0 + torch.tanh(math.sqrt(2.0 / math.pi) * (g + 0.044715 * g * g * g)))
    return (g * u).to(_dt(s["dst"]))


def run(s):
    if not own:
        if s["op"] == "adapter_add":
            return _plain_adapter_add(s)
        return _plain_norm_residual(s) if s["op"] == "norm_residual" else _plain_gated(s)
    from bit_gemm_block_amd import block
    if s["op"] == "adapter_add":
        return block.adapter_add(s["y"], s["x"], s["At"], s["Bt"], s["index"], ranks=s["ranks"], scales=s["scales"])
    if s["op"] == "norm_residual":
        h, x = block.norm_residual(
            s["h"], s["y"], post_norm=s["kind"], post_weight=s["post_weight"], post_bias=s["post_bias"], gate=s["gate"],
            gate_rows=s["gate_rows"], residual_scale=s["residual_scale"], pre_norm=s["kind"],
            pre_weight=s["pre_weight"], pre_bias=s["pre_bias"], eps=s["eps"], x_dtype=_dt(s["x"]))
        return {"h": h, "x": x}
    return block.gated_activation(s["gate"], s["up"], s["act"], out_dtype=_dt(s["dst"]))


# --------------------------------------------------------------------------
# What a pass cannot do without, and its result in 64 bits
# --------------------------------------------------------------------------
def work(case):
    size = {"float32": 4, "float16": 2}
    M = case["M"]
    if case["op"] == "adapter_add":
        K, N, R, e = case["K"], case["N"], case["rank"], size[case["dtype"]]
        used = min(case["adapters"], case["requests"])
        return {"bytes": M * K * e + used * R * (K + N) * e + 8 * M * N + 4 * M, "flops": 2 * M * R * (K + N)}
    if case["op"] == "norm_residual":
        C = case["C"]
        rows = -(-M // case["gate_rows"]) if case["gate_rows"] else 0
        per = 2 * size[case["h"]] + size[case["y"]] + size[case["x"]]
        return {"bytes": M * C * per + 4 * rows * C + (8 if case["bias"] else 4) * C, "flops": 16 * M * C}
    F = case["F"]
    return {"bytes": M * F * (2 * size[case["src"]] + size[case["dst"]]), "flops": 8 * M * F}


def _exact_norm(v, case, w, b, eps):
    d = v - (v.sum(1) / v.shape[1])[:, None] if case["kind"] == "layer" else v
    r = (d.square().sum(1) / d.shape[1] + eps).rsqrt()
    d = d * r[:, None] * w.double()
    return d + b.double() if b is not None else d


def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "adapter_add":
        out = s["y"].double()
        index, ranks, scales = s["index"].tolist(), s["ranks"].tolist(), s["scales"].double().tolist()
        for a in sorted(set(index) - {-1}):
            rows = torch.nonzero(s["index"] == a).flatten()
            r = ranks[a]
            t = s["x"][rows].double() @ s["At"][a, :r].double().t().contiguous()
            out[rows] += scales[a] * (t @ s["Bt"][a, :, :r].double().t().contiguous())
        return out
    if case["op"] == "norm_residual":
        h = _exact_norm(s["y"].double(), case, s["post_weight"], s["post_bias"], s["eps"])
        if s["gate"] is not None:
            h *= s["gate"].double().repeat_interleave(case["gate_rows"], 0)[:case["M"]]
        h = s["h"].double() + s["residual_scale"] * h
        return {"h": h, "x": _exact_norm(h, case, s["pre_weight"], s["pre_bias"], s["eps"])}
    g, u = s["gate"].double(), s["up"].double()
    if case["act"] == "silu":
        return u * g * torch.sigmoid(g)
    if case["act"] == "gelu":
        return u * g * torch.special.ndtr(g)
    return u * g * torch.sigmoid(2.0 * math.sqrt(2.0 / math.pi) * (g + 0.044715 * g ** 3))
