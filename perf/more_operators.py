"""Cases of the experts' 4-bit path and of the layer for few tokens: microscaled 4-bit quantisation and its values back, the
experts' products on such operands, the gated activation between two products with its gradient, and the experts of a whole
layer for the tokens of a decode step.

``run`` computes them in plain torch when ``own`` is false, and through the package's public calls when it is true."""

from __future__ import annotations

import math

import torch

own = False

F8 = torch.float8_e4m3fn
WIDE = 128                                     # e4m3: one scale for 128 values (weights: 128 x 128)
NARROW = 32                                    # 4 bits: one scale for 32 values along the contraction
DTYPES = {"bf16": torch.bfloat16, "fp32": torch.float32}


def listed():
    return [
        # a prefill's inputs: token rows gathered in dispatch order and quantised for the first product; read back as bf16
        {"name": "fp4-rows-gather", "op": "quantize", "T": 8195, "k": 8, "E": 64, "K": 4096, "N": 0, "dtype": "bf16", "cf": 1.25},
        # weights quantised once for serving and, for a path without a 4-bit product, read back
        {"name": "fp4-weights", "op": "quantize", "T": 0, "k": 1, "E": 16, "K": 4096, "N": 2048, "dtype": "fp32", "cf": 1.0},
        # one token's experts: 8 rows, 8 of 64 weight matrices read once
        {"name": "fp4-product-decode", "op": "matmul", "T": 1, "k": 8, "E": 64, "K": 4096, "N": 2048, "out": "bf16", "cf": 64.0},
        # a serving batch: every expert has a few rows, the weights are what is read
        {"name": "fp4-product-serve", "op": "matmul", "T": 64, "k": 8, "E": 64, "K": 4096, "N": 2048, "out": "bf16", "cf": 4.0},
        # a prefill: about a thousand rows an expert
        {"name": "fp4-product-prefill", "op": "matmul", "T": 8192, "k": 8, "E": 64, "K": 4096, "N": 2048, "out": "bf16", "cf": 1.25},
        # a few experts, widths that end inside a block of 128, assignments dropped at the capacity, 32-bit result
        {"name": "fp4-product-odd", "op": "matmul", "T": 3001, "k": 2, "E": 8, "K": 1440, "N": 1040, "out": "fp32", "cf": 1.0},
        # a training step's activation and its gradient on the rows of 32 experts
        {"name": "glu-train", "op": "glu", "M": 32836, "I": 2048, "dtype": "bf16", "bwd": True},
        # between a prefill's two products: the activation written as the second one's 4-bit operand, and that product
        {"name": "glu-fp4-down", "op": "down", "T": 2048, "k": 8, "E": 64, "I": 2048, "N": 4096, "dtype": "bf16", "cf": 1.25},
        # one token of a decode step through 8 of 64 experts in 4 bits
        {"name": "layer-one-token", "op": "layer", "kind": "fp4", "T": 1, "k": 8, "E": 64, "H": 4096, "I": 2048},
        # a small decode batch: most experts have a token or two
        {"name": "layer-sixteen", "op": "layer", "kind": "fp4", "T": 16, "k": 8, "E": 64, "H": 4096, "I": 2048},
        # a speculative step's few tokens, a small layer with odd widths, 8-bit weights
        {"name": "layer-odd", "op": "layer", "kind": "e4m3", "T": 5, "k": 3, "E": 24, "H": 1424, "I": 1040},
        # the largest decode batch of the call, 8-bit weights
        {"name": "layer-largest", "op": "layer", "kind": "e4m3", "T": 64, "k": 8, "E": 64, "H": 4096, "I": 2048},
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["quantize", "matmul", "matmul", "glu", "down", "layer", "layer", "layer"])
    E, k = rng.choice([8, 16, 64, 96]), rng.randint(1, 8)
    cf = rng.choice([1.0, 1.25, 2.0])
    dtype = rng.choice(["bf16", "fp32"])
    if op == "quantize":
        if rng.random() < 0.4:
            return {"op": op, "T": 0, "k": 1, "E": rng.randint(1, 24), "K": 32 * _log(rng, 1, 128), "N": 16 * _log(rng, 1, 128), "dtype": dtype, "cf": 1.0}
        return {"op": op, "T": _log(rng, 1, 5000), "k": k, "E": E, "K": 32 * _log(rng, 1, 128), "N": 0, "dtype": dtype, "cf": cf}
    if op == "matmul":
        return {"op": op, "T": _log(rng, 1, 6000), "k": k, "E": rng.choice([1, 8, 16, 64]) if k == 1 else E, "K": 32 * _log(rng, 2, 128), "N": 16 * _log(rng, 2, 128),
                "out": dtype, "cf": cf}
    if op == "glu":
        return {"op": op, "M": _log(rng, 1, 30000), "I": 16 * _log(rng, 1, 128), "dtype": dtype, "bwd": rng.random() < 0.6}
    if op == "down":
        return {"op": op, "T": _log(rng, 1, 2000), "k": k, "E": E, "I": 32 * _log(rng, 2, 64), "N": 16 * _log(rng, 4, 256), "dtype": dtype, "cf": cf}
    kind, E = rng.choice(["fp4", "e4m3"]), rng.choice([8, 24, 64])
    step = 32 if kind == "fp4" else 16
    return {"op": op, "kind": kind, "T": _log(rng, 1, 64), "k": k, "E": E, "H": step * _log(rng, 2, 4096 // step), "I": step * _log(rng, 2, 2048 // step)}


# -- inputs ------------------------------------------------------------------

def _routing(T, E, k, cf, gen):
    """A seeded skewed routing of T tokens to k of E experts and its capacity-limited dispatch: the arrays that the dispatch call gives."""
    w = -0.35 * torch.log(1.0 + torch.randperm(E, generator=gen, device="cuda").float())
    u = torch.rand(T, E, generator=gen, device="cuda").clamp_(1e-7, 1 - 1e-7)
    idx = (w - torch.log(-torch.log(u))).topk(k, dim=1).indices.to(torch.int32)
    flat = idx.reshape(-1).long()
    cap = math.ceil(-(-T * k // E) * cf)
    counts = torch.bincount(flat, minlength=E)
    offsets = torch.zeros(E + 1, dtype=torch.int32, device="cuda")
    offsets[1:] = counts.cumsum(0)
    return {"idx": idx, "perm": torch.argsort(flat, stable=True).to(torch.int32), "offsets": offsets, "kept": counts.clamp(max=cap).to(torch.int32),
            "most": int(counts.clamp(max=cap).max())}


def _activations(rows, cols, gen, dtype=torch.bfloat16):
    """Rows of unequal size with a few large channels, as hidden states have them."""
    x = torch.randn(rows, cols, generator=gen, device="cuda")
    x *= torch.exp(0.5 * torch.randn(rows, 1, generator=gen, device="cuda"))
    x *= torch.exp(0.7 * torch.randn(1, cols, generator=gen, device="cuda"))
    return x.to(dtype)


def _fp4_codes(x):
    """Codes [M, K/2] (two values a byte, the even column low) and scale codes [ceil(K/128), M, 4] of x's blocks of 32: a code s
    stands for 2^(s - 127), and the block's largest value over it lies in (3, 6]; a block of zeros has 127."""
    M, K = x.shape
    v = x.float().view(M, K // NARROW, NARROW)
    amax = v.abs().amax(2)
    m, e = torch.frexp(amax)
    s = torch.where(amax == 0, torch.full_like(e, 127), (e - 3 + (m > 0.75) + 127).clamp(min=1))
    v = v / (s << 23).view(torch.float32)[:, :, None]
    a = v.abs()
    code = (a > 0.25).to(torch.uint8)          # halfway between two values: the one with the even code
    code += a >= 0.75
    code += a > 1.25
    code += a >= 1.75
    code += a > 2.5
    code += a >= 3.5
    code += a > 5.0
    code = (code + 8 * torch.signbit(v).to(torch.uint8)).view(M, K // 2, 2)
    words = torch.full((M, -(-K // WIDE) * 4), 127, dtype=torch.uint8, device=x.device)
    words[:, :K // NARROW] = s.to(torch.uint8)
    return (code[:, :, 0] + 16 * code[:, :, 1]).contiguous(), words.view(M, -1, 4).transpose(0, 1).contiguous()


def _fp4_values(q, scale):
    """fp32 values [M, K] of codes and scale codes (1 to 254) as above."""
    M, K = q.shape[0], 2 * q.shape[1]
    half = torch.tensor([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0], device=q.device)
    sixteen = torch.cat([half, -half])
    pairs = torch.stack([sixteen.repeat(16), sixteen.repeat_interleave(16)], 1)
    s = (scale.int() << 23).view(torch.float32).transpose(0, 1).reshape(M, -1)[:, :K // NARROW]
    return (pairs[q.int()].view(M, -1, NARROW) * s[:, :, None]).view(M, K)


def _pow2_scale(amax):
    """The power of two s with amax / s in (224, 448]; 1 for a block of zeros."""
    m, e = torch.frexp(amax)
    s = torch.ldexp(torch.ones_like(amax), (e - 9 + (m > 0.875)).clamp(min=-126))
    return torch.where(amax == 0, torch.ones_like(s), s)


def _e4m3_weight(w):
    """Codes [N, K] and scales [ceil(N/128), ceil(K/128)] of blocks of 128 x 128."""
    N, K = w.shape
    pad = torch.nn.functional.pad(w, (0, -K % WIDE, 0, -N % WIDE)).view(-(-N // WIDE), WIDE, -(-K // WIDE), WIDE)
    scale = _pow2_scale(pad.abs().amax((1, 3)))
    q = (pad / scale[:, None, :, None]).to(F8).reshape(pad.shape[0] * WIDE, -1)[:N, :K]
    return q, scale


def _e4m3_values(q, scale):
    """fp32 values [E, N, K] of codes and scales [E, ceil(N/128), ceil(K/128)]."""
    E, N, K = q.shape
    wide = scale.repeat_interleave(WIDE, 1)[:, :N].repeat_interleave(WIDE, 2)[:, :, :K]
    return q.float() * wide


def _weights(kind, E, N, K, gen):
    """E experts' quantised weights [N, K]."""
    if kind == "fp4":
        q = torch.empty(E, N, K // 2, dtype=torch.uint8, device="cuda")
        scale = torch.empty(-(-K // WIDE), E, N, 4, dtype=torch.uint8, device="cuda")
        for e in range(E):
            q[e], scale[:, e] = _fp4_codes(torch.randn(N, K, generator=gen, device="cuda") / K ** 0.5)
    else:
        q = torch.empty(E, N, K, dtype=F8, device="cuda")
        scale = torch.empty(E, -(-N // WIDE), -(-K // WIDE), device="cuda")
        for e in range(E):
            q[e], scale[e] = _e4m3_weight(torch.randn(N, K, generator=gen, device="cuda") / K ** 0.5)
    return {"q": q, "scale": scale}


def prepare(case, seed):
    c = case
    gen = torch.Generator(device="cuda").manual_seed(int(seed))
    s = {"case": c}
    if c["op"] == "quantize":
        if c["N"]:
            s["x"] = (0.02 * torch.randn(c["E"], c["N"], c["K"], generator=gen, device="cuda")).to(DTYPES[c["dtype"]])
        else:
            s["r"] = _routing(c["T"], c["E"], c["k"], c["cf"], gen)
            s["x"] = _activations(c["T"], c["K"], gen, DTYPES[c["dtype"]])
        return s
    if c["op"] == "glu":
        s["h"] = _activations(c["M"], 2 * c["I"], gen, DTYPES[c["dtype"]])
        s["dy"] = (0.01 * torch.randn(c["M"], c["I"], generator=gen, device="cuda")).to(DTYPES[c["dtype"]])
        return s
    if c["op"] == "layer":
        s["idx"] = _routing(c["T"], c["E"], c["k"], 1.0, gen)["idx"]
        g = torch.rand(c["T"], c["k"], generator=gen, device="cuda") + 0.05
        s["gate"] = g / g.sum(1, keepdim=True)
        s["x"] = _activations(c["T"], c["H"], gen)
        s["w1"] = _weights(c["kind"], c["E"], 2 * c["I"], c["H"], gen)
        s["w2"] = _weights(c["kind"], c["E"], c["H"], c["I"], gen)
        return s
    s["r"] = _routing(c["T"], c["E"], c["k"], c["cf"], gen)
    M = c["T"] * c["k"]
    if c["op"] == "matmul":
        s["q"], s["scale"] = _fp4_codes(_activations(M, c["K"], gen))
        s["w"] = _weights("fp4", c["E"], c["N"], c["K"], gen)
        s["y"] = torch.zeros(M, c["N"], dtype=DTYPES[c["out"]], device="cuda")     # the rows of dropped assignments stay as they are
    else:
        s["h"] = _activations(M, 2 * c["I"], gen, DTYPES[c["dtype"]])
        s["w"] = _weights("fp4", c["E"], c["N"], c["I"], gen)
        s["y"] = torch.zeros(M, c["N"], dtype=torch.bfloat16, device="cuda")       # as above
    return s


# -- the plain forms and the package's calls -----------------------------------

def run(s):
    c = s["case"]
    return {"quantize": _quantize, "matmul": _matmul, "glu": _glu, "down": _down, "layer": _layer}[c["op"]](s, c)


def _quantize(s, c):
    x = s["x"]
    if own:
        import moe_expert_routing_router_gb300 as mr
        o = mr.moe_quantize_fp4(x) if c["N"] else mr.moe_quantize_fp4(x, perm=s["r"]["perm"], k=c["k"])
        return mr.moe_dequantize_fp4(o["q"], o["scale"])
    rows = x.view(-1, c["K"]) if c["N"] else x[s["r"]["perm"].long() // c["k"]]
    return _fp4_values(*_fp4_codes(rows)).to(torch.bfloat16).view(*x.shape[:-2], -1, c["K"])


def _expert_values(w):
    """fp32 values [E, N, K] of 4-bit or 8-bit weights."""
    q, scale = w["q"], w["scale"]
    if q.dtype != torch.uint8:
        return _e4m3_values(q, scale)
    E, N, half = q.shape
    return _fp4_values(q.reshape(E * N, half), scale.reshape(scale.shape[0], E * N, 4)).view(E, N, 2 * half)


def _experts(a, w, r, y):
    """The rows of every expert times its weights, written to y."""
    i = torch.arange(r["most"], device=y.device)[None, :]
    live = i < r["kept"].long()[:, None]
    rows = torch.where(live, r["offsets"][:-1].long()[:, None] + i, torch.zeros_like(i))
    y[rows[live]] = torch.bmm(a[rows], w.transpose(1, 2))[live].to(y.dtype)
    return y


def _matmul(s, c):
    r = s["r"]
    if own:
        import moe_expert_routing_router_gb300 as mr
        return mr.moe_expert_matmul_fp4(s["q"], s["scale"], s["w"]["q"], s["w"]["scale"], r["offsets"], r["kept"], out=s["y"])
    return _experts(_fp4_values(s["q"], s["scale"]), _expert_values(s["w"]), r, s["y"])


def _gated(h):
    I = h.shape[-1] // 2
    g = h[..., :I].float()
    return g / (1.0 + torch.exp(-g)) * h[..., I:].float()


def _glu(s, c):
    h, dy = s["h"], s["dy"]
    if own:
        import moe_expert_routing_router_gb300 as mr
        out = {"y": mr.moe_expert_glu(h)}
        if c["bwd"]:
            out["dh"] = mr.moe_expert_glu_bwd(h, dy)
        return out
    out = {"y": _gated(h).to(h.dtype)}
    if c["bwd"]:
        g, u, d = h[:, :c["I"]].float(), h[:, c["I"]:].float(), dy.float()
        sg = 1.0 / (1.0 + torch.exp(-g))
        out["dh"] = torch.cat([d * u * sg * (1.0 + g * (1.0 - sg)), d * g * sg], 1).to(h.dtype)
    return out


def _down(s, c):
    r = s["r"]
    if own:
        import moe_expert_routing_router_gb300 as mr
        a = mr.moe_expert_glu(s["h"], form="fp4")
        return mr.moe_expert_matmul_fp4(a["q"], a["scale"], s["w"]["q"], s["w"]["scale"], r["offsets"], r["kept"], out=s["y"])
    return _experts(_fp4_values(*_fp4_codes(_gated(s["h"]))), _expert_values(s["w"]), r, s["y"])


def _layer(s, c):
    x, idx, gate, w1, w2 = s["x"], s["idx"], s["gate"], s["w1"], s["w2"]
    if own:
        import moe_expert_routing_router_gb300 as mr
        return mr.moe_layer_small(x, idx, gate, w1, w2)
    e = torch.unique(idx).long()                                          # the experts that have tokens
    share = (gate[:, :, None] * (idx[:, :, None] == e)).sum(1)            # [T, experts]

    def pick(w):
        return {"q": w["q"].view(torch.uint8)[e].view(w["q"].dtype), "scale": w["scale"][:, e] if c["kind"] == "fp4" else w["scale"][e]}

    h = torch.matmul(x.float()[None], _expert_values(pick(w1)).transpose(1, 2))
    y = torch.matmul(_gated(h), _expert_values(pick(w2)).transpose(1, 2))  # [experts, T, H]
    return (y * share.t()[:, :, None]).sum(0).to(x.dtype)


# -- the definitions in 64 bits --------------------------------------------------

def exact(case, seed):
    c, s = case, prepare(case, seed)
    if c["op"] == "quantize":
        x = s["x"]
        if not c["N"]:
            x = x[torch.div(s["r"]["perm"], c["k"], rounding_mode="floor")]
        return _exact_round(x.double())
    if c["op"] == "glu":
        I = c["I"]
        g, u = s["h"][:, :I].double(), s["h"][:, I:].double()
        out = {"y": g * torch.sigmoid(g) * u}
        if c["bwd"]:
            dh, d = torch.empty_like(s["h"], dtype=torch.float64), s["dy"].double()
            dh[:, I:] = d * (g * torch.sigmoid(g))
            dh[:, :I] = d * u * (torch.sigmoid(g) + g * torch.sigmoid(g) * torch.sigmoid(-g))
            out["dh"] = dh
        return out
    if c["op"] == "layer":
        T, I = c["T"], c["I"]
        out = torch.zeros(T, c["H"], dtype=torch.float64, device="cuda")
        for e in range(c["E"]):
            t, j = torch.nonzero(s["idx"] == e, as_tuple=True)
            if len(t):
                h = s["x"][t].double() @ _exact_weight(s["w1"], e).t()
                act = h[:, :I] * torch.sigmoid(h[:, :I]) * h[:, I:]
                out.index_add_(0, t, s["gate"][t, j].double()[:, None] * (act @ _exact_weight(s["w2"], e).t()))
        return out
    out, first, kept = s["y"].double(), s["r"]["offsets"].tolist(), s["r"]["kept"].tolist()
    if c["op"] == "down":
        h = s["h"].double()
        a = _exact_round(h[:, :c["I"]] * torch.sigmoid(h[:, :c["I"]]) * h[:, c["I"]:])
    else:
        a = _exact_read(s["q"], s["scale"])
    for e in range(c["E"]):
        if kept[e]:
            at = slice(first[e], first[e] + kept[e])
            out[at] = a[at] @ _exact_weight(s["w"], e).t()
    return out


def _exact_round(x):
    """x as its 4-bit blocks give it back: s times the nearest of 0, 1/2, 1, 3/2, 2, 3, 4, 6, s the least power of two with |x| <= 6 s."""
    v = x.reshape(-1, NARROW)
    top = v.abs().amax(1, keepdim=True)
    some = torch.where(top > 0, top, torch.full_like(top, 6.0))
    n = torch.ceil(torch.log2(some / 6.0))
    n = torch.where(6.0 * torch.exp2(n - 1) >= some, n - 1, n)
    n = torch.where(6.0 * torch.exp2(n) < some, n + 1, n).clamp(min=-126)
    v = v / torch.exp2(n)
    step = torch.exp2(torch.floor(torch.log2(v.abs().clamp(min=1.0))) - 1)   # half of a value's binade; ties go to the even multiple
    return (torch.round(v / step) * step * torch.exp2(n)).view(x.shape)


def _exact_read(q, scale):
    """float64 values of 4-bit codes [M, K/2] with scale codes [ceil(K/128), M, 4]."""
    M, K = q.shape[0], 2 * q.shape[1]
    out = torch.empty(M, K, dtype=torch.float64, device="cuda")
    for odd in (0, 1):
        code = torch.div(q, 16, rounding_mode="floor") if odd else q % 16
        sign, exponent, fraction = code >= 8, torch.div(code % 8, 2, rounding_mode="floor").double(), (code % 2).double()
        size = torch.where(exponent == 0, fraction / 2, torch.exp2(exponent - 1) * (1 + fraction / 2))
        out[:, odd::2] = torch.where(sign, -size, size)
    for b in range(K // NARROW):
        out[:, b * NARROW:(b + 1) * NARROW] *= torch.exp2(scale[b // 4, :, b % 4].double() - 127)[:, None]
    return out


def _exact_weight(w, e):
    if w["q"].dtype == torch.uint8:
        return _exact_read(w["q"][e], w["scale"][:, e])
    v = w["q"][e].double()
    for i in range(w["scale"].shape[1]):
        for j in range(w["scale"].shape[2]):
            v[i * WIDE:(i + 1) * WIDE, j * WIDE:(j + 1) * WIDE] *= w["scale"][e, i, j].double()
    return v


# -- what a pass cannot do without -------------------------------------------------

def _busy(T, k, E):
    """Experts that a routing as above gives tokens, on average: expert r is among a token's k with probability 1 - exp(-a (1+r)^-0.35),
    a such that these sum to k."""
    w = [(1 + r) ** -0.35 for r in range(E)]
    if k >= E:
        return float(E)
    lo, hi = 0.0, 1e3
    for _ in range(60):
        a = (lo + hi) / 2
        lo, hi = (a, hi) if sum(1 - math.exp(-a * v) for v in w) < k else (lo, a)
    return sum(1 - math.exp(-lo * v * T) for v in w)


def work(case):
    c = case
    if c["op"] == "glu":
        size, n = 2 if c["dtype"] == "bf16" else 4, c["M"] * c["I"]
        return {"bytes": n * size * (8 if c["bwd"] else 3), "flops": n * (20 if c["bwd"] else 6)}    # the gradient reads h once more
    if c["op"] == "quantize":
        size = 2 if c["dtype"] == "bf16" else 4
        rows = c["E"] * c["N"] if c["N"] else c["T"] * c["k"]
        read = rows if c["N"] else c["T"]
        return {"bytes": c["K"] * (read * size + rows * (2 * 17 / 32 + 2)), "flops": 3 * rows * c["K"]}   # codes and scales are written, and read back
    if c["op"] == "layer":
        size, n = 17 / 32 if c["kind"] == "fp4" else 1.0, 3 * c["H"] * c["I"]
        return {"bytes": _busy(c["T"], c["k"], c["E"]) * n * size + 4 * c["T"] * c["H"] + 8 * c["T"] * c["k"], "flops": 2 * c["T"] * c["k"] * n}
    M, K = c["T"] * c["k"], c["K"] if c["op"] == "matmul" else c["I"]
    live = _busy(c["T"], c["k"], c["E"])
    size = 4 if c["op"] == "matmul" and c["out"] == "fp32" else 2
    a = 17 / 32 if c["op"] == "matmul" else 2 * (2 if c["dtype"] == "bf16" else 4)
    return {"bytes": M * K * a + live * c["N"] * K * 17 / 32 + M * c["N"] * size, "flops": 2 * M * K * c["N"]}
