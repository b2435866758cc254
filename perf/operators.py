"""Cases of the mixture-of-experts layer's operators behind the router: scored group-limited routing with its gradient,
block-scaled 8-bit quantisation, the experts' 8-bit matrix products (forward and weight gradient) and the gated combine.

``run`` computes them in plain torch when ``own`` is false, and through the package's public calls when it is true."""

from __future__ import annotations

import math

import numpy as np
import torch

own = False

F8 = torch.float8_e4m3fn
BLOCK = 128                                    # one scale stands for a block of 128
DTYPES = {"bf16": torch.bfloat16, "fp32": torch.float32}


def listed():
    return [
        # one token of a decode step: sigmoid scores, a balance bias, 4 of 8 expert groups, 8 picks
        {"name": "route-decode", "op": "route", "T": 1, "E": 256, "k": 8, "dtype": "bf16", "score": "sigmoid", "bias": True,
         "groups": 8, "keep": 4, "group_score": "top2", "renorm": True, "scale": 2.5, "bwd": False},
        # a training step's whole batch: the same routing with its bias update and gradient
        {"name": "route-train", "op": "route", "T": 131072, "E": 256, "k": 8, "dtype": "bf16", "score": "sigmoid", "bias": True,
         "groups": 8, "keep": 4, "group_score": "top2", "renorm": True, "scale": 2.5, "bwd": True},
        # fp32 logits, softmax scores taken as they are (dense gradient), the best group by its largest score, odd length
        {"name": "route-softmax-odd", "op": "route", "T": 16381, "E": 384, "k": 6, "dtype": "fp32", "score": "softmax", "bias": False,
         "groups": 12, "keep": 5, "group_score": "max", "renorm": False, "scale": 16.0, "bwd": True},
        # the experts' inputs of a prefill: token rows gathered in dispatch order and quantised for the first product
        {"name": "quantize-gather", "op": "quantize", "form": "rows", "T": 8195, "k": 8, "E": 64, "K": 4096, "dtype": "bf16", "gather": True, "cf": 1.25},
        # a gradient's rows quantised along the tokens, every expert's rows padded to whole blocks: the weight gradient's operand
        {"name": "quantize-cols", "op": "quantize", "form": "cols", "T": 5003, "k": 6, "E": 64, "K": 2048, "dtype": "bf16", "gather": False, "cf": 1.25},
        # one token's experts: 8 rows, 8 of 64 weight matrices read once
        {"name": "experts-decode", "op": "matmul", "T": 1, "k": 8, "E": 64, "K": 4096, "N": 2048, "out": "bf16", "cf": 64.0},
        # a serving batch: every expert has a few rows, the weights are what is read
        {"name": "experts-serve", "op": "matmul", "T": 64, "k": 8, "E": 64, "K": 4096, "N": 2048, "out": "bf16", "cf": 4.0},
        # a prefill: about a thousand rows an expert
        {"name": "experts-prefill", "op": "matmul", "T": 8192, "k": 8, "E": 64, "K": 4096, "N": 2048, "out": "bf16", "cf": 1.25},
        # a few experts, widths that end inside a block, assignments dropped at the capacity, 32-bit result
        {"name": "experts-odd", "op": "matmul", "T": 3001, "k": 2, "E": 8, "K": 1424, "N": 1040, "out": "fp32", "cf": 1.0},
        # the weight gradient of a training step: a contraction over every expert's own rows
        {"name": "experts-wgrad", "op": "wgrad", "T": 8209, "k": 4, "E": 32, "K": 2048, "N": 2048, "cf": 1.25},
        # the experts' rows of a few decoded tokens gathered back and summed by gate
        {"name": "combine-decode", "op": "combine", "T": 16, "k": 8, "E": 64, "H": 4096, "dtype": "bf16", "cf": 2.0, "bwd": False},
        # a training step's combine with its gradients, some assignments dropped
        {"name": "combine-train", "op": "combine", "T": 16384, "k": 6, "E": 64, "H": 2048, "dtype": "bf16", "cf": 1.0, "bwd": True},
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["route", "route", "quantize", "quantize", "matmul", "matmul", "wgrad", "combine"])
    if op == "route":
        groups = rng.choice([1, 2, 4, 6, 8, 12])
        E = groups * rng.randint(3, 384 // groups)
        keep = rng.randint(max(1, groups // 3), groups)
        k = rng.randint(1, min(8, keep * (E // groups)))
        score = rng.choice(["sigmoid", "softmax"])
        return {"op": op, "T": _log(rng, 1, 100000), "E": E, "k": k, "dtype": rng.choice(["bf16", "fp32"]), "score": score, "bias": rng.random() < 0.6,
                "groups": groups, "keep": keep, "group_score": rng.choice(["top2", "max"]), "renorm": rng.random() < 0.6,
                "scale": rng.choice([1.0, 2.5, 16.0]), "bwd": rng.random() < 0.7}
    E, k = rng.choice([8, 16, 64, 96]), rng.randint(1, 8)
    cf = rng.choice([1.0, 1.25, 2.0])
    if op == "quantize":
        form = rng.choice(["rows", "cols", "weights"])
        if form == "weights":
            return {"op": op, "form": form, "T": rng.randint(1, 9), "k": 1, "E": rng.randint(1, 24), "K": 16 * _log(rng, 8, 256), "N": 16 * _log(rng, 8, 128),
                    "dtype": rng.choice(["bf16", "fp32"]), "gather": False, "cf": cf}
        return {"op": op, "form": form, "T": _log(rng, 1, 5000), "k": k, "E": E, "K": 16 * _log(rng, 4, 256), "dtype": rng.choice(["bf16", "fp32"]),
                "gather": rng.random() < 0.5, "cf": cf}
    if op == "matmul":
        return {"op": op, "T": _log(rng, 1, 6000), "k": k, "E": rng.choice([1, 8, 16, 64]) if k == 1 else E, "K": 16 * _log(rng, 8, 256), "N": 16 * _log(rng, 4, 128),
                "out": rng.choice(["bf16", "fp32"]), "cf": cf}
    if op == "wgrad":
        return {"op": op, "T": _log(rng, 1, 4000), "k": k, "E": rng.choice([8, 16, 32]), "K": 16 * _log(rng, 8, 128), "N": 16 * _log(rng, 8, 128), "cf": cf}
    return {"op": op, "T": _log(rng, 1, 8000), "k": k, "E": E, "H": rng.choice([_log(rng, 64, 4096), 16 * _log(rng, 4, 256)]), "dtype": rng.choice(["bf16", "fp32"]),
            "cf": cf, "bwd": rng.random() < 0.6}


# -- inputs ------------------------------------------------------------------

def _routing(T, E, k, cf, gen):
    """A seeded skewed routing of T tokens to k of E experts and its capacity-limited dispatch: the arrays that the dispatch call gives."""
    w = -0.35 * torch.log(1.0 + torch.randperm(E, generator=gen, device="cuda").float())
    u = torch.rand(T, E, generator=gen, device="cuda").clamp_(1e-7, 1 - 1e-7)
    idx = (w - torch.log(-torch.log(u))).topk(k, dim=1).indices.to(torch.int32)
    flat = idx.reshape(-1).long()
    cap = math.ceil(-(-T * k // E) * cf)
    perm = torch.argsort(flat, stable=True)
    counts = torch.bincount(flat, minlength=E)
    offsets = torch.zeros(E + 1, dtype=torch.int64, device="cuda")
    offsets[1:] = counts.cumsum(0)
    rank = torch.arange(T * k, device="cuda") - offsets[flat[perm]]
    slot = torch.empty(T * k, dtype=torch.int64, device="cuda")
    slot[perm] = torch.where(rank < cap, rank, torch.full_like(rank, -1))
    i32 = torch.int32
    return {"idx": idx, "perm": perm.to(i32), "slot": slot.to(i32), "offsets": offsets.to(i32), "kept": counts.clamp(max=cap).to(i32),
            "most": int(counts.clamp(max=cap).max())}


def _activations(rows, cols, gen, dtype=torch.bfloat16):
    """Rows of unequal size with a few large channels, as hidden states have them."""
    x = torch.randn(rows, cols, generator=gen, device="cuda")
    x *= torch.exp(0.5 * torch.randn(rows, 1, generator=gen, device="cuda"))
    x *= torch.exp(0.7 * torch.randn(1, cols, generator=gen, device="cuda"))
    return x.to(dtype)


def _pow2_scale(amax):
    """The power of two s with amax / s in (224, 448], the largest e4m3 value; 1 for a block of zeros, NaN for one that is not finite."""
    m, e = torch.frexp(amax)
    s = torch.ldexp(torch.ones_like(amax), (e - 9 + (m > 0.875)).clamp(min=-126))
    return torch.where(amax == 0, torch.ones_like(s), torch.where(amax.isfinite(), s, torch.full_like(s, math.nan)))


def _quantize_rows(x):
    """q [M, K] e4m3 and scale [ceil(K/128), M] of x's blocks of one row by 128 columns."""
    M, K = x.shape
    pad = torch.nn.functional.pad(x.float(), (0, -K % BLOCK)).view(M, -1, BLOCK)
    scale = _pow2_scale(pad.abs().amax(2))
    q = (pad / scale[:, :, None]).to(F8).view(M, -1)[:, :K].contiguous()
    return q, scale.t().contiguous()


def _quantize_weights(w):
    """q [E, N, K] e4m3 and scale [E, ceil(N/128), ceil(K/128)] of w's blocks of 128 by 128."""
    E, N, K = w.shape
    pad = torch.nn.functional.pad(w.float(), (0, -K % BLOCK, 0, -N % BLOCK))
    pad = pad.view(E, (N + BLOCK - 1) // BLOCK, BLOCK, (K + BLOCK - 1) // BLOCK, BLOCK)
    scale = _pow2_scale(pad.abs().amax((2, 4)))
    q = (pad / scale[:, :, None, :, None]).to(F8).reshape(E, pad.shape[1] * BLOCK, -1)[:, :N, :K].contiguous()
    return q, scale.contiguous()


def _columns(r, M, E, most):
    """Where the padded layout along the tokens keeps expert e's i-th row: the rows [E, C] they come from (M where there is none) and their columns."""
    blocks = (r["kept"].long() + BLOCK - 1) // BLOCK
    first = (blocks.cumsum(0) - blocks) * BLOCK
    C = -(-max(most, 1) // BLOCK) * BLOCK
    i = torch.arange(C, device="cuda")[None, :]
    rows = torch.where(i < r["kept"].long()[:, None], r["offsets"][:-1].long()[:, None] + i, torch.full_like(i, M))
    cols = first[:, None] + i
    return rows, cols, i < (blocks * BLOCK)[:, None]


def _width(M, E):
    return BLOCK * ((M + (BLOCK - 1) * E) // BLOCK)


def _quantize_cols(x, r, token, q, scale):
    """Writes q [K, width] e4m3 and scale [width/128, K]: blocks of 128 of an expert's rows by one column, the ends padded with zeros."""
    K, M, E = x.shape[1], token.numel(), r["kept"].numel()
    rows, cols, live = _columns(r, M, E, r["most"])
    xs = torch.cat([x, torch.zeros_like(x[:1])])                         # a row of zeros behind the last
    src = torch.cat([token, token.new_full((1,), x.shape[0])])
    at, cat = rows[live], cols[live]                                     # whole blocks of live columns
    v = xs[src[at]].float().view(-1, BLOCK, K)
    s = _pow2_scale(v.abs().amax(1))
    q.t()[cat] = (v / s[:, None, :]).to(F8).view(-1, K)
    scale[cat[::BLOCK] // BLOCK] = s
    return q, scale


def prepare(case, seed):
    c = case
    gen = torch.Generator(device="cuda").manual_seed(int(seed))
    s = {"case": c}
    if c["op"] == "route":
        z = 1.2 * torch.randn(c["T"], c["E"], generator=gen, device="cuda") - 0.5
        s["logits"] = (z + 0.8 * torch.randn(c["E"], generator=gen, device="cuda")).to(DTYPES[c["dtype"]])
        # a bias that updates of 0.001 have led to
        s["bias"] = 0.001 * torch.randint(-150, 151, (c["E"],), generator=gen, device="cuda").float() if c["bias"] else None
        s["dgate"] = torch.randn(c["T"], c["k"], generator=gen, device="cuda")
        return s
    if c["op"] == "quantize" and c["form"] == "weights":
        s["w"] = (torch.randn(c["E"], c["N"], c["K"], generator=gen, device="cuda") * 0.02).to(DTYPES[c["dtype"]])
        return s
    r = s["r"] = _routing(c["T"], c["E"], c["k"], c["cf"], gen)
    M = c["T"] * c["k"]
    if c["op"] == "quantize":
        s["x"] = _activations(c["T"] if c["gather"] else M, c["K"], gen, DTYPES[c["dtype"]])
        if c["form"] == "cols":                                          # its columns behind the last expert's stay as they are
            s["q"] = torch.zeros(c["K"], _width(M, c["E"]), device="cuda").to(F8)
            s["scale"] = torch.zeros(_width(M, c["E"]) // BLOCK, c["K"], device="cuda")
    elif c["op"] == "matmul":
        s["q"], s["scale"] = _quantize_rows(_activations(M, c["K"], gen))
        s["wq"], s["wscale"] = _quantize_weights(torch.randn(c["E"], c["N"], c["K"], generator=gen, device="cuda") * 0.02)
        # the rows of dropped assignments stay as they are
        s["y"] = torch.zeros(M, c["N"], dtype=DTYPES[c["out"]], device="cuda")
    elif c["op"] == "wgrad":
        token = torch.arange(M, device="cuda")
        for name, cols, sigma in (("dy", c["N"], 0.01), ("x", c["K"], 1.0)):
            q = torch.zeros(cols, _width(M, c["E"]), device="cuda").to(F8)
            scale = torch.ones(_width(M, c["E"]) // BLOCK, cols, device="cuda")
            s[name + "q"], s[name + "scale"] = _quantize_cols(_activations(M, cols, gen) * sigma, r, token, q, scale)
    else:
        dt = DTYPES[c["dtype"]]
        s["y"] = torch.randn(M, c["H"], generator=gen, device="cuda").to(dt)
        g = torch.rand(c["T"], c["k"], generator=gen, device="cuda") + 0.05
        s["gate"] = g / g.sum(1, keepdim=True)
        s["dout"] = torch.randn(c["T"], c["H"], generator=gen, device="cuda").to(dt)
        s["dy"] = torch.zeros(M, c["H"], dtype=dt, device="cuda")        # as above
    return s


# -- the plain forms and the package's calls -----------------------------------

def run(s):
    c = s["case"]
    return {"route": _route, "quantize": _quantize, "matmul": _matmul, "wgrad": _wgrad, "combine": _combine}[c["op"]](s, c)


def _route(s, c):
    z, b, k, G = s["logits"], s["bias"], c["k"], c["groups"]
    if own:
        import moe_expert_routing_router_gb300 as mr
        r = mr.moe_route_fwd(z, k, score=c["score"], bias=b, n_groups=G, topk_groups=c["keep"], group_score=c["group_score"],
                             renorm=c["renorm"], scale=c["scale"], bias_gamma=0.001, bias_out=c["bias"])
        out = {"idx": r["idx"], "gate": r["gate"], "counts": r["counts"]}
        if c["bias"]:
            out["bias"] = r["bias_out"]
        if c["bwd"]:
            out["dlogits"] = mr.moe_route_bwd(z, r["idx"], s["dgate"], score=c["score"], renorm=c["renorm"], scale=c["scale"])
        return out
    T, E = z.shape
    zd = z.double()                            # scores next to one another decide picks: in 64 bits
    if c["score"] == "sigmoid":
        sd = 1.0 / (1.0 + torch.exp(-zd))
    else:
        p = torch.exp(zd - zd.amax(1, keepdim=True))
        sd = p / p.sum(1, keepdim=True)
    choice = sd + b.double() if b is not None else sd
    order = choice if b is not None else zd    # without a bias the scores are in the logits' order
    per = choice.view(T, G, E // G).sort(dim=2, descending=True).values
    per = per[:, :, :2].sum(2) if c["group_score"] == "top2" else order.view(T, G, E // G).amax(2)
    best = per.sort(dim=1, descending=True, stable=True).indices[:, :c["keep"]]
    open_ = torch.zeros(T, G, dtype=torch.bool, device=z.device).scatter_(1, best, True)
    order = torch.where(open_.repeat_interleave(E // G, 1), order, torch.full_like(order, -math.inf))
    idx = order.sort(dim=1, descending=True, stable=True).indices[:, :k]
    zf = z.float().gather(1, idx)
    if c["score"] == "softmax" and not c["renorm"]:
        sc = sd.gather(1, idx).float()
    elif c["score"] == "softmax":
        sc = torch.exp(zf - zf.amax(1, keepdim=True))
    else:
        sc = 1.0 / (1.0 + torch.exp(-zf))
    w = sc / sc.sum(1, keepdim=True) if c["renorm"] else sc
    counts = torch.bincount(idx.reshape(-1), minlength=E)
    out = {"idx": idx.to(torch.int32), "gate": c["scale"] * w, "counts": counts.to(torch.int32)}
    if b is not None:
        out["bias"] = b + 0.001 * torch.sign(T * k - counts * E).float()
    if c["bwd"]:
        dg = c["scale"] * s["dgate"]
        if c["renorm"]:
            dz = w * (dg - (w * dg).sum(1, keepdim=True))
            if c["score"] == "sigmoid":
                dz = dz / (1.0 + torch.exp(zf))
            out["dlogits"] = torch.zeros(T, E, device=z.device).scatter_(1, idx, dz)
        elif c["score"] == "sigmoid":
            out["dlogits"] = torch.zeros(T, E, device=z.device).scatter_(1, idx, dg * sc / (1.0 + torch.exp(zf)))
        else:
            dp = torch.zeros(T, E, device=z.device).scatter_(1, idx, dg)
            out["dlogits"] = sd.float() * (dp - (sc * dg).sum(1, keepdim=True))
    return out


def _quantize(s, c):
    if c["form"] == "weights":
        if own:
            import moe_expert_routing_router_gb300 as mr
            r = mr.moe_quantize_weights(s["w"])
            return {"q": r["q"], "scale": r["scale"]}
        q, scale = _quantize_weights(s["w"])
        return {"q": q, "scale": scale}
    x, r = s["x"], s["r"]
    if own:
        import moe_expert_routing_router_gb300 as mr
        perm = r["perm"] if c["gather"] else None
        if c["form"] == "rows":
            o = mr.moe_quantize_rows(x, perm=perm, k=c["k"])
        else:
            o = mr.moe_quantize_cols(x, r["offsets"], r["kept"], perm=perm, k=c["k"], out={"q": s["q"], "scale": s["scale"]})
        return {"q": o["q"], "scale": o["scale"]}
    token = r["perm"].long() // c["k"] if c["gather"] else torch.arange(x.shape[0], device=x.device)
    if c["form"] == "rows":
        q, scale = _quantize_rows(x[token])
    else:
        q, scale = _quantize_cols(x, r, token, s["q"], s["scale"])
    return {"q": q, "scale": scale}


def _matmul(s, c):
    if own:
        import moe_expert_routing_router_gb300 as mr
        return mr.moe_expert_matmul(s["q"], s["scale"], s["wq"], s["wscale"], s["r"]["offsets"], s["r"]["kept"], out=s["y"])
    r, y = s["r"], s["y"]
    M, K = s["q"].shape
    a = s["q"].float() * s["scale"].repeat_interleave(BLOCK, 0)[:K].t()
    w = s["wq"].float() * s["wscale"].repeat_interleave(BLOCK, 1)[:, :c["N"]].repeat_interleave(BLOCK, 2)[:, :, :K]
    i = torch.arange(r["most"], device=y.device)[None, :]
    live = i < r["kept"].long()[:, None]
    rows = torch.where(live, r["offsets"][:-1].long()[:, None] + i, torch.zeros_like(i))
    y[rows[live]] = torch.bmm(a[rows], w.transpose(1, 2))[live].to(y.dtype)
    return y


def _wgrad(s, c):
    r = s["r"]
    if own:
        import moe_expert_routing_router_gb300 as mr
        return mr.moe_expert_wgrad(s["dyq"], s["dyscale"], s["xq"], s["xscale"], r["kept"])
    _, cols, live = _columns(r, c["T"] * c["k"], c["E"], r["most"])
    cols = torch.where(live, cols, torch.zeros_like(cols))
    dy = (s["dyq"].float() * s["dyscale"].repeat_interleave(BLOCK, 0).t())[:, cols] * live          # [N, E, C]
    x = (s["xq"].float() * s["xscale"].repeat_interleave(BLOCK, 0).t())[:, cols]
    return torch.bmm(dy.transpose(0, 1), x.permute(1, 2, 0))


def _combine(s, c):
    r, y, gate = s["r"], s["y"], s["gate"]
    if own:
        import moe_expert_routing_router_gb300 as mr
        out = {"out": mr.moe_expert_combine(y, r["idx"], r["slot"], r["offsets"], gate=gate)}
        if c["bwd"]:
            g = mr.moe_expert_combine_bwd(s["dout"], y, r["idx"], r["slot"], r["offsets"], gate, out={"dy": s["dy"]})
            out |= {"dy": g["dy"], "dgate": g["dgate"]}
        return out
    slot = r["slot"].long().view(c["T"], c["k"])
    live = slot >= 0
    pos = torch.where(live, r["offsets"].long()[r["idx"].long()] + slot, torch.zeros_like(slot))
    rows = y.float()[pos] * live[:, :, None]
    out = {"out": (rows * gate[:, :, None]).sum(1).to(y.dtype)}
    if c["bwd"]:
        d = s["dout"].float()[:, None, :]
        out["dgate"] = (rows * d).sum(2)
        s["dy"][pos[live]] = (gate[:, :, None] * d)[live].to(y.dtype)
        out["dy"] = s["dy"]
    return out


# -- the definitions in 64 bits --------------------------------------------------

def exact(case, seed):
    c, s = case, prepare(case, seed)
    if c["op"] == "route":
        return _exact_route(c, s)
    if c["op"] == "quantize":
        return _exact_quantize(c, s)
    r, E = s["r"], c["E"]
    first, kept = r["offsets"].tolist(), r["kept"].tolist()
    if c["op"] == "matmul":
        out = s["y"].double()
        for e in range(E):
            if kept[e]:
                at = slice(first[e], first[e] + kept[e])
                a, w = s["q"][at].double(), s["wq"][e].double()
                for j in range(s["scale"].shape[0]):
                    a[:, j * BLOCK:(j + 1) * BLOCK] *= s["scale"][j, at].double()[:, None]
                    for i in range(s["wscale"].shape[1]):
                        w[i * BLOCK:(i + 1) * BLOCK, j * BLOCK:(j + 1) * BLOCK] *= s["wscale"][e, i, j].double()
                out[at] = a @ w.t()
        return out
    if c["op"] == "wgrad":
        out, block = torch.zeros(E, c["N"], c["K"], dtype=torch.float64, device="cuda"), 0
        for e in range(E):
            for _ in range(-(-kept[e] // BLOCK)):
                at = slice(block * BLOCK, (block + 1) * BLOCK)
                dy = s["dyq"][:, at].double() * s["dyscale"][block].double()[:, None]
                out[e] += dy @ (s["xq"][:, at].double() * s["xscale"][block].double()[:, None]).t()
                block += 1
        return out
    slot, idx = r["slot"].view(c["T"], c["k"]), r["idx"]
    out = torch.zeros(c["T"], c["H"], dtype=torch.float64, device="cuda")
    dy, dgate = s["dy"].double(), torch.zeros(c["T"], c["k"], dtype=torch.float64, device="cuda")
    for j in range(c["k"]):
        t = torch.nonzero(slot[:, j] >= 0)[:, 0]
        at = (r["offsets"][idx[t, j].long()] + slot[t, j]).long()
        g = s["gate"][t, j].double()[:, None]
        out[t] += g * s["y"][at].double()
        if c["bwd"]:
            dgate[t, j] = (s["y"][at].double() * s["dout"][t].double()).sum(1)
            dy[at] = g * s["dout"][t].double()
    return {"out": out, "dgate": dgate, "dy": dy} if c["bwd"] else {"out": out}


def _exact_route(c, s):
    z = s["logits"].double().cpu().numpy()
    T, E = z.shape
    k, G = c["k"], c["groups"]
    if c["score"] == "sigmoid":
        p = np.where(z >= 0, 1.0, np.exp(np.minimum(z, 0))) / (1.0 + np.exp(-np.abs(z)))
    else:
        p = np.exp(z - z.max(1, keepdims=True))
        p /= p.sum(1, keepdims=True)
    value = z
    choice = p
    if s["bias"] is not None:
        value = choice = p + s["bias"].double().cpu().numpy()
    if c["group_score"] == "max":
        top = value.reshape(T, G, -1).max(2)
    else:
        top = np.partition(choice.reshape(T, G, -1), -2, axis=2)[:, :, -2:].sum(2)
    rank = np.argsort(np.argsort(-top, axis=1, kind="stable"), axis=1, kind="stable")
    shut = np.repeat(rank >= c["keep"], E // G, axis=1)
    idx = np.argsort(np.where(shut, np.inf, -value), axis=1, kind="stable")[:, :k]
    q = np.take_along_axis(p, idx, 1)
    total = q.sum(1, keepdims=True) if c["renorm"] else 1.0
    counts = np.bincount(idx.ravel(), minlength=E)
    out = {"idx": idx.astype(np.int32), "gate": c["scale"] * q / total, "counts": counts.astype(np.int32)}
    if s["bias"] is not None:
        out["bias"] = s["bias"].double().cpu().numpy() + np.float64(np.float32(0.001)) * np.sign(T * k - counts * E)
    if c["bwd"]:
        dq = c["scale"] * s["dgate"].double().cpu().numpy()
        if c["renorm"]:
            dq = (dq - (dq * q).sum(1, keepdims=True) / total) / total
        dp = np.zeros((T, E))
        np.put_along_axis(dp, idx, dq, 1)
        out["dlogits"] = dp * p * (1.0 - p) if c["score"] == "sigmoid" else p * (dp - (dp * p).sum(1, keepdims=True))
    return out


def _scale_of(amax):
    """2^n for the least n with amax <= 448 * 2^n."""
    some = torch.where(amax > 0, amax, torch.full_like(amax, 448.0))
    n = torch.ceil(torch.log2(some / 448.0))
    n = torch.where(448.0 * torch.exp2(n - 1) >= some, n - 1, n)
    n = torch.where(448.0 * torch.exp2(n) < some, n + 1, n).clamp(min=-126)
    return torch.exp2(n)


def _round_e4m3(v):
    """v rounded to the nearest multiple of its binade's eighth, ties to even; 2^-9 is the smallest step."""
    step = torch.exp2(torch.floor(torch.log2(v.abs().clamp(min=2.0 ** -20))).clamp(min=-6) - 3)
    return torch.round(v / step) * step


def _exact_quantize(c, s):
    K, M, dev = c["K"], c["T"] * c["k"], {"dtype": torch.float64, "device": "cuda"}
    if c["form"] == "weights":
        w = s["w"].double()
        q, scale = torch.empty_like(w), torch.empty(c["E"], -(-c["N"] // BLOCK), -(-K // BLOCK), **dev)
        for i in range(scale.shape[1]):
            for j in range(scale.shape[2]):
                at = np.s_[:, i * BLOCK:(i + 1) * BLOCK, j * BLOCK:(j + 1) * BLOCK]
                scale[:, i, j] = _scale_of(w[at].abs().amax((1, 2)))
                q[at] = _round_e4m3(w[at] / scale[:, i, j][:, None, None])
        return {"q": q, "scale": scale}
    r, x = s["r"], s["x"].double()
    x = x[torch.div(r["perm"], c["k"], rounding_mode="floor")] if c["gather"] else x
    if c["form"] == "rows":
        q, scale = torch.empty(M, K, **dev), torch.empty(-(-K // BLOCK), M, **dev)
        for j in range(scale.shape[0]):
            at = np.s_[:, j * BLOCK:(j + 1) * BLOCK]
            scale[j] = _scale_of(x[at].abs().amax(1))
            q[at] = _round_e4m3(x[at] / scale[j][:, None])
        return {"q": q, "scale": scale}
    width, block = _width(M, c["E"]), 0
    q, scale = torch.zeros(K, width, **dev), torch.zeros(width // BLOCK, K, **dev)
    for a, n in zip(r["offsets"].tolist(), r["kept"].tolist()):
        for i in range(0, n, BLOCK):
            v = x[a + i:a + min(n, i + BLOCK)]
            scale[block] = _scale_of(v.abs().amax(0))
            q[:, block * BLOCK:block * BLOCK + len(v)] = _round_e4m3(v / scale[block]).t()
            block += 1
    return {"q": q, "scale": scale}


# -- what a pass cannot do without -------------------------------------------------

def work(case):
    c = case
    T, k, E = c["T"], c["k"], c["E"]
    M = T * k
    if c["op"] == "route":
        size = 2 if c["dtype"] == "bf16" else 4
        n = T * E * size + M * 8 + E * 4 + (E * 8 if c["bias"] else 0)
        return {"bytes": n + (T * E * 4 + M * 4 if c["bwd"] else 0), "flops": T * E * 8}
    if c["op"] == "quantize":
        size = 2 if c["dtype"] == "bf16" else 4
        if c["form"] == "weights":
            return {"bytes": E * c["N"] * c["K"] * (size + 1), "flops": 2 * E * c["N"] * c["K"]}
        rows = T if c["gather"] else M
        return {"bytes": rows * c["K"] * size + M * c["K"] + M * c["K"] // 32, "flops": 2 * M * c["K"]}
    if c["op"] == "matmul":
        size, live = 2 if c["out"] == "bf16" else 4, min(E, M)   # each expert that has rows is read once
        return {"bytes": M * c["K"] * 33 / 32 + live * c["N"] * c["K"] + M * c["N"] * size, "flops": 2 * M * c["K"] * c["N"]}
    if c["op"] == "wgrad":
        return {"bytes": M * (c["K"] + c["N"]) * 33 / 32 + E * c["K"] * c["N"] * 4, "flops": 2 * M * c["K"] * c["N"]}
    size = 2 if c["dtype"] == "bf16" else 4
    n = M * c["H"] * size + T * c["H"] * size + M * 12
    if c["bwd"]:
        n += T * c["H"] * size + 2 * M * c["H"] * size + M * 16
    return {"bytes": n, "flops": 2 * M * c["H"] * (3 if c["bwd"] else 1)}
