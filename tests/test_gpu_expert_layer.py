"""The expert side's operators together, as a layer runs them: routing, dispatch, two
quantised products with an activation between them, combine; and the whole backward.

Forward and gradients are compared with the same layer in float64 torch autograd,
which quantises where the layer does (codes are compared exactly elsewhere) and
passes gradients through the quantisation.  Bounds are against the norm of the
whole result: bf16 hidden values (2^-8 each) are quantised to e4m3, where one
rounding moves a value by up to 2^-4 of itself; the layer makes such roundings
twice on the way to the output and three times on the way to a gradient, from
values that differ in their last bf16 bit, which can cross to the neighbouring
code (a step of 2^-3) with probability 2^-8 / 2^-3 = 2^-5 each: a relative
difference of 2^-3 * 2^-2.5 = 0.022 in the norm per such rounding, and 0.07 for
three that add up.
"""

import numpy as np
import pytest
import torch

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def mr(native_lib):
    import moe_expert_routing_router_gb300 as m
    return m


def weights(E, N, K, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return torch.randn(E, N, K, generator=g, device="cuda") / K ** 0.5


def forward(mr, x, logits, bias, w1, w2, cf, route):
    """The layer's calls; everything that the backward needs."""
    r = mr.moe_route_fwd(logits, bias=bias, **route)
    E, k = logits.shape[1], route["k"]
    d = mr.moe_dispatch(r["idx"], E, cf)
    a = mr.moe_quantize_rows(x, perm=d["perm"], k=k)
    h = mr.moe_expert_matmul(a["q"], a["scale"], w1["q"], w1["scale"], d["offsets"], d["kept"])
    act = torch.nn.functional.silu(h.float()).to(torch.bfloat16)
    b = mr.moe_quantize_rows(act)
    y = mr.moe_expert_matmul(b["q"], b["scale"], w2["q"], w2["scale"], d["offsets"], d["kept"])
    out = mr.moe_expert_combine(y, r["idx"], d["slot"], d["offsets"], gate=r["gate"])
    return {"r": r, "d": d, "h": h, "act": act, "y": y, "out": out}


def backward(mr, dout, x, logits, w1, w2, route, s):
    r, d, k = s["r"], s["d"], route["k"]
    c = mr.moe_expert_combine_bwd(dout, s["y"], r["idx"], d["slot"], d["offsets"], r["gate"])
    dyq = mr.moe_quantize_rows(c["dy"])
    dact = mr.moe_expert_matmul(dyq["q"], dyq["scale"], w2["qt"], w2["scalet"], d["offsets"], d["kept"])
    cols = lambda t, **kw: mr.moe_quantize_cols(t, d["offsets"], d["kept"], **kw)  # noqa: E731
    dyc, actc = cols(c["dy"]), cols(s["act"])
    dw2 = mr.moe_expert_wgrad(dyc["q"], dyc["scale"], actc["q"], actc["scale"], d["kept"])
    hf = s["h"].float()
    sg = torch.sigmoid(hf)
    dh = (dact.float() * sg * (1 + hf * (1 - sg))).to(torch.bfloat16)
    dhq, dhc, xc = mr.moe_quantize_rows(dh), cols(dh), cols(x, perm=d["perm"], k=k)
    dw1 = mr.moe_expert_wgrad(dhc["q"], dhc["scale"], xc["q"], xc["scale"], d["kept"])
    dxr = mr.moe_expert_matmul(dhq["q"], dhq["scale"], w1["qt"], w1["scalet"], d["offsets"], d["kept"])
    dx = mr.moe_expert_combine(dxr, r["idx"], d["slot"], d["offsets"])
    dz = mr.moe_route_bwd(logits, r["idx"], c["dgate"], **{n: route[n] for n in ("score", "scale")})
    return {"dx": dx, "dw1": dw1, "dw2": dw2, "dz": dz}


class Through(torch.autograd.Function):
    @staticmethod
    def forward(ctx, x, q):
        return q

    @staticmethod
    def backward(ctx, g):
        return g, None


def stands_for(q, scale):
    """The values of row-quantised codes."""
    return q.double() * scale.repeat_interleave(128, 0)[:q.shape[1]].t().double()


def weight_values(w):
    return w["q"].double() * w["scale"].repeat_interleave(128, 1)[:, :w["q"].shape[1]].repeat_interleave(128, 2)[:, :, :w["q"].shape[2]].double()


def reference(mr, x, logits, w1, w2, s, route, dout):
    """The layer in float64 autograd with the calls' picks."""
    T, E = logits.shape
    k = route["k"]
    idx, slot = s["r"]["idx"].long(), s["d"]["slot"].long().view(T, k)
    xd, zd = x.double().requires_grad_(), logits.double().requires_grad_()
    w1d, w2d = weight_values(w1).requires_grad_(), weight_values(w2).requires_grad_()
    sc = torch.sigmoid(zd) if route["score"] == "sigmoid" else torch.softmax(zd, 1)
    sp = sc.gather(1, idx)
    gate = route["scale"] * sp / sp.sum(1, keepdim=True)
    qx = mr.moe_quantize_rows(x)
    xq = Through.apply(xd, stands_for(qx["q"], qx["scale"]))
    out = torch.zeros(T, w2d.shape[1], dtype=torch.float64, device="cuda")
    for e in range(E):
        t, j = torch.nonzero((idx == e) & (slot >= 0), as_tuple=True)
        if not len(t):
            continue
        h = xq[t] @ w1d[e].t()
        act = torch.nn.functional.silu(h)
        qa = mr.moe_quantize_rows(act.detach().to(torch.bfloat16))
        y = Through.apply(act, stands_for(qa["q"], qa["scale"])) @ w2d[e].t()
        out = out.index_add(0, t, gate[t, j][:, None] * y)
    out.backward(dout.double())
    return out.detach(), {"dx": xd.grad, "dw1": w1d.grad, "dw2": w2d.grad, "dz": zd.grad}


def off(a, b):
    return float((a.double() - b).norm() / b.norm())


@pytest.mark.parametrize("T,E,H,inner,cf,route", [
    (500, 16, 512, 272, 1.0, dict(k=4, score="sigmoid", n_groups=4, topk_groups=2, scale=2.5)),
    (65, 8, 144, 128, 2.0, dict(k=2, score="softmax", scale=1.0)),
    (1, 64, 256, 400, 64.0, dict(k=8, score="sigmoid", n_groups=8, topk_groups=4, scale=1.0)),
])
def test_layer_and_its_gradients(mr, T, E, H, inner, cf, route):
    g = torch.Generator(device="cuda").manual_seed(T)
    x = torch.randn(T, H, generator=g, device="cuda").to(torch.bfloat16)
    logits = torch.randn(T, E, generator=g, device="cuda")
    bias = 0.001 * torch.randint(-100, 101, (E,), generator=g, device="cuda").float()
    w1 = mr.moe_quantize_weights(weights(E, inner, H, 1), transposed=True)
    w2 = mr.moe_quantize_weights(weights(E, H, inner, 2), transposed=True)
    dout = torch.randn(T, H, generator=g, device="cuda").to(torch.bfloat16)
    s = forward(mr, x, logits, bias, w1, w2, cf, route)
    got = backward(mr, dout, x, logits, w1, w2, route, s)
    out, want = reference(mr, x, logits, w1, w2, s, route, dout)
    if T == 500:
        assert int(s["d"]["n_dropped"]) > 0
    assert off(s["out"], out) < 0.022 * 2
    for name in want:
        assert off(got[name], want[name]) < 0.07, (name, off(got[name], want[name]))
    assert mr.moe_expert_device_status() == 0


def test_a_captured_step_repeats(mr):
    """Forward and backward as one graph on new inputs: the same bits as eager calls."""
    T, E, H, inner, route = 200, 16, 256, 128, dict(k=4, score="sigmoid", n_groups=4, topk_groups=2, scale=1.0)
    w1 = mr.moe_quantize_weights(weights(E, inner, H, 1), transposed=True)
    w2 = mr.moe_quantize_weights(weights(E, H, inner, 2), transposed=True)
    x, logits = torch.zeros(T, H, dtype=torch.bfloat16, device="cuda"), torch.zeros(T, E, device="cuda")
    dout = torch.zeros(T, H, dtype=torch.bfloat16, device="cuda")
    bias = torch.zeros(E, device="cuda")

    def step():
        s = forward(mr, x, logits, bias, w1, w2, 8.0, route)
        return {**backward(mr, dout, x, logits, w1, w2, route, s), "out": s["out"]}

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step()                                                   # the dispatch's workspace of this stream
    side.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        held = step()
    for seed in range(3):
        g = torch.Generator(device="cuda").manual_seed(seed)
        x.copy_(torch.randn(T, H, generator=g, device="cuda"))
        logits.copy_(torch.randn(T, E, generator=g, device="cuda"))
        dout.copy_(torch.randn(T, H, generator=g, device="cuda"))
        graph.replay()
        want = step()
        torch.cuda.synchronize()
        for name in want:
            assert torch.equal(held[name], want[name]), name
