"""Layers with the gated activation, as they are run: routing, dispatch, quantisation, the two products with the
activation between them and combine, on 8-bit operands with the whole backward, on 4-bit ones forward; and
the routing with the layer for few tokens.

8 bits, against float64 autograd that quantises where the layer does in the forward and passes gradients through, in
the norm of the whole: one rounding to e4m3 moves a value by up to 2^-4 of itself, evenly, 2^-4 / 3^(1/2) = 0.036 in
the norm.  h has bf16's 2^-8 in both halves, so that an activation's code is the neighbour (a step of 2^-3) with
probability 2 * 2^-8 / 2^-3 = 2^-4: 2^-3 * 2^-2 = 0.031.  The output has the latter and bf16's own rounding: 0.05.  A
gradient has two roundings that the reference does not make (dy and dh, or one of them and the activation's):
2 * 0.036 + 0.031 = 0.10.

4 bits, call by call against float64 of what the call was given: codes of x exactly; products within K * 2^-24 of the sum
of their terms' sizes, and half a bf16 step; an activation's code within its rounding, a fifth of the value or a
fourth of the block's scale; the sum over a token's experts within a rounding of each term.
"""

import numpy as np
import pytest
import torch

import experts_reference as experts_ref
import layer_reference as ref

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def mr(native_lib):
    import moe_expert_routing_router_gb300 as m
    yield m
    assert m.moe_expert_device_status() == 0


def wide(t):
    return t.double().cpu().numpy()


def random(shape, seed, scale=1.0):
    return scale * torch.randn(*shape, generator=torch.Generator(device="cuda").manual_seed(seed), device="cuda")


def off(a, b):
    return float((a.double() - b).norm() / b.norm())


# ---- 8 bits, trained -------------------------------------------------------------

def forward(mr, x, z, w1, w2, cf, route):
    r = mr.moe_route_fwd(z, **route)
    d = mr.moe_dispatch(r["idx"], z.shape[1], cf)
    place = (d["offsets"], d["kept"])
    a = mr.moe_quantize_rows(x, perm=d["perm"], k=route["k"])
    h = mr.moe_expert_matmul(a["q"], a["scale"], w1["q"], w1["scale"], *place)
    b = mr.moe_expert_glu(h, form="e4m3")
    y = mr.moe_expert_matmul(b["q"], b["scale"], w2["q"], w2["scale"], *place)
    return {"r": r, "d": d, "h": h, "y": y, "out": mr.moe_expert_combine(y, r["idx"], d["slot"], d["offsets"], gate=r["gate"])}


def backward(mr, dout, x, z, w1, w2, route, s):
    r, d, h, k = s["r"], s["d"], s["h"], route["k"]
    place = (d["offsets"], d["kept"])
    cols = lambda t, **kw: mr.moe_quantize_cols(t, *place, **kw)  # noqa: E731
    wgrad = lambda a, b: mr.moe_expert_wgrad(a["q"], a["scale"], b["q"], b["scale"], d["kept"])  # noqa: E731
    c = mr.moe_expert_combine_bwd(dout, s["y"], r["idx"], d["slot"], d["offsets"], r["gate"])
    q = mr.moe_quantize_rows(c["dy"])
    dact = mr.moe_expert_matmul(q["q"], q["scale"], w2["qt"], w2["scalet"], *place)
    dh = mr.moe_expert_glu_bwd(h, dact)
    q = mr.moe_quantize_rows(dh)
    dx = mr.moe_expert_combine(mr.moe_expert_matmul(q["q"], q["scale"], w1["qt"], w1["scalet"], *place), r["idx"], d["slot"], d["offsets"])
    return {"dx": dx, "dw1": wgrad(cols(dh), cols(x, perm=d["perm"], k=k)), "dw2": wgrad(cols(c["dy"]), cols(mr.moe_expert_glu(h))),
            "dz": mr.moe_route_bwd(z, r["idx"], c["dgate"], **{n: route[n] for n in ("score", "scale")})}


class Through(torch.autograd.Function):
    @staticmethod
    def forward(ctx, x, q):
        return q

    @staticmethod
    def backward(ctx, g):
        return g, None


def rounded(mr, x):
    q = mr.moe_quantize_rows(x.detach().float())
    return Through.apply(x, q["q"].double() * q["scale"].repeat_interleave(128, 0)[:x.shape[1]].t().double())


def weight_values(w):
    s = w["scale"].repeat_interleave(128, 1)[:, :w["q"].shape[1]].repeat_interleave(128, 2)[:, :, :w["q"].shape[2]]
    return (w["q"].double() * s.double()).requires_grad_()


def reference(mr, x, z, w1, w2, s, route, dout):
    idx, slot = s["r"]["idx"].long(), s["d"]["slot"].long().view(len(x), -1)
    xd, zd, w1d, w2d = x.double().requires_grad_(), z.double().requires_grad_(), weight_values(w1), weight_values(w2)
    sc = (torch.sigmoid(zd) if route["score"] == "sigmoid" else torch.softmax(zd, 1)).gather(1, idx)
    gate = route["scale"] * sc / sc.sum(1, keepdim=True)
    xq, out = rounded(mr, xd), torch.zeros(len(x), w2d.shape[1], dtype=torch.float64, device="cuda")
    for e in range(z.shape[1]):
        t, j = torch.nonzero((idx == e) & (slot >= 0), as_tuple=True)
        if len(t):
            g, u = (xq[t] @ w1d[e].t()).chunk(2, dim=1)
            out = out.index_add(0, t, gate[t, j][:, None] * (rounded(mr, torch.nn.functional.silu(g) * u) @ w2d[e].t()))
    out.backward(dout.double())
    return out.detach(), {"dx": xd.grad, "dw1": w1d.grad, "dw2": w2d.grad, "dz": zd.grad}


@pytest.mark.parametrize("T,E,H,inner,cf,route", [
    (500, 16, 512, 272, 1.0, dict(k=4, score="sigmoid", scale=2.5)),
    (65, 8, 144, 128, 2.0, dict(k=2, score="softmax", scale=1.0)),
    (1, 64, 256, 400, 64.0, dict(k=8, score="sigmoid", scale=1.0)),
])
def test_8_bits_and_gradients(mr, T, E, H, inner, cf, route):
    x, z, dout = random((T, H), T).to(torch.bfloat16), random((T, E), T + 1), random((T, H), T + 2).to(torch.bfloat16)
    w1 = mr.moe_quantize_weights(random((E, 2 * inner, H), 1, H ** -0.5), transposed=True)
    w2 = mr.moe_quantize_weights(random((E, H, inner), 2, inner ** -0.5), transposed=True)
    s = forward(mr, x, z, w1, w2, cf, route)
    got = backward(mr, dout, x, z, w1, w2, route, s)
    out, want = reference(mr, x, z, w1, w2, s, route, dout)
    if T == 500:
        assert int(s["d"]["n_dropped"]) > 0
    assert off(s["out"], out) < 0.05
    for name in want:
        assert off(got[name], want[name]) < 0.10, (name, off(got[name], want[name]))


# ---- 4 bits, served --------------------------------------------------------------

def serve(mr, x, z, w1, w2, cf, k, outs=None):
    """The calls of a forward; rows of dropped assignments hold what `outs` held."""
    r = mr.moe_route_fwd(z, k)
    d = mr.moe_dispatch(r["idx"], z.shape[1], cf)
    h_out, y_out = (torch.zeros(len(x) * k, n, dtype=torch.bfloat16, device="cuda") for n in (w1["q"].shape[1], w2["q"].shape[1])) if outs is None else outs
    a = mr.moe_quantize_fp4(x, perm=d["perm"], k=k)
    h = mr.moe_expert_matmul_fp4(a["q"], a["scale"], w1["q"], w1["scale"], d["offsets"], d["kept"], out=h_out)
    b = mr.moe_expert_glu(h, form="fp4")
    y = mr.moe_expert_matmul_fp4(b["q"], b["scale"], w2["q"], w2["scale"], d["offsets"], d["kept"], out=y_out)
    return {"r": r, "d": d, "a": a, "h": h, "b": b, "y": y, "out": mr.moe_expert_combine(y, r["idx"], d["slot"], d["offsets"], gate=r["gate"])}


def close(got, want, size, K, live):
    bound = K * ref.U32 * size
    experts_ref.assert_near("product", wide(got)[live], want[live], (bound * (1 + ref.U16) + np.abs(want) * ref.U16)[live])


@pytest.mark.parametrize("T,k,E,H,inner,cf", [(300, 4, 16, 288, 160, 1.0), (1, 8, 32, 512, 96, 32.0), (129, 2, 4, 1056, 544, 1.25)])
def test_4_bits(mr, T, k, E, H, inner, cf):
    x, z = random((T, H), T).to(torch.bfloat16), random((T, E), T + 1)
    w1, w2 = (mr.moe_quantize_fp4(random(s, i, s[2] ** -0.5)) for i, s in ((1, (E, 2 * inner, H)), (2, (E, H, inner))))
    s = serve(mr, x, z, w1, w2, cf, k)
    offsets, kept, perm = (s["d"][n].cpu().numpy() for n in ("offsets", "kept", "perm"))
    rows = experts_ref.expert_rows(offsets, kept, T * k)
    live = np.zeros(T * k, dtype=bool)
    for at, n in rows:
        live[at:at + n] = True
    if cf == 1.0:
        assert not live.all()

    read = lambda c: ref.read(c["q"].cpu().numpy(), c["scale"].cpu().numpy())  # noqa: E731
    code, n = ref.quantize_fp4(wide(x)[perm // k])
    assert np.array_equal(s["a"]["q"].cpu().numpy(), ref.pack(code)) and np.array_equal(s["a"]["scale"].cpu().numpy(), ref.fold(n))
    close(s["h"], *ref.products(read(s["a"]), read(w1), rows), H, live)
    assert not wide(s["h"])[~live].any()
    act, unit = ref.glu(wide(s["h"])), np.repeat(2.0 ** (ref.unfold(s["b"]["scale"].cpu().numpy(), inner).astype(float) - 127), 32, axis=1)
    assert (np.abs(read(s["b"]) - act) <= np.maximum(np.abs(act) / 5, unit / 4) * 1.0001).all()
    close(s["y"], *ref.products(read(s["b"]), read(w2), rows), inner, live)
    want, size = experts_ref.combine(wide(s["y"]), s["r"]["idx"].cpu().numpy(), s["d"]["slot"].cpu().numpy(), offsets, wide(s["r"]["gate"]))
    experts_ref.assert_near("out", wide(s["out"]), want, 2 * k * ref.U32 * size + np.abs(want) * ref.U16)


def decode(mr, x, z, w1, w2, k):
    r = mr.moe_route_fwd(z, k, score="softmax")
    return r["idx"], r["gate"], mr.moe_layer_small(x, r["idx"], r["gate"], w1, w2)


@pytest.mark.parametrize("kind", ["fp4", "e4m3"])
def test_few_tokens(mr, kind):
    """Bound: as of the layer's own test, by the norm: bf16's half step and a fourth of it."""
    T, k, E, H, inner = 11, 4, 32, 320, 160
    x, z = random((T, H), 5).to(torch.bfloat16), random((T, E), 6)
    quantize = mr.moe_quantize_fp4 if kind == "fp4" else mr.moe_quantize_weights
    w1, w2 = (quantize(random(s, i, s[2] ** -0.5)) for i, s in ((1, (E, 2 * inner, H)), (2, (E, H, inner))))
    idx, gate, out = decode(mr, x, z, w1, w2, k)
    if kind == "fp4":
        v1, v2 = (ref.read(w["q"].cpu().numpy(), w["scale"].cpu().numpy()) for w in (w1, w2))
    else:
        v1, v2 = (weight_values(w).detach().cpu().numpy() for w in (w1, w2))
    want, _ = ref.layer(wide(x), idx.cpu().numpy(), wide(gate), v1, v2)
    assert np.linalg.norm(wide(out) - want) <= 1.25 * ref.U16 * np.linalg.norm(want)


# ---- captured --------------------------------------------------------------------

def test_captured_forwards_repeat(mr):
    """Both serving paths as one graph, on new inputs and two streams: the bits of eager calls."""
    T, k, E, H, inner = 40, 4, 16, 256, 128
    w1, w2 = (mr.moe_quantize_fp4(random(s, i, s[2] ** -0.5)) for i, s in ((1, (E, 2 * inner, H)), (2, (E, H, inner))))
    streams = [torch.cuda.Stream() for _ in range(2)]
    x, z = ([torch.zeros(T, n, dtype=d, device="cuda") for _ in streams] for n, d in ((H, torch.bfloat16), (E, torch.float32)))
    outs = [[torch.zeros(T * k, n, dtype=torch.bfloat16, device="cuda") for n in (2 * inner, H)] for _ in streams]

    def both(i):
        return serve(mr, x[i], z[i], w1, w2, 1.0, k, outs[i])["out"], decode(mr, x[i], z[i], w1, w2, k)[2]

    graphs, got = [], []
    both(0)
    torch.cuda.synchronize()
    for i in range(2):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            got.append(both(i))
        graphs.append(g)
    for seed in range(3):
        for i in range(2):
            x[i].copy_(random((T, H), 10 * seed + i))
            z[i].copy_(random((T, E), 10 * seed + i + 5))
        torch.cuda.synchronize()
        for s, g in zip(streams, graphs):
            with torch.cuda.stream(s):
                g.replay()
        torch.cuda.synchronize()
        seen = [[t.clone() for t in pair] for pair in got]
        for i in range(2):
            for a, b in zip(seen[i], both(i)):
                assert torch.equal(a, b)
