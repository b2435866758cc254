"""GPU parity of the experts of a layer for few tokens against float64.

Bound of a result, with U = 2^-24.  One sum of a product's 16 terms and the sum so far loses at most
17 * 2^-25 + 2^-23 of its terms' sizes S; a warp forms 8 of them for 128 of the contraction, whose sums are then scaled
and added (3 roundings each, and 16 warps' parts): all in all less than (110 + 3 * K / 2048) U S for a contraction of K.
  activation: off by that in g and u, by the sigmoid's (|g| + 8) U, and by its rounding to 11 bits, 2^-11, or 2^-39
              of the largest of its 128
  result:     the activations' times |gate w2|, the second sum's own, a rounding for each of k gates, and half a bf16 step, 2^-8
Such a bound adds up what in fact averages, so the norm of all is held too: by the bf16 rounding, at most 2^-8, and a quarter
of that for the rest (the activations' roundings are independent: 2^-11 of the norm).
"""

import numpy as np
import pytest
import torch

import layer_reference as ref

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def mr(native_lib):
    import moe_expert_routing_router_gb300 as m
    return m


def wide(t):
    return t.double().cpu().numpy()


def i32(a):
    return torch.as_tensor(np.asarray(a), dtype=torch.int32).cuda()


def weights(mr, kind, E, N, K, seed):
    g = torch.Generator().manual_seed(seed)
    w = (torch.randn(E, N, K, generator=g) * torch.exp(0.5 * torch.randn(E, N, 1, generator=g)) / K ** 0.5).cuda()
    return mr.moe_quantize_fp4(w) if kind == "fp4" else {n: t for n, t in mr.moe_quantize_weights(w).items()}


def stands_for(w):
    if w["q"].dtype is torch.uint8:
        return ref.read(w["q"].cpu().numpy(), w["scale"].cpu().numpy())
    s = wide(w["scale"]).repeat(128, axis=1).repeat(128, axis=2)
    return wide(w["q"]) * s[:, :w["q"].shape[1], :w["q"].shape[2]]


def inputs(T, k, E, H, seed):
    g = torch.Generator().manual_seed(seed)
    x = (torch.randn(T, H, generator=g) * torch.exp(0.7 * torch.randn(1, H, generator=g)) * torch.exp(torch.randn(T, 1, generator=g))).to(torch.bfloat16)
    idx = torch.stack([torch.randperm(max(E, k), generator=g)[:k] % E for _ in range(T)]).to(torch.int32)
    gate = torch.rand(T, k, generator=g) + 0.05
    return x.cuda(), idx.cuda(), (gate / gate.sum(1, keepdim=True)).cuda()


def expected(x, idx, gate, w1, w2):
    """(results, their bounds)."""
    T, k = idx.shape
    H, I = x.shape[1], w2.shape[2]
    out, bound = np.zeros((T, H)), np.zeros((T, H))
    n1, n2 = (110 + 3 * H / 2048) * ref.U32, (110 + 3 * I / 2048 + 2 * k) * ref.U32
    for t in range(T):
        for j in range(k):
            e = idx[t, j]
            if not 0 <= e < len(w1):
                continue
            h, size = w1[e] @ x[t], np.abs(w1[e]) @ np.abs(x[t])
            g, u, dg, du = h[:I], h[I:], n1 * size[:I], n1 * size[I:]
            s = ref.sigmoid(g)
            act = g * s * u
            slope = 1.1                                          # the largest of |d (g sigmoid(g)) / dg|
            block = np.abs(np.pad(act, (0, -I % 128))).reshape(-1, 128).max(axis=1).repeat(128)[:I]
            off = slope * dg * np.abs(u) + np.abs(g * s) * du + slope * dg * du + np.abs(act) * ((np.abs(g) + 8) * ref.U32)
            off += (np.abs(act) + off) * 2.0 ** -11 + block * 2.0 ** -39
            v, a = np.abs(w2[e]), abs(gate[t, j])
            out[t] += gate[t, j] * (w2[e] @ act)
            bound[t] += a * (v @ (off + n2 * (np.abs(act) + off)))
    return out, bound + (np.abs(out) + bound) * ref.U16 + 2.0 ** -134


def check(got, want, bound):
    got = wide(got)
    off = np.abs(got - want)
    assert (off <= bound).all(), float((off / bound).max())
    assert np.linalg.norm(got - want) <= 1.25 * ref.U16 * np.linalg.norm(want)


CASES = [
    (1, 1, 1, 32, 32, "fp4", "fp4"), (1, 8, 16, 512, 256, "fp4", "fp4"), (2, 3, 8, 160, 96, "fp4", "fp4"), (5, 3, 24, 1424, 1040, "e4m3", "e4m3"),
    (7, 2, 5, 2080, 288, "fp4", "fp4"), (16, 4, 8, 256, 544, "e4m3", "fp4"), (9, 8, 8, 288, 144, "fp4", "e4m3"), (64, 8, 16, 128, 128, "fp4", "fp4"),
    (64, 1, 1, 192, 64, "fp4", "fp4"), (64, 2, 2, 144, 272, "e4m3", "e4m3"), (33, 5, 6, 416, 32, "fp4", "fp4"), (3, 2, 1024, 64, 32, "fp4", "fp4"),
    (20, 1, 1, 16384, 32, "fp4", "fp4"), (12, 1, 1, 64, 16384, "e4m3", "e4m3"), (1, 2, 2, 16, 16, "e4m3", "e4m3"), (40, 1, 1, 4096, 64, "e4m3", "e4m3"),
    (64, 8, 1024, 32, 32, "fp4", "fp4"), (50, 7, 700, 64, 32, "fp4", "fp4"), (64, 8, 513, 48, 32, "e4m3", "fp4"),
]


@pytest.mark.parametrize("T,k,E,H,I,kind1,kind2", CASES)
def test_layer(mr, T, k, E, H, I, kind1, kind2):
    x, idx, gate = inputs(T, k, E, H, T + H)
    w1, w2 = weights(mr, kind1, E, 2 * I, H, 1), weights(mr, kind2, E, H, I, 2)
    got = mr.moe_layer_small(x, idx, gate, w1, w2)
    assert got.shape == (T, H) and got.dtype is torch.bfloat16
    check(got, *expected(wide(x), idx.cpu().numpy(), wide(gate), stands_for(w1), stands_for(w2)))


@pytest.mark.parametrize("kind", ["fp4", "e4m3"])
def test_no_expert_and_the_same_expert_twice(mr, kind):
    """Indices outside the experts add nothing; a token of them alone gets zeros; a repeated one counts twice."""
    T, k, E, H, I = 6, 3, 4, 160, 96
    x, _, gate = inputs(T, k, E, H, 0)
    idx = np.array([[0, 1, 2], [-1, -1, -1], [3, 3, 1], [4, 1 << 30, -(1 << 31)], [2, 2, 2], [-1, 0, 9]])
    w1, w2 = weights(mr, kind, E, 2 * I, H, 1), weights(mr, kind, E, H, I, 2)
    got = mr.moe_layer_small(x, i32(idx), gate, w1, w2)
    check(got, *expected(wide(x), idx, wide(gate), stands_for(w1), stands_for(w2)))
    assert not bool(got[1].any()) and not bool(got[3].any())
    none = torch.full((T, H), 5.0, dtype=torch.bfloat16, device="cuda")
    assert not bool(mr.moe_layer_small(x, i32(np.full((T, k), -1)), gate, w1, w2, out=none).any())


@pytest.mark.parametrize("kind,T,E,H,I,spread", [("e4m3", 64, 3, 288, 160, 0.0), ("fp4", 12, 8, 288, 160, 0.0), ("e4m3", 64, 3, 1056, 544, 3.0), ("fp4", 12, 8, 1056, 544, 3.0),
                                                 ("fp4", 16, 8, 2080, 1056, 3.0), ("e4m3", 21, 4, 2080, 1056, 3.0)])
def test_a_token_alone_and_among_others(mr, kind, T, E, H, I, spread):
    """The same bits, whatever its place among its experts' tokens and the passes over them (4-bit weights: of up to 4), also
    where sums of values of very different sizes are rounded at every step."""
    k = 2
    x, _, gate = inputs(T, k, E, H, 3)
    x = (x.float() * torch.exp(spread * torch.randn(T, H, generator=torch.Generator().manual_seed(4))).cuda()).to(torch.bfloat16)
    t = np.arange(T)
    idx = i32(np.stack([2 * t % E, (2 * t + 1) % E], axis=1))      # fp4: three or four tokens an expert
    w1, w2 = weights(mr, kind, E, 2 * I, H, 1), weights(mr, kind, E, H, I, 2)
    base = mr.moe_layer_small(x, idx, gate, w1, w2)
    for part in ([0], [T - 1], [5, 4, 3], list(range(2, T // 2 + 3))):
        got = mr.moe_layer_small(x[part].contiguous(), idx[part].contiguous(), gate[part].contiguous(), w1, w2)
        assert torch.equal(got, base[part])


@pytest.mark.parametrize("kind", ["fp4", "e4m3"])
def test_repeated_calls_give_the_same_bits(mr, kind):
    x, idx, gate = inputs(64, 4, 5, 288, 3)
    w1, w2 = weights(mr, kind, 5, 320, 288, 1), weights(mr, kind, 5, 288, 160, 2)
    base = mr.moe_layer_small(x, idx, gate, w1, w2)
    assert all(torch.equal(base, mr.moe_layer_small(x, idx, gate, w1, w2)) for _ in range(5))


@pytest.mark.parametrize("kind", ["fp4", "e4m3"])
def test_not_finite(mr, kind):
    """An infinity or a NaN of a token stays with it, one of an expert's weights with its tokens."""
    T, k, E, H, I = 5, 1, 3, 160, 96
    x, _, gate = inputs(T, k, E, H, 4)
    idx = i32([[0], [0], [1], [1], [2]])
    w1, w2 = weights(mr, kind, E, 2 * I, H, 1), weights(mr, kind, E, H, I, 2)
    base = mr.moe_layer_small(x, idx, gate, w1, w2)
    bad = x.clone()
    bad[1, 3], bad[2, 150] = float("inf"), float("nan")
    got = mr.moe_layer_small(bad, idx, gate, w1, w2)
    assert torch.equal(got[[0, 3, 4]], base[[0, 3, 4]]) and not bool(got[1:3].isfinite().any())
    s = w2["scale"].clone()
    if kind == "fp4":
        s[0, 1, 7, 2] = 255
    else:
        s[1, 0, 0] = float("nan")
    got = mr.moe_layer_small(x, idx, gate, w1, {**w2, "scale": s})
    rows = slice(7, 8) if kind == "fp4" else slice(0, 128)
    assert bool(got[2:4, rows].isnan().all()) and torch.equal(got[[0, 1, 4]], base[[0, 1, 4]])
    if kind == "fp4":
        keep = [i for i in range(H) if i != 7]
        assert torch.equal(got[:, keep], base[:, keep])


@pytest.mark.parametrize("size", [1e-30, 1e30, 2.0 ** -120])
def test_values_far_from_one(mr, size):
    """Values of x as far as bf16 reaches, with weights that bring them back."""
    T, k, E, H, I = 3, 1, 2, 256, 64
    x, idx, gate = inputs(T, k, E, H, 5)
    x = (x.float() * size).to(torch.bfloat16)
    w1, w2 = weights(mr, "fp4", E, 2 * I, H, 1), weights(mr, "fp4", E, H, I, 2)
    shift = int(round(np.log2(1 / size)))
    w1["scale"] = (w1["scale"].int() + shift).clamp(1, 254).to(torch.uint8)
    got = mr.moe_layer_small(x, idx, gate, w1, w2)
    check(got, *expected(wide(x), idx.cpu().numpy(), wide(gate), stands_for(w1), stands_for(w2)))


def test_bytes_behind_the_last_column(mr):
    """Scale bytes that stand for no column may be anything."""
    T, k, E, H, I = 4, 2, 4, 160, 96
    x, idx, gate = inputs(T, k, E, H, 6)
    w1, w2 = weights(mr, "fp4", E, 2 * I, H, 1), weights(mr, "fp4", E, H, I, 2)
    base = mr.moe_layer_small(x, idx, gate, w1, w2)
    w1["scale"][1, :, :, 1:] = 255
    w2["scale"][0, :, :, 3:] = 255
    assert torch.equal(mr.moe_layer_small(x, idx, gate, w1, w2), base)


def test_weights_past_32_bits(mr):
    """The last of so many experts that codes and scales lie past 2^31."""
    E, H, I = 600, 2048, 1024
    w1 = {"q": torch.zeros(E, 2 * I, H, dtype=torch.uint8, device="cuda").view(torch.float8_e4m3fn), "scale": torch.ones(E, 16, 16, device="cuda")}
    w2 = {"q": torch.zeros(E, H, I, dtype=torch.uint8, device="cuda").view(torch.float8_e4m3fn), "scale": torch.ones(E, 16, 8, device="cuda")}
    a, b = weights(mr, "e4m3", 1, 2 * I, H, 1), weights(mr, "e4m3", 1, H, I, 2)
    for w, part in ((w1, a), (w2, b)):
        w["q"].view(torch.uint8)[-1:] = part["q"].view(torch.uint8)
        w["scale"][-1:] = part["scale"]
    x, _, gate = inputs(3, 1, 1, H, 7)
    got = mr.moe_layer_small(x, i32([[E - 1], [5], [E - 1]]), gate, w1, w2)
    want = mr.moe_layer_small(x, i32([[0], [-1], [0]]), gate, a, b)
    assert torch.equal(got, want) and bool(want.any())


def test_captured_and_concurrent_calls(mr):
    """Two graphs on two streams at once, new inputs, and eager calls beside them: the bits of eager calls."""
    E, H, I, k = 8, 512, 256, 2
    w1, w2 = weights(mr, "fp4", E, 2 * I, H, 1), weights(mr, "fp4", E, H, I, 2)
    sets = []
    for T in (1, 9):
        x, idx, gate = inputs(T, k, E, H, T)
        s = torch.cuda.Stream()
        s.wait_stream(torch.cuda.current_stream())
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, stream=s):
            for _ in range(3):
                held = mr.moe_layer_small(x, idx, gate, w1, w2)
        sets.append((s, g, held, x, idx, gate))
    for seed in range(3):
        fresh = []
        for s, g, held, x, idx, gate in sets:
            new = inputs(x.shape[0], k, E, H, 50 + seed)
            for t, v in zip((x, idx, gate), new):
                t.copy_(v)
            fresh.append(new)
        torch.cuda.synchronize()
        for _ in range(5):
            for s, g, *_ in sets:
                with torch.cuda.stream(s):
                    g.replay()
            mr.moe_layer_small(*fresh[0], w1, w2)
        torch.cuda.synchronize()
        for (_, _, held, *_), new in zip(sets, fresh):
            assert torch.equal(held, mr.moe_layer_small(*new, w1, w2))


def test_a_given_stream(mr):
    E, H, I = 4, 256, 128
    x, idx, gate = inputs(4, 2, E, H, 1)
    w1, w2 = weights(mr, "e4m3", E, 2 * I, H, 1), weights(mr, "e4m3", E, H, I, 2)
    want = mr.moe_layer_small(x, idx, gate, w1, w2)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    got = mr.moe_layer_small(x, idx, gate, w1, w2, stream=s)
    s.synchronize()
    assert torch.equal(got, want)


def test_refusals(mr):
    E, H, I, k = 4, 64, 32, 2
    x, idx, gate = inputs(4, k, E, H, 1)
    w1, w2 = weights(mr, "fp4", E, 2 * I, H, 1), weights(mr, "fp4", E, H, I, 2)
    ok = dict(x=x, idx=idx, gate=gate, w1=w1, w2=w2)
    mr.moe_layer_small(**ok)
    for name, value in (("x", x.float()), ("x", x[:, ::2]), ("idx", idx.long()), ("idx", idx[:2]), ("gate", gate.double()), ("gate", gate[:, :1].contiguous()),
                        ("w1", w2), ("w2", w1), ("w1", w1["q"]), ("w1", {"q": w1["q"]}), ("w1", {**w1, "scale": w1["scale"].float()}),
                        ("w2", weights(mr, "fp4", E + 1, H, I, 2)), ("w2", {**w2, "scale": w2["scale"][:, :, :8].contiguous()}), ("out", torch.zeros(4, H, device="cuda"))):
        with pytest.raises(ValueError):
            mr.moe_layer_small(**{**ok, name: value})
    big = inputs(65, k, E, H, 1)
    with pytest.raises((ValueError, mr._native.MoeRouterError)):
        mr.moe_layer_small(*big, w1, w2)
    with pytest.raises((ValueError, mr._native.MoeRouterError)):
        mr.moe_layer_small(x[:0], idx[:0], gate[:0], w1, w2)
