"""The experts of a layer for few tokens, where the sizes of values and of scales are far from one: against float64, by the
bounds of test_gpu_layer_small.  A token's power of two, a weights' scale and the product of both may each lie anywhere in
fp32, and beyond it, as long as the sums do not."""

import numpy as np
import pytest
import torch

import layer_reference as ref
from test_gpu_layer_small import check, expected, i32, inputs, stands_for, weights, wide

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def mr(native_lib):
    import moe_expert_routing_router_gb300 as m
    return m


def shifted(w, n, rows=slice(None)):
    """The weights times 2^n, of some rows (e4m3: whole blocks of 128 rows)."""
    s = w["scale"].clone()
    if s.dtype is torch.uint8:
        s[:, :, rows] = (s[:, :, rows].int() + n).clamp(0, 254).to(torch.uint8)
    else:
        b = slice(None) if rows == slice(None) else slice(rows.start // 128, None)
        s[:, b] = (s[:, b].double() * 2.0 ** n).float()
    return {**w, "scale": s}


def layer(mr, x, idx, gate, w1, w2):
    got = mr.moe_layer_small(x, idx, gate, w1, w2)
    want, bound = expected(wide(x), idx.cpu().numpy(), wide(gate), stands_for(w1), stands_for(w2))
    assert np.isfinite(want).all() and np.median(np.abs(want)) > 2.0 ** -100
    check(got, want, bound)


# Up to 2, 4, 8 tokens of an expert and more take different arithmetic or products side by side; of 4 experts' 8 are taken at a time.
TOKENS = [(1, 1), (2, 1), (4, 1), (5, 1), (8, 1), (9, 1), (16, 1), (9, 4), (33, 1)]


@pytest.mark.parametrize("kind", ["fp4", "e4m3"])
@pytest.mark.parametrize("T,E", TOKENS)
@pytest.mark.parametrize("top", [127, 124, 116, 64, -60, -100, -112])
def test_tokens_of_any_size(mr, kind, T, E, top):
    """The largest value of x is just below 2^top (or, in whole numbers of 2^-126, bf16's smallest); weights bring the sums back."""
    H, I = 288, 256
    x, _, gate = inputs(T, 1, E, H, 5)
    x = (x.double() * (2.0 ** top * 0.99 / float(x.abs().max()))).to(torch.bfloat16)
    w1, w2 = shifted(weights(mr, kind, E, 2 * I, H, 1), 8 - top), weights(mr, kind, E, H, I, 2)
    layer(mr, x, i32(np.zeros((T, 1))), gate, w1, w2)


@pytest.mark.parametrize("kind", ["fp4", "e4m3"])
@pytest.mark.parametrize("T,E", TOKENS)
@pytest.mark.parametrize("up,down,gates", [(110, -112, 0), (-110, 108, 0), (60, 60, -118), (-60, -60, 120), (-100, 0, 100), (70, -20, -50)])
def test_activations_of_any_size(mr, kind, T, E, up, down, gates):
    """The activations are near 2^up, the second product's weights near 2^down, and the gates bring the result back."""
    H, I = 288, 256
    x, _, gate = inputs(T, 1, E, H, 6)
    w1, w2 = shifted(weights(mr, kind, E, 2 * I, H, 1), up, slice(I, 2 * I)), shifted(weights(mr, kind, E, H, I, 2), down)
    x = (x.float() / x.float().abs().amax(1, keepdim=True)).to(torch.bfloat16)
    layer(mr, x, i32(np.zeros((T, 1))), (gate.double() * 2.0 ** gates).float(), w1, w2)


@pytest.mark.parametrize("kind", ["fp4", "e4m3"])
@pytest.mark.parametrize("T", [1, 4, 5, 9, 16])
def test_a_large_value_that_meets_zero(mr, kind, T):
    """A power times a scale of 2^129, past fp32, whose sum is a number: the value that has the power has the weight 0."""
    H, I, n = 128, 128, 24 if kind == "e4m3" else 18
    x = torch.zeros(T, H)
    x[:, 0], x[:, 40] = 2.0 ** 127, 2.0 ** 92                      # the power is 2^113
    w = torch.zeros(1, 2 * I, H)
    w[:, :, 40] = 1.0                                            # a scale of 2^-8 (4 bits: 2^-2), 2^16 once it is shifted
    make = mr.moe_quantize_fp4 if kind == "fp4" else mr.moe_quantize_weights
    w1, w2 = make(w.cuda()), make(torch.ones(1, H, I).cuda())
    w1 = shifted(shifted(w1, n), -100 - n, slice(I, 2 * I))
    # g = 2^(92 + n), whose sigmoid is 1, and u = 2^-8; the 128 activations are added up
    got = mr.moe_layer_small(x.to(torch.bfloat16).cuda(), i32(np.zeros((T, 1))), torch.full((T, 1), 2.0 ** -(91 + n), device="cuda"), w1, w2)
    assert np.array_equal(wide(got), np.ones((T, H)))


@pytest.mark.parametrize("kind,T", [("fp4", 4), ("fp4", 2), ("e4m3", 16), ("e4m3", 5)])
@pytest.mark.parametrize("top", [120, -120])
def test_a_token_far_from_one_leaves_the_others(mr, kind, T, top):
    """The other tokens of its expert keep their bits, also where sums of values of very different sizes are rounded at every step."""
    E, H, I = 1, 1056, 544
    x, _, gate = inputs(T, 1, E, H, 3)
    x = (x.float() * torch.exp(3.0 * torch.randn(T, H, generator=torch.Generator().manual_seed(4))).cuda()).to(torch.bfloat16)
    idx, w1, w2 = i32(np.zeros((T, 1))), weights(mr, kind, E, 2 * I, H, 1), weights(mr, kind, E, H, I, 2)
    base = mr.moe_layer_small(x, idx, gate, w1, w2)
    far = x.clone()
    far[1] = (x[1].double() * 2.0 ** top / float(x[1].abs().max())).to(torch.bfloat16)
    got = mr.moe_layer_small(far, idx, gate, w1, w2)
    others = [t for t in range(T) if t != 1]
    assert torch.equal(got[others], base[others]) and not torch.equal(got[1], base[1])


def uneven(w, steps, seed, tail=0):
    """4-bit weights with a word's exponents `steps` apart, in an order of each word's own, the largest as they were; `tail`
    more behind the last column, where any byte may be."""
    s = w["scale"]
    g = torch.Generator().manual_seed(seed)
    order = torch.argsort(torch.rand(*s.shape, generator=g), dim=3).cuda()
    s = (s.int() - torch.tensor(steps, device="cuda")[order]).clamp(min=0)
    blocks = w["q"].shape[2] // 16
    if blocks % 4 and tail:
        s[-1, :, :, blocks % 4:] = tail
    return {"q": w["q"], "scale": s.to(torch.uint8)}


@pytest.mark.parametrize("T,E", TOKENS)
@pytest.mark.parametrize("steps", [(0, 7, 15, 23), (0, 1, 22, 24), (0, 24, 30, 31), (0, 33, 50, 90), (0, 0, 0, 25)])
def test_scales_far_apart_in_a_word(mr, T, E, steps):
    """Four exponents that differ by up to 23 and by more, also where all that a token has in the largest block is zero."""
    H, I = 288, 160
    x, _, gate = inputs(T, 1, E, H, 7)
    w1, w2 = (uneven(weights(mr, "fp4", E, n, k, i), steps, i, 200) for n, k, i in ((2 * I, H, 1), (H, I, 2)))
    idx = i32(np.zeros((T, 1)))
    layer(mr, x, idx, gate, w1, w2)
    # of every word of the gates' and the others' first 16 rows, the last block is the largest by far: tokens have zeros there
    s = w1["scale"].clone()
    s[:, :, :, 3] = 150
    s[:, :, :, 0] = 150 - steps[3]
    x = x.clone().view(T, H)
    x[:, 96:128] = 0
    x[:, 224:256] = 0
    layer(mr, x, idx, gate, {"q": w1["q"], "scale": s}, w2)


@pytest.mark.parametrize("T,E", TOKENS)
def test_a_block_of_zeros_beside_small_ones(mr, T, E):
    """The scale of a block of zeros is 1, far above those of weights near 2^-40."""
    H, I = 288, 160
    x, _, gate = inputs(T, 1, E, H, 8)
    w = torch.randn(E, 2 * I, H, generator=torch.Generator().manual_seed(1))
    w[:, I:] *= 2.0 ** -40
    w[:, :, 32:64] = 0
    w[:, :, 256:] = 0
    w1, w2 = mr.moe_quantize_fp4((w / H ** 0.5).cuda()), shifted(weights(mr, "fp4", E, H, I, 2), 40)
    layer(mr, x, i32(np.zeros((T, 1))), gate, w1, w2)


@pytest.mark.parametrize("steps", [(0, 3, 7, 9), (0, 33, 50, 90)])
def test_equal_tokens_of_one_expert(mr, steps):
    """Nine, of which eight are taken at a time and the last one alone: their results differ by roundings."""
    E, H, I, T = 4, 288, 160, 9
    x, _, gate = inputs(1, 1, E, H, 9)
    x, gate = x.expand(T, H).contiguous(), gate.expand(T, 1).contiguous()
    w1, w2 = (uneven(weights(mr, "fp4", E, n, k, i), steps, i) for n, k, i in ((2 * I, H, 1), (H, I, 2)))
    x[:, :32] = 0
    got = mr.moe_layer_small(x, i32(np.zeros((T, 1))), gate, w1, w2)
    want, bound = expected(wide(x), np.zeros((T, 1), dtype=int), wide(gate), stands_for(w1), stands_for(w2))
    check(got, want, bound)
    assert all(torch.equal(got[0], got[t]) for t in range(1, 8))


@pytest.mark.parametrize("kind", ["fp4", "e4m3"])
@pytest.mark.parametrize("T", [1, 4, 5, 9])
@pytest.mark.parametrize("length", [2016, 2048, 2080, 4096, 4064, 6144, 8160, 8192, 8224, 12288, 16352, 16384])
def test_contractions_that_fill_the_warps_and_others(mr, kind, T, length):
    """Lengths of both products at, just below and above those that all warps share evenly."""
    for H, I in ((length, 32), (32, length)):
        x, _, gate = inputs(T, 1, 1, H, T + length)
        layer(mr, x, i32(np.zeros((T, 1))), gate, weights(mr, kind, 1, 2 * I, H, 1), weights(mr, kind, 1, H, I, 2))


@pytest.mark.parametrize("T,E", TOKENS)
def test_bytes_behind_the_last_column(mr, T, E):
    """Scale bytes that stand for no column may be anything, however many tokens an expert has."""
    H, I = 288, 160
    x, _, gate = inputs(T, 1, E, H, 10)
    idx, w1, w2 = i32(np.zeros((T, 1))), weights(mr, "fp4", E, 2 * I, H, 1), weights(mr, "fp4", E, H, I, 2)
    base = mr.moe_layer_small(x, idx, gate, w1, w2)
    for byte in (255, 254, 0):
        w1["scale"][2, :, :, 1:] = byte
        w2["scale"][1, :, :, 1:] = byte
        assert torch.equal(mr.moe_layer_small(x, idx, gate, w1, w2), base)


@pytest.mark.parametrize("kind", ["fp4", "e4m3"])
@pytest.mark.parametrize("T,E", TOKENS)
def test_not_a_number(mr, kind, T, E):
    """A NaN scale, of a row or of a block of weights, is its results', and an infinite or NaN value its token's."""
    H, I = 288, 160
    x, _, gate = inputs(T, 1, E, H, 11)
    idx, w1, w2 = i32(np.zeros((T, 1))), weights(mr, kind, E, 2 * I, H, 1), weights(mr, kind, E, H, I, 2)
    base = mr.moe_layer_small(x, idx, gate, w1, w2)
    s = w2["scale"].clone()
    if kind == "fp4":
        s[1, 0, 7, 0] = 255
    else:
        s[0, 1, 1] = float("nan")
    rows = torch.zeros(H, dtype=torch.bool, device="cuda")
    rows[slice(7, 8) if kind == "fp4" else slice(128, 256)] = True
    got = mr.moe_layer_small(x, idx, gate, w1, {**w2, "scale": s})
    assert bool(got[:, rows].isnan().all())
    if kind == "e4m3" or T <= 4:
        assert torch.equal(got[:, ~rows], base[:, ~rows])
    else:                                                        # the tiles of that row are computed by blocks: other roundings
        off = (got[:, ~rows].double() - base[:, ~rows].double()).norm() / base.double().norm()
        assert float(off) <= 2.0 ** -8 and bool(got[:, ~rows].isfinite().all())
    bad = x.clone()
    bad[0, 3] = float("inf")
    bad[-1, 287] = float("nan")
    got = mr.moe_layer_small(bad, idx, gate, w1, w2)
    others = list(range(1, T - 1))
    assert torch.equal(got[others], base[others]) and not bool(got[[0, T - 1]].isfinite().any())


def exact_weights(w, e):
    """Expert e's weights in float64, on the GPU, from their codes and scales."""
    q, scale = w["q"][e], w["scale"]
    if q.dtype is torch.uint8:
        code = torch.stack([q & 15, q >> 4], 2).flatten(1).long()
        sizes = torch.tensor(ref.FP4, dtype=torch.float64, device="cuda")
        v = torch.where(code >= 8, -sizes[code % 8], sizes[code % 8])
        n = scale[:, e].transpose(0, 1).flatten(1)[:, :code.shape[1] // 32].double()
        return v * torch.exp2(n - 127).repeat_interleave(32, 1)
    s = scale[e].double().repeat_interleave(128, 0)[:q.shape[0]].repeat_interleave(128, 1)[:, :q.shape[1]]
    return q.double() * s


def check_on_gpu(got, x, idx, gate, w1, w2):
    """test_gpu_layer_small's comparison, for sizes that numpy would take long for."""
    (T, H), k, I = x.shape, idx.shape[1], w1["q"].shape[1] // 2
    out, bound = (torch.zeros(T, H, dtype=torch.float64, device="cuda") for _ in range(2))
    n1, n2 = (110 + 3 * H / 2048) * ref.U32, (110 + 3 * I / 2048 + 2 * k) * ref.U32
    for e in range(w1["q"].shape[0]):
        t, j = torch.nonzero(idx == e, as_tuple=True)
        if len(t) == 0:
            continue
        w, v = exact_weights(w1, e), x[t].double()
        h, size = v @ w.t(), v.abs() @ w.abs().t()
        g, u, dg, du = h[:, :I], h[:, I:], n1 * size[:, :I], n1 * size[:, I:]
        s = torch.sigmoid(g)
        act = g * s * u
        block = torch.nn.functional.pad(act.abs(), (0, -I % 128)).view(len(t), -1, 128).amax(2).repeat_interleave(128, 1)[:, :I]
        off = 1.1 * dg * u.abs() + (g * s).abs() * du + 1.1 * dg * du + act.abs() * ((g.abs() + 8) * ref.U32)
        off += (act.abs() + off) * 2.0 ** -11 + block * 2.0 ** -39
        w, a = exact_weights(w2, e), gate[t, j].double()[:, None]
        out.index_add_(0, t, a * (act @ w.t()))
        bound.index_add_(0, t, a.abs() * ((off + n2 * (act.abs() + off)) @ w.abs().t()))
    bound = bound + (out.abs() + bound) * ref.U16 + 2.0 ** -134
    off = (got.double() - out).abs()
    assert bool((off <= bound).all()), float((off / bound).max())
    assert float((got.double() - out).norm()) <= 1.25 * ref.U16 * float(out.norm())


def made_weights(kind, E, N, K, seed):
    """Quantised weights near 1 / sqrt(K), made on the GPU."""
    g = torch.Generator(device="cuda").manual_seed(seed)
    top = -int(np.log2(K) / 2)
    if kind == "fp4":
        return {"q": torch.randint(0, 256, (E, N, K // 2), dtype=torch.uint8, generator=g, device="cuda"),
                "scale": torch.randint(125 + top, 128 + top, (-(-K // 128), E, N, 4), dtype=torch.uint8, generator=g, device="cuda")}
    q = torch.empty(E, N, K, dtype=torch.float8_e4m3fn, device="cuda")
    for e in range(E):
        q[e] = (64 * torch.randn(N, K, generator=g, device="cuda")).clamp(-448, 448).to(torch.float8_e4m3fn)
    n = torch.randint(-8, -5, (E, -(-N // 128), -(-K // 128)), generator=g, device="cuda") + top
    return {"q": q, "scale": torch.exp2(n.float())}


@pytest.mark.parametrize("kind", ["fp4", "e4m3"])
@pytest.mark.parametrize("T,k,E,H,I", [(64, 8, 64, 4096, 2048), (64, 2, 3, 128, 16384), (64, 2, 4, 16384, 128), (37, 3, 5, 160, 8224), (16, 8, 64, 2048, 768)])
def test_many_tiles_of_experts_with_many_tokens(mr, kind, T, k, E, H, I):
    """More tiles of an expert on an SM than are taken again at a time for more tokens than are staged; once with a token
    far from one among them."""
    x, idx, gate = inputs(T, k, E, H, 12)
    x = (x.float() / x.float().abs().amax(1, keepdim=True) * 4).to(torch.bfloat16)
    w1, w2 = made_weights(kind, E, 2 * I, H, 1), made_weights(kind, E, H, I, 2)
    got = mr.moe_layer_small(x, idx, gate, w1, w2)
    check_on_gpu(got, x, idx, gate, w1, w2)
    far = x.clone()
    far[5] = (far[5].double() * 2.0 ** -115).to(torch.bfloat16)
    check_on_gpu(mr.moe_layer_small(far, idx, gate, w1, w2), far, idx, gate, w1, w2)
