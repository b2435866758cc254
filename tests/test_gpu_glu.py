"""GPU parity of the gated activation and its gradient against float64.

Bounds, in roundings of 2^-24: t = exp(-|g|) is within 4 (expf one unit in the last place, twice that
allowed) for fp32, and 2 |g| + 4 for bf16, whose exponent |g| log2(e) is rounded once with a rounded
constant, before an ex2 that is within 2 units; 1 + t adds 1, the reciprocal (one unit) 2, t times it
1: a sigmoid is within 4 + 4 or 2 |g| + 8 of them.  y has two more products, du two, dg three and
the sum 1 + g (1 - s), whose terms may cancel: its bound goes by their sizes.  Below 2^-126 a sigmoid is
off by up to 2^-148, times what multiplies it.  A bf16 result adds half a step, 2^-8 of it.
"""

import numpy as np
import pytest
import torch

import experts_reference as experts_ref
import layer_reference as ref

pytestmark = pytest.mark.gpu
DTYPES = [torch.bfloat16, torch.float32]
TINY = 2.0 ** -148


@pytest.fixture(scope="module")
def mr(native_lib):
    import moe_expert_routing_router_gb300 as m
    return m


def wide(t):
    return t.double().cpu().numpy()


def hidden(M, I, dtype, seed=0, sigma=2.0):
    g = torch.Generator().manual_seed(seed + M + I)
    h = sigma * torch.randn(M, 2 * I, generator=g)
    h[0, :5] = torch.tensor([0.0, -0.0, 88.0, -88.0, -1.2784645])   # the gate's slope is 0 at the last
    h[-1, :3] = torch.tensor([-100.0, 100.0, -20.0])
    return h.to(dtype)


def roundings(g, dtype):
    return 10 + (2 * np.abs(g) if dtype is torch.bfloat16 else 0)


def bound(h, dtype):
    g, u = np.split(h, 2, axis=1)
    y = np.abs(ref.glu(h))
    return y * roundings(g, dtype) * ref.U32 + (1 + np.abs(g * u)) * TINY


def half_step(y, dtype):
    return np.abs(y) * ref.U16 + 2.0 ** -134 if dtype is torch.bfloat16 else 0.0


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("M,I", [(1, 16), (3, 144), (100, 512), (257, 1040), (33, 4096)])
def test_value_and_gradient(mr, M, I, dtype):
    h = hidden(M, I, dtype)
    dy = torch.randn(M, I, generator=torch.Generator().manual_seed(1)).to(dtype)
    hw, dw = wide(h), wide(dy)
    y = mr.moe_expert_glu(h.cuda())
    assert y.dtype is dtype
    want = ref.glu(hw)
    experts_ref.assert_near("y", wide(y), want, bound(hw, dtype) * (1 + ref.U16) + half_step(want, dtype))
    dh = mr.moe_expert_glu_bwd(h.cuda(), dy.cuda())
    g, u = np.split(hw, 2, axis=1)
    s, c = ref.sigmoid(g), ref.sigmoid(-g)
    want = ref.glu_bwd(hw, dw)
    n = roundings(g, dtype) * ref.U32
    terms = np.concatenate([np.abs(dw * u) * s * (1 + np.abs(g) * c) * (2 * n + 4 * ref.U32), np.abs(dw * g) * s * n], axis=1)
    tiny = np.concatenate([1 + np.abs(dw * u) * (1 + np.abs(g)), 1 + np.abs(dw * g)], axis=1) * TINY
    experts_ref.assert_near("dh", wide(dh), want, (terms + tiny) * (1 + ref.U16) + half_step(want, dtype))


def test_gradient_against_differences(mr):
    """Of fp32 values: the difference of two values over 2^-6 is the slope within the third derivative's share."""
    M, I, step = 16, 64, 2.0 ** -6
    h = hidden(M, I, torch.float32, sigma=1.0).cuda()
    dh = mr.moe_expert_glu_bwd(h, torch.ones(M, I, device="cuda"))
    for half in (0, 1):
        d = torch.zeros_like(h)
        d[:, half * I:(half + 1) * I] = step
        got = (mr.moe_expert_glu(h + d).double() - mr.moe_expert_glu(h - d).double()) / (2 * step)
        want = dh[:, half * I:(half + 1) * I].double()
        # |third derivative of g sigmoid(g)| < 1; the values' roundings, 16 * 2^-24 each, and those of h +- d, over the step
        size = (h.abs()[:, :I] + 1) * (h.abs()[:, I:] + 1)
        assert bool(((got - want).abs() <= size.double() * (step ** 2 / 6 + 34 * ref.U32 / step)).all())


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("form", ["fp4", "e4m3"])
@pytest.mark.parametrize("M,I", [(1, 32), (3, 160), (100, 512), (65, 1056)])
def test_quantized(mr, M, I, dtype, form):
    """A scale is that of the block's largest value, a code the nearest of its value, each moved by its bound at most."""
    h = hidden(M, I, dtype)
    hw = wide(h)
    y, off = ref.glu(hw), bound(hw, dtype)
    y[:, :1] += 0.0
    got = mr.moe_expert_glu(h.cuda(), form=form)
    block = 32 if form == "fp4" else 128
    pad = lambda a: np.pad(a, ((0, 0), (0, -I % block))).reshape(M, -1, block)  # noqa: E731
    lo, hi = (pad(np.maximum(np.abs(y) - off, 0)).max(axis=2), pad(np.abs(y) + off).max(axis=2))
    if form == "fp4":
        n = ref.unfold(got["scale"].cpu().numpy(), I).astype(np.int64)
        assert ((n == ref.fp4_exponent(lo)) | (n == ref.fp4_exponent(hi))).all()
        s = np.repeat(2.0 ** (n - 127.0), 32, axis=1)
        back = ref.values(ref.unpack(got["q"].cpu().numpy()))
        near = [ref.values(ref.round_fp4((y + d) / s)) for d in (-off, off)]
        assert np.array_equal(got["scale"].cpu().numpy(), ref.fold(n))
    else:
        scale = wide(got["scale"]).T
        assert ((scale == experts_ref.block_scale(lo)) | (scale == experts_ref.block_scale(hi))).all()
        s = np.repeat(scale, 128, axis=1)[:, :I]
        back = wide(got["q"])
        near = [experts_ref.round_e4m3(np.clip((y + d) / s, -448, 448)) for d in (-off, off)]
    assert ((back == near[0]) | (back == near[1])).all()


@pytest.mark.parametrize("form", ["fp4", "e4m3"])
def test_not_finite_block(mr, form):
    h = hidden(4, 256, torch.float32)
    h[1, 130] = float("nan")
    h[2, 256 + 5] = float("inf")
    got = mr.moe_expert_glu(h.cuda(), form=form)
    bad = (got["scale"].cpu().numpy() == 255).any(axis=2) if form == "fp4" else np.isnan(wide(got["scale"]))
    want = np.zeros((2, 4), dtype=bool)
    want[1, 1] = want[0, 2] = True
    assert np.array_equal(bad, want)


def test_rows_past_32_bits(mr):
    M, I = 40_000, 32_768
    h = torch.zeros(M, 2 * I, dtype=torch.bfloat16, device="cuda")
    tail = hidden(2, I, torch.bfloat16)
    h[-2:] = tail.cuda()
    alone = tail.cuda()
    y = mr.moe_expert_glu(h)
    assert torch.equal(y[-2:], mr.moe_expert_glu(alone)) and not bool(y[:-2].any())
    del y
    dy = torch.ones(M, I, dtype=torch.bfloat16, device="cuda")
    assert torch.equal(mr.moe_expert_glu_bwd(h, dy)[-2:], mr.moe_expert_glu_bwd(alone, dy[:2]))
    for form in ("fp4", "e4m3"):
        a, b = mr.moe_expert_glu(h, form=form), mr.moe_expert_glu(alone, form=form)
        assert torch.equal(a["q"].view(torch.uint8)[-2:], b["q"].view(torch.uint8)) and torch.equal(a["scale"][:, -2:], b["scale"])


def test_refusals(mr):
    h = torch.zeros(4, 64, device="cuda")
    y = torch.zeros(4, 32, device="cuda")
    for call in (lambda: mr.moe_expert_glu(h[:, :63].contiguous()), lambda: mr.moe_expert_glu(h, form="int8"), lambda: mr.moe_expert_glu(h, out={"q": y}),
                 lambda: mr.moe_expert_glu(h, form="fp4", out=y), lambda: mr.moe_expert_glu(h.half()), lambda: mr.moe_expert_glu(h[:, ::2]),
                 lambda: mr.moe_expert_glu(h, out=y.bfloat16()), lambda: mr.moe_expert_glu_bwd(h, y.bfloat16()), lambda: mr.moe_expert_glu_bwd(h, y[:2])):
        with pytest.raises(ValueError):
            call()
    for call in (lambda: mr.moe_expert_glu(h[:, :48].contiguous()), lambda: mr.moe_expert_glu(h[:, :32].contiguous(), form="fp4")):
        with pytest.raises(mr._native.MoeRouterError):            # I = 24; I = 16 for a form with blocks of 32
            call()
