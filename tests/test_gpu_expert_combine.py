"""GPU parity of the gated combine and its gradient against float64.

Bounds: out is a sum of k fused products in fp32 (k roundings of 2^-24 against
the sum of sizes) and one rounding to its type; dy is one product rounded to
its type (and once to fp32 on the way to bf16); dgate adds H products in fp32
in some order (H roundings against the sum of sizes).
"""

import numpy as np
import pytest
import torch

import experts_reference as ref

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def mr(native_lib):
    import moe_expert_routing_router_gb300 as m
    return m


def wide(t):
    return t.float().cpu().numpy().astype(np.float64)


def i32(a):
    return torch.as_tensor(np.asarray(a), dtype=torch.int32).cuda()


def make(T, k, E, H, capacity, dtype, seed=0):
    rng = np.random.default_rng(seed)
    idx = np.stack([rng.permutation(E)[:k] for _ in range(T)])
    _, slot, offsets, _ = ref.dispatch(idx, E, capacity)
    g = torch.Generator().manual_seed(seed)
    y = torch.randn(T * k, H, generator=g).to(dtype)
    gate = torch.rand(T, k, generator=g)
    dout = torch.randn(T, H, generator=g).to(dtype)
    return idx, slot, offsets, y, gate, dout


CASES = [(1, 1, 1, 1, 9), (1, 8, 8, 4096, 9), (17, 8, 16, 2048, 5), (300, 6, 8, 1040, 150), (33, 2, 4, 7, 9), (9, 3, 5, 1000, 0), (5, 8, 64, 4100, 1),
         (260, 4, 8, 264, 999)]


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("T,k,E,H,capacity", CASES)
def test_combine_and_gradient(mr, T, k, E, H, capacity, dtype):
    idx, slot, offsets, y, gate, dout = make(T, k, E, H, capacity, dtype)
    dropped = np.ones(T * k, bool)
    rows = (offsets[idx.ravel()] + slot)[slot >= 0]
    dropped[rows] = False
    y[torch.from_numpy(dropped)] = float("nan")                  # rows of dropped assignments are not read
    u = ref.U16 if dtype == torch.bfloat16 else ref.U32
    args = (i32(idx), i32(slot), i32(offsets))
    for g in (gate, None):
        got = mr.moe_expert_combine(y.cuda(), *args, gate=None if g is None else g.cuda())
        want, size = ref.combine(wide(y), idx, slot, offsets, None if g is None else wide(g))
        ref.assert_near("out", wide(got), want, k * ref.U32 * size * (1 + u) + u * np.abs(want))
    dy = torch.full_like(y, 5.0).cuda()
    got = mr.moe_expert_combine_bwd(dout.cuda(), y.cuda(), *args, gate.cuda(), out={"dy": dy})
    assert got["dy"] is dy
    want_dy, want_dg, size = np.full((T * k, H), 5.0), np.zeros((T, k)), np.zeros((T, k))
    yd, dd, gd = wide(y), wide(dout), wide(gate)
    for t in range(T):
        for j in range(k):
            s = slot[t * k + j]
            if s >= 0:
                r = offsets[idx[t, j]] + s
                want_dy[r] = gd[t, j] * dd[t]
                want_dg[t, j] = yd[r] @ dd[t]
                size[t, j] = np.abs(yd[r]) @ np.abs(dd[t])
    ref.assert_near("dy", wide(dy), want_dy, (u + 2 * ref.U32) * np.abs(want_dy))
    ref.assert_near("dgate", wide(got["dgate"]), want_dg, H * ref.U32 * size)


def test_misaligned_views_and_repeats(mr):
    idx, slot, offsets, y, gate, dout = make(50, 4, 8, 256, 99, torch.bfloat16)
    args = (i32(idx), i32(slot), i32(offsets))
    flat = torch.zeros(y.numel() + 1, dtype=torch.bfloat16, device="cuda")
    shifted = flat[1:].view_as(y)
    shifted.copy_(y)
    want = mr.moe_expert_combine(y.cuda(), *args, gate=gate.cuda())
    assert torch.equal(mr.moe_expert_combine(shifted, *args, gate=gate.cuda()), want)
    a = mr.moe_expert_combine_bwd(dout.cuda(), y.cuda(), *args, gate.cuda())
    b = mr.moe_expert_combine_bwd(dout.cuda(), shifted, *args, gate.cuda())
    c = mr.moe_expert_combine_bwd(dout.cuda(), y.cuda(), *args, gate.cuda())
    assert torch.equal(a["dy"], b["dy"]) and torch.equal(a["dgate"], c["dgate"])


def test_positions_outside_the_arrays_stay_inside(mr):
    idx, slot, offsets, y, gate, dout = make(20, 2, 4, 64, 99, torch.float32)
    for i, s, o in (([[9, -1]] * 20, slot, offsets), (idx, slot + (1 << 30), offsets), (idx, slot, offsets - 1000)):
        out = mr.moe_expert_combine(y.cuda(), i32(i), i32(s), i32(o), gate=gate.cuda())
        g = mr.moe_expert_combine_bwd(dout.cuda(), y.cuda(), i32(i), i32(s), i32(o), gate.cuda())
        assert not out.any() and not g["dgate"].any()


def test_a_slot_that_is_no_tensor_is_refused(mr):
    idx, slot, offsets, y, gate, dout = make(20, 2, 4, 64, 99, torch.float32)
    for bad in (None, 5, i32(slot).cpu(), i32(slot)[:-1]):
        with pytest.raises(ValueError, match="slot"):
            mr.moe_expert_combine(y.cuda(), i32(idx), bad, i32(offsets), gate=gate.cuda())
