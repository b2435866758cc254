"""The gated activation's gradient where the product of two of its three factors passes fp32 and that of all three does not,
by the bounds of test_gpu_glu."""

import numpy as np
import pytest
import torch

import experts_reference as experts_ref
import layer_reference as ref
from test_gpu_glu import DTYPES, half_step, roundings, wide

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def mr(native_lib):
    import moe_expert_routing_router_gb300 as m
    return m


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("dy,u", [(1e30, 1e30), (-1e38, 1e4), (3e20, -3e38), (2.0, 3.3e38)])
def test_large_factors_of_a_small_slope(mr, dtype, dy, u):
    M, I = 3, 96
    g = -torch.linspace(1.0, 85.0, I).repeat(M, 1)                # slopes from 0.07 to 1e-35
    h = torch.cat([g, torch.full((M, I), u)], 1).to(dtype)
    d = torch.full((M, I), dy).to(dtype)
    got = wide(mr.moe_expert_glu_bwd(h.cuda(), d.cuda()))[:, :I]
    hw, dw = wide(h), wide(d)
    gw, uw = np.split(hw, 2, axis=1)
    want = ref.glu_bwd(hw, dw)[:, :I]
    s, c = ref.sigmoid(gw), ref.sigmoid(-gw)
    n = roundings(gw, dtype) * ref.U32
    size = np.abs(dw * uw) * s * (1 + np.abs(gw) * c)            # of the two terms of 1 + g (1 - s), which may cancel
    near = np.abs(want) < 3.3e38                                 # finite in either type
    assert near.any() and (np.abs(dw * uw) > 3.5e38).all()
    bound = size * (2 * n + 4 * ref.U32) * (1 + ref.U16) + half_step(want, dtype)
    experts_ref.assert_near("dg", got[near], want[near], bound[near])
    past = np.abs(want) > 3.5e38
    assert np.array_equal(got[past], np.sign(want[past]) * np.inf)
