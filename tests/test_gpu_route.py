"""GPU parity of the scored, group-limited routing and its gradient against float64.

Picks and counts are compared exactly.  Bounds of the floating outputs, with D
the row's spread of finite logits (the argument of an exponential is rounded to
2^-24 of itself, which moves the exponential by 2^-24 D of its value):
  gate     (2 D + 96) * 2^-24 of itself: two argument roundings; a sum of at most 64
           values per lane, 5 steps across lanes and 8 picks (77 roundings); ex2.approx
           (4 units of 2^-24), expf, quotient, 1 + e and scale (8)
  dlogits  the same bound twice (shares and differences of them), against the sum of the
           sizes of the gradient's terms
and FLT_MIN (times the scale) absolutely, where an exponential underflows.
"""

import numpy as np
import pytest
import torch

import experts_reference as ref

pytestmark = pytest.mark.gpu
FLT_MIN = 2.0 ** -126


@pytest.fixture(scope="module")
def mr(native_lib):
    import moe_expert_routing_router_gb300 as m
    return m


def logits_of(T, E, dtype, seed, spread=1.5):
    rng = np.random.default_rng(seed)
    z = torch.from_numpy((rng.standard_normal((T, E)) * spread + rng.standard_normal(E)).astype(np.float32))
    return z.to(dtype)


def bias_of(E, seed):
    return (np.random.default_rng(seed).integers(-150, 151, E) * 0.001).astype(np.float32)


def widen(z):
    return z.float().numpy().astype(np.float64)


def spread_of(z):
    f = np.where(np.isfinite(z), z, np.nan)
    with np.errstate(all="ignore"):
        import warnings
        with warnings.catch_warnings():
            warnings.simplefilter("ignore")
            d = np.nanmax(np.abs(f), axis=1, keepdims=True) * 2
    return np.minimum(np.nan_to_num(d), 400.0)       # beyond about 200 every exponential is 0 or 1


def check(mr, z, k, score="sigmoid", bias=None, n_groups=1, topk_groups=1, group_score="top2", renorm=True, scale=1.0, gamma=0.01):
    zd = widen(z)
    T, E = zd.shape
    b = None if bias is None else torch.from_numpy(bias).cuda()
    got = mr.moe_route_fwd(z.cuda(), k, score=score, bias=b, n_groups=n_groups, topk_groups=topk_groups,
                           group_score=group_score, renorm=int(renorm), scale=scale, bias_gamma=gamma, bias_out=True)
    idx = ref.choose(zd, k, score, bias, n_groups, topk_groups, group_score)
    gi = got["idx"].cpu().numpy()
    assert np.array_equal(gi, idx), f"{(gi != idx).any(axis=1).sum()} rows of {T} pick other experts"
    counts = np.bincount(idx.ravel(), minlength=E)
    assert np.array_equal(got["counts"].cpu().numpy(), counts)
    w = ref.pick_weights(zd, idx, score, renorm)
    eps = (2 * spread_of(zd) + 96) * ref.U32
    ref.assert_near("gate", got["gate"].cpu().numpy(), scale * w, scale * (eps * w + FLT_MIN))
    b0 = np.zeros(E, np.float32) if bias is None else bias
    want_b = (b0 + np.float32(gamma) * np.sign(T * k - counts * E).astype(np.float32)).astype(np.float32)
    assert np.array_equal(got["bias_out"].cpu().numpy(), want_b)
    return got, idx, zd


def check_bwd(mr, z, idx, score, renorm, scale, seed=3):
    zd = widen(z)
    T, k = idx.shape
    E = zd.shape[1]
    dgate = np.random.default_rng(seed).standard_normal((T, k)).astype(np.float32)
    got = mr.moe_route_bwd(z.cuda(), torch.from_numpy(idx.astype(np.int32)).cuda(), torch.from_numpy(dgate).cuda(),
                           score=score, renorm=int(renorm), scale=scale).cpu().numpy()
    want = ref.route_grad(zd, idx, dgate, score, renorm, scale)
    live = (idx >= 0) & (idx < E)
    safe = np.where(live, idx, 0)
    size = np.zeros((T, E))
    dg = np.abs(np.where(live, dgate, 0.0)).astype(np.float64) * abs(scale)
    s = ref.scores(zd, score)
    if renorm:
        zz = np.where(live, np.take_along_axis(zd, safe, 1), -np.inf)
        w = ref.pick_weights(zz, np.arange(k)[None, :].repeat(T, 0), score, True)
        term = w * (dg + (w * dg).sum(axis=1, keepdims=True))
    else:
        w = np.take_along_axis(s, safe, 1)
        term = w * dg
    for j in range(k):
        np.add.at(size, (np.arange(T), safe[:, j]), np.where(live[:, j], term[:, j], 0.0))
    if score == "softmax" and not renorm:
        size += s * (w * dg).sum(axis=1, keepdims=True)
    eps = 2 * (2 * spread_of(zd) + 96) * ref.U32
    ref.assert_near("dlogits", got, want, eps * size + 8 * abs(scale) * FLT_MIN)
    return got


SHAPES = [  # T, E, k, groups, kept groups
    (1, 256, 8, 8, 4), (33, 256, 8, 8, 4), (257, 64, 6, 8, 3), (129, 384, 6, 12, 5), (1, 1, 1, 1, 1), (70, 2, 2, 1, 1),
    (65, 60, 4, 4, 2), (31, 7, 3, 1, 1), (40, 1024, 8, 32, 8), (37, 1020, 8, 17, 5), (32, 1000, 7, 1, 1), (300, 160, 6, 8, 3),
    (50, 9, 1, 3, 1), (41, 96, 8, 32, 3), (1031, 8, 2, 1, 1), (45, 30, 5, 6, 1),
]


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("score", ["sigmoid", "softmax"])
@pytest.mark.parametrize("shape", SHAPES, ids=lambda s: "x".join(map(str, s)))
def test_routing_and_gradient(mr, shape, score, dtype):
    T, E, k, G, keep = shape
    z = logits_of(T, E, dtype, seed=T + E)
    for group_score in ("top2", "max"):
        for bias in (None, bias_of(E, 5)):
            for renorm in (True, False):
                _, idx, _ = check(mr, z, k, score, bias, G, keep, group_score, renorm, 2.5)
    for renorm in (True, False):
        check_bwd(mr, z, idx, score, renorm, 2.5)


@pytest.mark.parametrize("score", ["sigmoid", "softmax"])
@pytest.mark.parametrize("group_score", ["top2", "max"])
def test_ties_go_to_the_lower_index(mr, score, group_score):
    rng = np.random.default_rng(0)
    z = torch.from_numpy(rng.integers(-1, 2, (600, 64)).astype(np.float32)).to(torch.bfloat16)
    z[:, 3] = -0.0
    for bias in (None, np.zeros(64, np.float32), (rng.integers(-1, 2, 64) * 0.25).astype(np.float32)):
        check(mr, z, 8, score, bias, 8, 3, group_score)
        check(mr, z, 8, score, bias)


@pytest.mark.parametrize("score", ["sigmoid", "softmax"])
@pytest.mark.parametrize("grouped", [False, True])
def test_choice_values_that_fp32_cannot_tell_apart(mr, score, grouped):
    """Biases that make an expert's choice value equal another's to about one fp32
    rounding, either way: the picks are those of double precision."""
    rng = np.random.default_rng(11)
    E, T = 64, 500
    row = rng.standard_normal(E).astype(np.float32)
    s = ref.scores(row[None].astype(np.float64), score)[0]
    bias = np.zeros(E, np.float32)
    bias[1::2] = (s[0::2] - s[1::2]).astype(np.float32)           # pairs (0, 1), (2, 3), ... all but equal
    z = np.repeat(row[None], T, 0)
    z[:, 1::2] = np.nextafter(z[:, 1::2], np.where(rng.random((T, E // 2)) < 0.5, -9, 9).astype(np.float32))
    if grouped:                                                   # whole groups all but equal
        z[:, 32:] = z[:, :32]
        bias[32:] = bias[:32]
        z[:, 40] = np.nextafter(z[:, 40], np.float32(9))
    zt = torch.from_numpy(z)
    for group_score in ("top2", "max"):
        check(mr, zt, 8, score, bias, 4 if grouped else 1, 2 if grouped else 1, group_score)
    check(mr, zt, 8, score, None, 4, 2, "top2")


@pytest.mark.parametrize("shape", [(512, 8, 4), (1024, 8, 4), (96, 32, 5), (510, 17, 9)], ids=lambda s: "x".join(map(str, s)))
@pytest.mark.parametrize("biased", [False, True])
@pytest.mark.parametrize("score", ["sigmoid", "softmax"])
def test_groups_that_fp32_cannot_tell_apart(mr, shape, score, biased):
    """Groups whose two largest are another group's, or next to them, among many experts;
    in some rows groups of one expert or of none, and groups of experts all alike."""
    E, G, keep = shape
    T, gs = 700, E // G
    rng = np.random.default_rng(E + G)
    z = (rng.standard_normal((T, G, gs)) * 1.5).astype(np.float32)
    bias = np.repeat(bias_of(gs, 5)[None], G, 0).ravel() if biased else None
    for t in range(T):
        for g in range(1, G, 2):                                  # the group before it, in another order, half of them moved
            z[t, g] = z[t, g - 1] if biased else rng.permutation(z[t, g - 1])
            if rng.random() < 0.5:
                i = int(np.argmax(z[t, g]))
                z[t, g, i] = np.nextafter(z[t, g, i], np.float32(9 if rng.random() < 0.5 else -9))
    z[600:620, :, 1:] = -np.inf
    z[620:640, : G // 2] = -np.inf
    z[640:660] = z[640:660, :, :1]
    z = torch.from_numpy(z.reshape(T, E))
    for group_score in ("top2", "max"):
        check(mr, z, 4, score, bias, G, keep, group_score)
        check(mr, z.to(torch.bfloat16), 4, score, bias, G, keep, group_score)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("score", ["sigmoid", "softmax"])
def test_masked_logits(mr, score, dtype):
    T, E, k, G = 64, 64, 6, 8
    z = logits_of(T, E, dtype, seed=4)
    rng = np.random.default_rng(2)
    z[torch.from_numpy(rng.random((T, E)) < 0.5)] = -float("inf")
    z[0] = -float("inf")                                         # nothing left
    z[1] = -float("inf")
    z[1, 37] = 0.5                                               # one expert left
    z[2] = torch.finfo(dtype).min                                # the lowest finite value everywhere
    z[3, :32] = torch.finfo(dtype).min
    z[4, 10:20] = float("nan")
    z[5] = float("nan")
    z[6] = -float("inf")
    z[6, ::8] = torch.arange(8).to(dtype)                        # one expert a group
    for bias in (None, bias_of(E, 1)):
        for group_score in ("top2", "max"):
            for renorm in (True, False):
                got, idx, zd = check(mr, z, k, score, bias, G, 3, group_score, renorm)
                assert (got["gate"][0] == 0).all() and (got["gate"][5] == 0).all()
                grad = check_bwd(mr, z, idx, score, renorm, 1.0)
                assert np.isfinite(grad).all() and not grad[0].any()


@pytest.mark.parametrize("score", ["sigmoid", "softmax"])
def test_gates_keep_their_digits_where_scores_underflow(mr, score):
    z = logits_of(100, 32, torch.float32, seed=6) - 300.0
    got, _, _ = check(mr, z, 4, score, None, renorm=True)
    assert abs(got["gate"].sum(1) - 1).max() < 1e-5
    z[:, 0] = 250.0                                              # a saturated expert beside them
    check(mr, z, 4, score, None, renorm=True)
    check(mr, z, 4, score, None, renorm=False)
    check_bwd(mr, z, np.tile(np.arange(4), (100, 1)), score, True, 1.0)


def test_row_results_do_not_depend_on_the_batch(mr):
    z = logits_of(300, 256, torch.bfloat16, seed=8).cuda()
    b = torch.from_numpy(bias_of(256, 9)).cuda()
    args = dict(bias=b, n_groups=8, topk_groups=4, scale=2.5)
    whole = mr.moe_route_fwd(z, 8, **args)
    again = mr.moe_route_fwd(z, 8, **args)
    for key in whole:
        assert torch.equal(whole[key], again[key])
    for t in (0, 17, 299):
        one = mr.moe_route_fwd(z[t:t + 1].contiguous(), 8, **args)
        assert torch.equal(one["idx"][0], whole["idx"][t]) and torch.equal(one["gate"][0], whole["gate"][t])


def test_bias_in_place_and_preallocated_outputs(mr):
    z = logits_of(500, 64, torch.bfloat16, seed=1).cuda()
    for T in (20, 500):                                          # one CTA, many
        bias = torch.zeros(64, device="cuda")
        want = mr.moe_route_fwd(z[:T].contiguous(), 4, bias=bias, bias_gamma=0.5, bias_out=True)
        out = {"idx": torch.empty(T, 4, dtype=torch.int32, device="cuda"), "gate": torch.empty(T, 4, device="cuda"),
               "counts": torch.full((64,), 99, dtype=torch.int32, device="cuda")}
        got = mr.moe_route_fwd(z[:T].contiguous(), 4, bias=bias, bias_gamma=0.5, bias_out=bias, out=out)
        assert got["bias_out"] is bias and got["counts"] is out["counts"]
        for key in ("idx", "gate", "counts", "bias_out"):
            assert torch.equal(got[key], want[key]), key


@pytest.mark.parametrize("score,renorm", [("sigmoid", True), ("sigmoid", False), ("softmax", True), ("softmax", False)])
def test_gradient_of_repeated_and_foreign_picks(mr, score, renorm):
    z = logits_of(40, 33, torch.float32, seed=2)
    rng = np.random.default_rng(1)
    idx = rng.integers(0, 33, (40, 5))
    idx[:, 1] = idx[:, 0]                                        # the same expert twice
    idx[::3, 2] = -1                                             # no expert
    idx[::5, 3] = 33
    check_bwd(mr, z, idx, score, renorm, 1.5)


def test_misaligned_views(mr):
    """Logits that start two or four bytes past a vector boundary, and a gradient that does."""
    for dtype in (torch.bfloat16, torch.float32):
        flat = torch.zeros(64 * 256 + 1, dtype=dtype, device="cuda")
        z = flat[1:].view(64, 256)
        z.copy_(logits_of(64, 256, dtype, seed=3))
        want = mr.moe_route_fwd(z.clone(), 8, n_groups=8, topk_groups=4)
        got = mr.moe_route_fwd(z, 8, n_groups=8, topk_groups=4)
        assert all(torch.equal(got[k], want[k]) for k in got)
        dg = torch.randn(64, 8, device="cuda")
        dl = torch.zeros(64 * 256 + 1, device="cuda")[1:].view(64, 256)
        for score, renorm in (("sigmoid", 1), ("softmax", 0)):
            a = mr.moe_route_bwd(z, got["idx"], dg, score=score, renorm=renorm, dlogits=dl)
            assert torch.equal(a, mr.moe_route_bwd(z.clone(), got["idx"], dg, score=score, renorm=renorm))


def test_captured_and_replayed_on_another_stream(mr):
    z = logits_of(200, 64, torch.bfloat16, seed=5).cuda()
    bias = torch.zeros(64, device="cuda")
    out = {"idx": torch.empty(200, 4, dtype=torch.int32, device="cuda"), "gate": torch.empty(200, 4, device="cuda"),
           "counts": torch.empty(64, dtype=torch.int32, device="cuda")}
    dl = torch.empty(200, 64, device="cuda")
    dg = torch.randn(200, 4, device="cuda")
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=s):
        mr.moe_route_fwd(z, 4, bias=bias, bias_gamma=0.01, bias_out=bias, out=out, stream=s)
        mr.moe_route_bwd(z, out["idx"], dg, dlogits=dl, stream=s)
    b = torch.zeros(64, device="cuda")
    for step in range(3):
        z.copy_(logits_of(200, 64, torch.bfloat16, seed=50 + step))
        g.replay()
        want = mr.moe_route_fwd(z, 4, bias=b, bias_gamma=0.01, bias_out=True)
        b = want["bias_out"]
        torch.cuda.synchronize()
        assert torch.equal(out["idx"], want["idx"]) and torch.equal(out["counts"], want["counts"]) and torch.equal(bias, b)
        assert torch.equal(dl, mr.moe_route_bwd(z, want["idx"], dg))


def test_a_large_batch_and_64_bit_offsets(mr):
    """T * E passes 2^31 elements; rows at both ends are compared."""
    T, E, k = 2 ** 23 + 5, 264, 4
    z = torch.zeros(T, E, dtype=torch.bfloat16, device="cuda")
    part = logits_of(300, E, torch.bfloat16, seed=12)
    z[-300:] = part.cuda()
    z[:300] = part.cuda()
    got = mr.moe_route_fwd(z, k, n_groups=8, topk_groups=3)
    want = mr.moe_route_fwd(part.cuda(), k, n_groups=8, topk_groups=3)
    for at in (slice(0, 300), slice(T - 300, T)):
        assert torch.equal(got["idx"][at], want["idx"]) and torch.equal(got["gate"][at], want["gate"])
    assert int(got["counts"].sum()) == T * k
    dg = torch.ones(T, k, device="cuda")
    dg[-300:] = torch.randn(300, k, device="cuda")
    d = mr.moe_route_bwd(z, got["idx"], dg)
    assert torch.equal(d[-300:], mr.moe_route_bwd(part.cuda(), want["idx"], dg[-300:].contiguous()))


@pytest.mark.parametrize("E,G", [(256, 8), (64, 1), (1024, 32), (40, 5)])
def test_counts_and_bias_of_every_way_to_launch(mr, E, G):
    """One CTA, one cluster, many CTAs, and both sides of where they change over."""
    for T in (1, 8, 16, 17, 32, 33, 64, 65, 128, 129, 256, 257, 512, 513, 700):
        z = logits_of(T, E, torch.bfloat16, seed=T)
        check(mr, z, 4, "sigmoid", bias_of(E, 5), G, max(1, G // 2))


def test_bias_in_place_of_one_cluster(mr):
    """The bias that the rows read is overwritten only behind the last row."""
    T, E = 300, 256
    z, bias = logits_of(T, E, torch.float32, 4), bias_of(E, 6)
    want = mr.moe_route_fwd(z.cuda(), 8, bias=torch.from_numpy(bias).cuda(), n_groups=8, topk_groups=4, bias_gamma=0.5, bias_out=True)
    for _ in range(20):
        b = torch.from_numpy(bias).cuda()
        got = mr.moe_route_fwd(z.cuda(), 8, bias=b, n_groups=8, topk_groups=4, bias_gamma=0.5, bias_out=b)
        assert torch.equal(b, want["bias_out"]) and torch.equal(got["idx"], want["idx"]) and torch.equal(got["counts"], want["counts"])


@pytest.mark.parametrize("grouped", [False, True])
@pytest.mark.parametrize("copies", [1, 2, 3, 7, 40])
def test_a_larger_value_behind_equal_ones(mr, copies, grouped):
    """Experts with the same logit and bias, and behind them one whose choice value is larger only in
    double precision."""
    T, E = 70, 96
    z = np.full((T, E), -2.0, np.float32)
    bias = np.full(E, 0.1, np.float32)
    bias[7] = 0.2
    z[:, 7] = 3.5625
    at = np.r_[10:10 + copies]
    z[:, at] = 17.125
    z[::2, 60], z[1::2, 61] = 19.125, 18.0
    for k in (1, 2, 3, 8):
        check(mr, torch.from_numpy(z), k, "sigmoid", bias, 4 if grouped else 1, 3 if grouped else 1, "max")
        check(mr, torch.from_numpy(z).to(torch.bfloat16), k, "sigmoid", bias, 4 if grouped else 1, 3 if grouped else 1, "top2")


@pytest.mark.parametrize("score", ["sigmoid", "softmax"])
@pytest.mark.parametrize("size", [10.0, 64.0, 1000.0, 4096.0, 1e6])
def test_groups_of_large_biases_that_cancel(mr, score, size):
    """A group's two largest of opposite sign and far larger than their sum: fp32 rounds each in
    proportion to its own size, and the groups taken are those of double precision."""
    rng = np.random.default_rng(int(size))
    for T, G, gs, keep in ((1500, 2, 2, 1), (700, 8, 2, 3), (300, 4, 5, 2)):
        z = np.tile(rng.standard_normal((T, 1, gs)), (1, G, 1))
        z = z + rng.uniform(-4, 4, (T, G, gs)) * size * 2.0 ** -24        # apart by what fp32 rounds the choice values by
        bias = np.full((G, gs), -2 * size, np.float32)
        bias[:, 0], bias[:, 1] = size, -size
        zt = torch.from_numpy(z.reshape(T, G * gs).astype(np.float32))
        for group_score in ("top2", "max"):
            check(mr, zt, 1, score, bias.ravel(), G, keep, group_score)
            check(mr, zt.to(torch.bfloat16), 2, score, bias.ravel(), G, keep, group_score)
        spread = rng.uniform(-size, size, G * gs).astype(np.float32)
        check(mr, zt, 2, score, spread, G, keep, "top2")
    z = torch.tensor([[0.0008, 0, 0, 0.00076]])
    bias = np.array([4096, -4096, 4096, -4096], np.float32)
    check(mr, z, 1, score, bias, 2, 1, "top2")
    check(mr, torch.tensor([[-0.377855, 1.951048, 0.551829, 0.608678]]), 1, score, np.array([1000.1, -1000, 900.1, -900], np.float32), 2, 1, "top2")


@pytest.mark.parametrize("score", ["sigmoid", "softmax"])
def test_groups_whose_sums_pass_fp32(mr, score):
    """Choice values near the largest fp32 number: their sums order groups as double precision has them."""
    z = logits_of(60, 12, torch.float32, seed=3)
    big = np.array([3.0e38, 2.9e38, -3e38, 3.1e38, 3.05e38, 0, 3.2e38, 3.3e38, 1, 3e38, -2e38, -3e38], np.float32)
    for bias in (big, np.roll(big, 3), -big):
        for keep in (1, 2, 3):
            check(mr, z, 2, score, bias, 4, keep, "top2")
            check(mr, z, 2, score, bias, 4, keep, "max")


@pytest.mark.parametrize("E,G", [(32, 8), (256, 8)])
def test_sigmoid_scores_at_the_end_of_double_precision(mr, E, G):
    """Scores between 1e-313 and 1e-305, which fp32 holds as 0: in their order all the same."""
    rng = np.random.default_rng(E)
    z = torch.from_numpy(rng.uniform(-720, -704, (200, E)).astype(np.float32))
    for bias in (None, np.zeros(E, np.float32)):
        check(mr, z, 4, "sigmoid", bias, G, 3, "top2")
        check(mr, z, 4, "sigmoid", bias, G, 3, "max")


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("E", [33, 100, 256, 384, 1000])
def test_softmax_gradient_of_confident_rows(mr, E, dtype):
    """A pick that has all of its row but 1e-4 to 1e-9: its gradient keeps the digits of what is left.
    Bound: a pick's is p (D r + sum_j p_j (D - D_j)) over the other picks, r the share of what is not
    picked and D an expert's sum of dgate; each share is off by (2 d + 96) 2^-24, d the row's spread,
    two of them are multiplied, and 16 roundings cover the sums over picks."""
    rng = np.random.default_rng(E)
    gaps = np.repeat([6.0, 10.0, 12.0, 14.0, 16.0, 18.0, 20.0], 8)
    T = len(gaps)
    z = rng.uniform(-1, 1, (T, E)) * 0.5
    top = rng.integers(0, E, T)
    z[np.arange(T), top] = gaps
    z = torch.from_numpy(z.astype(np.float32)).to(dtype)
    zd = widen(z)
    s = ref.scores(zd, "softmax")
    eps = (2 * (2 * (zd.max(1) - zd.min(1)) + 96) + 16)[:, None] * ref.U32
    for picks in (1, 2, 5, 8):
        idx = np.stack([rng.permutation(E)[:picks] for _ in range(T)])
        idx[:, 0] = top
        idx[::4, -1] = top[::4]                                      # the same expert twice
        idx[1::7, -1] = E                                            # no expert
        dgate = rng.standard_normal((T, picks)).astype(np.float32)
        got = mr.moe_route_bwd(z.cuda(), torch.from_numpy(idx.astype(np.int32)).cuda(), torch.from_numpy(dgate).cuda(),
                               score="softmax", renorm=0, scale=1.5).cpu().numpy()
        want = ref.route_grad(zd, idx, dgate, "softmax", False, 1.5)
        D, picked = np.zeros((T, E)), np.zeros((T, E), bool)
        for j in range(picks):
            live = idx[:, j] < E
            np.add.at(D, (np.arange(T)[live], idx[live, j]), 1.5 * dgate[live, j])
            picked[np.arange(T)[live], idx[live, j]] = True
        rest = np.where(picked, 0, s).sum(1, keepdims=True)
        size = s * (s * np.abs(D)).sum(1, keepdims=True)
        for t in range(T):
            for e in np.flatnonzero(picked[t]):
                o = picked[t].copy()
                o[e] = False
                size[t, e] = s[t, e] * (abs(D[t, e]) * rest[t, 0] + (s[t, o] * (abs(D[t, e]) + np.abs(D[t, o]))).sum())
        ref.assert_near("dlogits", got, want, eps * size + 8 * FLT_MIN)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("score", ["sigmoid", "softmax"])
@pytest.mark.parametrize("shift", [-300.0, -80.0, 0.0, 60.0])
def test_gates_within_the_spread_of_the_row(mr, shift, score, dtype):
    """Gates lose no digits by where a row's logits lie, only by how far they lie apart.  In units of
    2^-24 of a gate:
      shares     an exponential's argument z - max is rounded (d, the picks' spread, at most), expf
                 is off by 4, a sigmoid's own exponential, sum and quotient by 6: d + 10 on either
                 side of the share; 8 sums, quotient and scale: 2 d + 32
      softmax    d + 4 of the own exponential; the row's sum: arguments rounded three times, at the
                 mean distance from the maximum, below ln 1024 + 1 = 8: 24; ex2.approx 4; at most 23
                 additions; quotient and scale: d + 58
      sigmoid    exponential 4 on either side of 1 + e, sum, quotient and scale: 12
    and the smallest normal number where an exponential underflows."""
    for E, wide_by in ((24, 1.0), (256, 1.5), (1000, 2.0), (64, 15.0)):
        z = (logits_of(200, E, torch.float32, seed=E, spread=wide_by) + shift).to(dtype)
        zd = widen(z)
        for k in (1, 4, 8):
            for renorm in (True, False):
                got = mr.moe_route_fwd(z.cuda(), k, score=score, renorm=int(renorm), scale=2.5)
                idx = ref.choose(zd, k, score)
                assert np.array_equal(got["idx"].cpu().numpy(), idx)
                zp = np.take_along_axis(zd, idx, 1)
                d = zp.max(1, keepdims=True) - zp.min(1, keepdims=True)
                if renorm:
                    units = 2 * d + 32
                elif score == "softmax":
                    units = zd.max(1, keepdims=True) - zp + 58
                else:
                    units = 12
                w = ref.pick_weights(zd, idx, score, renorm)
                ref.assert_near("gate", got["gate"].cpu().numpy(), 2.5 * w, 2.5 * (units * ref.U32 * w + FLT_MIN))


@pytest.mark.parametrize("score", ["sigmoid", "softmax"])
def test_banned_groups_beside_masked_ones(mr, score):
    """Groups whose two largest sum below fp32's range, beside groups whose experts are all masked: the
    former come first, in the order of their sums."""
    z = logits_of(40, 12, torch.float32, seed=5)
    bias = np.full(12, -3.2e38, np.float32)
    bias[8:10], bias[6:8] = -3.1e38, -3.0e38
    for masked in ((0, 1), (0, 1, 4, 5), (4, 5, 10, 11), (0, 4, 8)):
        zm = z.clone()
        zm[:, list(masked)] = -float("inf")
        for keep in (1, 2, 3, 4, 5):
            check(mr, zm, 2, score, bias, 6, keep, "top2")
            check(mr, zm, 1, score, np.roll(bias, 3), 6, keep, "max")
