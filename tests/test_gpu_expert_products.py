"""GPU parity of the block-scaled quantisation, the experts' products and their weight gradient against float64.

Codes and scales are compared exactly.  Bounds of the products, against the sum
of the sizes of an element's terms: the tensor core adds a block's 128 products
in fp32 (at most 2^-23 of the running size each), the blocks' sums are scaled
(two roundings) and added (one each): (256 + 3 * blocks) * 2^-24; and half a
step of bf16, 2^-8 of the value, for a bf16 result.  Where every sum is a whole
number below 2^24 the result has to be exact.
"""

import numpy as np
import pytest
import torch

import experts_reference as ref

pytestmark = pytest.mark.gpu
F8 = torch.float8_e4m3fn


@pytest.fixture(scope="module")
def mr(native_lib):
    import moe_expert_routing_router_gb300 as m
    yield m
    assert m.moe_expert_device_status() == 0


def values(shape, seed, dtype=torch.bfloat16, sigma=1.0):
    g = torch.Generator().manual_seed(seed)
    x = torch.randn(*shape, generator=g) * sigma * torch.exp(0.8 * torch.randn(shape[0], *([1] * (len(shape) - 1)), generator=g))
    return x.to(dtype)


def wide(t):
    return t.float().cpu().numpy().astype(np.float64)


def i32(a):
    return torch.as_tensor(np.asarray(a), dtype=torch.int32).cuda()


def split(counts, kept=None):
    offsets = np.concatenate([[0], np.cumsum(counts)])
    return i32(offsets), None if kept is None else i32(kept), ref.expert_rows(offsets, kept, int(offsets[-1]))


# -- quantisation ------------------------------------------------------------------

@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("M,K", [(1, 16), (1, 128), (33, 144), (100, 512), (7, 1040), (65, 2064)])
def test_rows(mr, M, K, dtype):
    x = values((M, K), M + K, dtype)
    x[0, :16] = 0
    if K > 128:
        x[-1, :128] = 0                                          # a block of zeros
    got = mr.moe_quantize_rows(x.cuda())
    q, scale = ref.quantize_rows(wide(x))
    assert np.array_equal(wide(got["q"]), q) and np.array_equal(wide(got["scale"]), scale)


def test_rows_gathered(mr):
    T, k, E, K = 70, 3, 8, 272
    rng = np.random.default_rng(0)
    idx = np.stack([rng.permutation(E)[:k] for _ in range(T)])
    perm, _, _, _ = ref.dispatch(idx, E, 1000)
    x = values((T, K), 1)
    got = mr.moe_quantize_rows(x.cuda(), perm=i32(perm), k=k)
    q, scale = ref.quantize_rows(wide(x)[perm // k])
    assert np.array_equal(wide(got["q"]), q) and np.array_equal(wide(got["scale"]), scale)
    bad = perm.copy()
    bad[5], bad[6] = -1, T * k                                   # outside x: zeros
    got = mr.moe_quantize_rows(x.cuda(), perm=i32(bad), k=k)
    assert not wide(got["q"])[5:7].any() and (wide(got["scale"])[:, 5:7] == 1).all()


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_every_rounding_and_scale(mr, dtype):
    """All bf16 magnitudes next to a block maximum, values half-way between codes, tiny and huge blocks."""
    top = torch.tensor([448.0, 447.0, 449.0, 2.0 ** -133, 2.0 ** -126, 1.75 * 2.0 ** -120, 3.0e38, 1.0])
    x = torch.zeros(8 * 64, 128)
    codes = torch.from_numpy(ref.e4m3_values()).float()
    mid = (codes[:-1] + codes[1:]) / 2                           # ties
    for i in range(8 * 64):
        m = float(top[i // 64])
        g = torch.Generator().manual_seed(i)
        x[i] = torch.randn(128, generator=g) * m / 8
        if i % 4 == 0:
            x[i, :126] = mid[torch.randperm(126, generator=g)] * (2.0 ** torch.floor(torch.log2(torch.tensor(m))) / 256)
        x[i] = x[i].clamp(-m, m)
        x[i, 5] = m if i % 2 else -m
    x = x.to(dtype)
    got = mr.moe_quantize_rows(x.cuda())
    q, scale = ref.quantize_rows(wide(x))
    assert np.array_equal(wide(got["scale"]), scale)
    assert np.array_equal(wide(got["q"]), q)


def test_not_finite_blocks(mr):
    x = values((5, 384), 3, torch.float32)
    x[1, 130], x[2, 0], x[3, 383] = float("nan"), float("inf"), -float("inf")
    got = mr.moe_quantize_rows(x.cuda())
    s = wide(got["scale"])
    bad = np.zeros((3, 5), bool)
    bad[1, 1] = bad[0, 2] = bad[2, 3] = True
    assert np.array_equal(np.isnan(s), bad)
    ok = ref.quantize_rows(np.nan_to_num(wide(x), nan=0, posinf=0, neginf=0))
    assert np.array_equal(wide(got["q"])[[0, 4]], ok[0][[0, 4]])


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("counts,kept,K", [([1], None, 16), ([5, 0, 300, 128], None, 144), ([129, 127, 256, 1], [100, 127, 129, 0], 64),
                                           ([0, 0, 3], None, 80), ([40] * 70, [33] * 70, 32)])
def test_cols(mr, counts, kept, K, dtype):
    M, E = sum(counts), len(counts)
    x = values((M, K), M, dtype)
    x[:, 3] = 0
    offsets, kt, rows = split(counts, kept)
    width = mr.moe_quantize_cols_width(M, E)
    out = {"q": torch.full((K, width), 2.0, device="cuda").to(F8), "scale": torch.full((width // 128, K), 7.0, device="cuda")}
    mr.moe_quantize_cols(x.cuda(), offsets, kt, out=out)
    q, scale = ref.quantize_cols(wide(x), rows)
    n = q.shape[1]
    assert np.array_equal(wide(out["q"])[:, :n], q) and np.array_equal(wide(out["scale"])[:n // 128], scale)
    assert (wide(out["q"])[:, n:] == 2).all() and (wide(out["scale"])[n // 128:] == 7).all()     # left as they were
    if kept is None:
        token = np.random.default_rng(1).permutation(M * 2)[:M]                                  # gathered rows
        got = mr.moe_quantize_cols(x.cuda(), offsets, None, perm=i32(token), k=2)
        q, scale = ref.quantize_cols(wide(x)[token // 2], rows)
        assert np.array_equal(wide(got["q"])[:, :n], q) and np.array_equal(wide(got["scale"])[:n // 128], scale)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("E,N,K", [(1, 16, 16), (2, 128, 256), (3, 144, 272), (2, 272, 112)])
def test_weights(mr, E, N, K, dtype):
    w = values((E, N, K), N, dtype, 0.02)
    w[0, :128, :128] = 0
    got = mr.moe_quantize_weights(w.cuda(), transposed=True)
    q, scale = ref.quantize_weights(wide(w))
    assert np.array_equal(wide(got["q"]), q) and np.array_equal(wide(got["scale"]), scale)
    assert np.array_equal(wide(got["qt"]), q.transpose(0, 2, 1)) and np.array_equal(wide(got["scalet"]), scale.transpose(0, 2, 1))
    plain = mr.moe_quantize_weights(w.cuda())
    assert set(plain) == {"q", "scale"} and torch.equal(plain["q"].view(torch.uint8), got["q"].view(torch.uint8))


# -- products ------------------------------------------------------------------------

def operands(M, K, E, N, seed):
    g = torch.Generator().manual_seed(seed)
    q = (torch.randn(M, K, generator=g) * 60).clamp(-448, 448).to(F8).cuda()
    wq = (torch.randn(E, N, K, generator=g) * 60).clamp(-448, 448).to(F8).cuda()
    # any fp32 scales, not only powers of two
    scale = torch.exp(torch.randn(-(-K // 128), M, generator=g)).cuda()
    wscale = torch.exp(torch.randn(E, -(-N // 128), -(-K // 128), generator=g)).cuda()
    return q, scale, wq, wscale


def check_matmul(mr, counts, kept, K, N, dtype, seed=0):
    M, E = sum(counts), len(counts)
    q, scale, wq, wscale = operands(M, K, E, N, seed)
    offsets, kt, rows = split(counts, kept)
    out = torch.full((M, N), 3.0, dtype=dtype, device="cuda")
    got = mr.moe_expert_matmul(q, scale, wq, wscale, offsets, kt, out=out)
    assert got is out
    want, size = ref.matmul(wide(q), wide(scale), wide(wq), wide(wscale), rows)
    untouched = np.isnan(want)
    assert (wide(got)[untouched] == 3).all()
    bound = (256 + 3 * (-(-K // 128))) * ref.U32 * size
    if dtype == torch.bfloat16:
        bound = bound * (1 + ref.U16) + ref.U16 * np.abs(want)
    ref.assert_near("out", np.where(untouched, 0, wide(got)), np.where(untouched, 0, want), np.nan_to_num(bound))
    return got


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("counts,kept,K,N", [
    ([1], None, 16, 16), ([128], None, 128, 128), ([3, 0, 1], None, 144, 48), ([130, 5, 64], [129, 0, 64], 272, 272),
    ([1] * 8, None, 512, 528), ([300, 17, 0, 200], None, 1040, 144), ([40] * 9, [33] * 9, 640, 256), ([257], None, 2064, 304),
    ([700, 650, 1], [700, 600, 1], 384, 512), ([2] * 200, None, 144, 64),
])
def test_matmul(mr, counts, kept, K, N, dtype):
    check_matmul(mr, counts, kept, K, N, dtype, seed=N)


def test_whole_number_products_are_exact(mr):
    """Sums that fp32 holds exactly: nothing may be lost in the tensor core or the registers."""
    g = torch.Generator().manual_seed(1)
    for M, K, E, N in ((200, 4096, 2, 256), (3, 1024, 3, 144)):
        q = torch.randint(-8, 9, (M, K), generator=g).float().to(F8).cuda()
        wq = torch.randint(-8, 9, (E, N, K), generator=g).float().to(F8).cuda()
        scale = 2.0 ** torch.randint(0, 3, (K // 128, M), generator=g).float().cuda()
        wscale = 2.0 ** torch.randint(0, 2, (E, -(-N // 128), K // 128), generator=g).float().cuda()
        offsets, _, rows = split([M // E] * (E - 1) + [M - M // E * (E - 1)])
        got = mr.moe_expert_matmul(q, scale, wq, wscale, offsets, out_dtype=torch.float32)
        want, size = ref.matmul(wide(q), wide(scale), wide(wq), wide(wscale), rows)
        assert size.max() < 2 ** 24 and np.array_equal(wide(got), want)


def test_plain_product_without_offsets(mr):
    q, scale, wq, wscale = operands(77, 400, 1, 208, 5)
    got = mr.moe_expert_matmul(q, scale, wq, wscale)
    want = mr.moe_expert_matmul(q, scale, wq, wscale, i32([0, 77]))
    assert torch.equal(got, want) and got.dtype == torch.bfloat16


def test_rows_do_not_depend_on_one_another(mr):
    """A row alone, among few and among many (both tile widths): the same bits.  Not-a-number codes in
    other rows, dropped ones and behind the last stay there."""
    K, N, E = 512, 384, 2
    q, scale, wq, wscale = operands(600, K, E, N, 9)
    offsets, kept, _ = split([300, 300], [250, 300])
    base = mr.moe_expert_matmul(q, scale, wq, wscale, offsets, kept, out_dtype=torch.float32)
    bad = q.clone()
    bad.view(torch.uint8)[7] = 0x7f
    bad.view(torch.uint8)[250:300] = 0x7f
    scale2 = scale.clone()
    scale2[2, 11] = float("nan")
    out = torch.zeros(600, N, device="cuda")
    got = mr.moe_expert_matmul(bad, scale2, wq, wscale, offsets, kept, out=out)
    keep = torch.ones(600, dtype=torch.bool, device="cuda")
    keep[7] = keep[11] = False
    keep[250:300] = False
    assert torch.equal(got[keep], base[keep]) and got[7].isnan().all() and got[11].isnan().all() and not got[250:300].any()
    for r in (0, 249, 300, 599):
        one = mr.moe_expert_matmul(q[r:r + 1].contiguous(), scale[:, r:r + 1].contiguous(), wq, wscale,
                                   i32([0, 1, 1] if r < 300 else [0, 0, 1]), out_dtype=torch.float32)
        assert torch.equal(one[0], base[r])


def test_positions_outside_the_arrays_stay_inside(mr):
    """Offsets and counts that do not belong to the arrays give some result, and no access outside."""
    q, scale, wq, wscale = operands(64, 128, 3, 64, 2)
    for offsets, kept in (([0, 900, 64, 64], [9, 9, 9]), ([-5, 30, 20, 1 << 30], None), ([64, 64, 64, 64], None),
                          ([0, 10, 20, 30], [-3, 1 << 30, 5])):
        mr.moe_expert_matmul(q, scale, wq, wscale, i32(offsets), None if kept is None else i32(kept))
        mr.moe_quantize_cols(values((64, 64), 1).cuda(), i32(offsets), None if kept is None else i32(kept))
    torch.cuda.synchronize()
    d = torch.zeros(32, 256, device="cuda").to(F8)
    s = torch.ones(2, 32, device="cuda")
    for kept in ([1 << 30, 5, 7], [-1, 300, 1], [256, 256, 256]):
        mr.moe_expert_wgrad(d, s, d, s, i32(kept))
    torch.cuda.synchronize()


@pytest.mark.parametrize("counts,kept,N,K", [([1], None, 16, 16), ([128, 128], None, 128, 256), ([5, 0, 300, 129], None, 144, 272),
                                             ([0, 0], None, 32, 48), ([260, 70, 600], [200, 70, 513], 304, 528), ([40] * 20, None, 64, 320)])
def test_wgrad(mr, counts, kept, N, K):
    M, E = max(sum(counts), 1), len(counts)
    offsets, kt, rows = split(counts, kept)
    dy, x = values((M, N), 1, sigma=0.01), values((M, K), 2)
    # not-a-number in the columns behind the last expert's must not be read into any sum
    width = mr.moe_quantize_cols_width(M, E)
    outs = [{"q": torch.full((c, width), float("nan"), device="cuda").to(F8), "scale": torch.full((width // 128, c), float("nan"), device="cuda")} for c in (N, K)]
    dq = mr.moe_quantize_cols(dy.cuda(), offsets, kt, out=outs[0])
    xq = mr.moe_quantize_cols(x.cuda(), offsets, kt, out=outs[1])
    kt = kt if kt is not None else i32(counts)
    got = mr.moe_expert_wgrad(dq["q"], dq["scale"], xq["q"], xq["scale"], kt)
    d64, x64 = ref.quantize_cols(wide(dy), rows), ref.quantize_cols(wide(x), rows)
    want, size = ref.wgrad(*d64, *x64, rows)
    blocks = max(-(-n // 128) for _, n in rows) if rows else 0
    ref.assert_near("dw", wide(got), want, (256 + 3 * blocks) * ref.U32 * size)
    for e, (_, n) in enumerate(rows):
        if n == 0:
            assert not wide(got)[e].any()


def test_wgrad_with_any_scales(mr):
    g = torch.Generator().manual_seed(3)
    N, K, counts = 160, 288, [200, 128, 10]
    rows = ref.expert_rows(np.concatenate([[0], np.cumsum(counts)]), None, sum(counts))
    width = mr.moe_quantize_cols_width(sum(counts), 3)
    dq, xq = ((torch.randn(n, width, generator=g) * 40).clamp(-448, 448).to(F8).cuda() for n in (N, K))
    ds, xs = (torch.exp(torch.randn(width // 128, n, generator=g)).cuda() for n in (N, K))
    got = mr.moe_expert_wgrad(dq, ds, xq, xs, i32(counts))
    want, size = ref.wgrad(wide(dq), wide(ds), wide(xq), wide(xs), rows)
    ref.assert_near("dw", wide(got), want, (256 + 3 * 2) * ref.U32 * size)


def test_results_past_32_bit_offsets(mr):
    """Operand and result positions past 2^31; rows at both ends are compared with a small call's."""
    M, K, N = 2 ** 31 // 4096 + 300, 4096, 4112
    part = torch.randint(-8, 9, (300, K), generator=torch.Generator().manual_seed(0)).float().to(F8).cuda()
    q = torch.zeros(M, K, dtype=torch.uint8, device="cuda").view(F8)
    q.view(torch.uint8)[:300] = part.view(torch.uint8)
    q.view(torch.uint8)[-300:] = part.view(torch.uint8)
    scale = torch.ones(K // 128, M, device="cuda")
    _, _, wq, wscale = operands(1, K, 1, N, 1)
    got = mr.moe_expert_matmul(q, scale, wq, wscale)
    want = mr.moe_expert_matmul(part, torch.ones(K // 128, 300, device="cuda"), wq, wscale)
    assert torch.equal(got[:300], want) and torch.equal(got[-300:], want)
    x = torch.zeros(M, K, dtype=torch.bfloat16, device="cuda")
    x[-300:] = part.to(torch.bfloat16)
    r = mr.moe_quantize_rows(x)
    w = mr.moe_quantize_rows(x[-300:].contiguous())
    assert torch.equal(r["q"][-300:].view(torch.uint8), w["q"].view(torch.uint8)) and torch.equal(r["scale"][:, -300:], w["scale"])


def test_captured_and_concurrent_calls(mr):
    """Two graphs on two streams at once, and eager calls beside them: no state is shared."""
    sets = []
    for i in range(2):
        q, scale, wq, wscale = operands(300, 512, 4, 256, 20 + i)
        offsets, kept, _ = split([100, 0, 150, 50], [90, 0, 150, 50])
        out = torch.zeros(300, 256, dtype=torch.bfloat16, device="cuda")
        want = mr.moe_expert_matmul(q, scale, wq, wscale, offsets, kept, out=torch.zeros_like(out))
        sets.append((q, scale, wq, wscale, offsets, kept, out, want))
    graphs = []
    streams = [torch.cuda.Stream() for _ in sets]
    torch.cuda.synchronize()
    for s, (q, scale, wq, wscale, offsets, kept, out, _) in zip(streams, sets):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, stream=s):
            for _ in range(3):
                mr.moe_expert_matmul(q, scale, wq, wscale, offsets, kept, out=out, stream=s)
        graphs.append(g)
    for _ in range(5):
        for s, g in zip(streams, graphs):
            with torch.cuda.stream(s):
                g.replay()
        mr.moe_expert_matmul(*sets[0][:6], out=torch.zeros_like(sets[0][6]))
    torch.cuda.synchronize()
    for *_, out, want in sets:
        assert torch.equal(out, want)


def test_an_expired_wait_is_reported(mr, native_lib):
    """A pipeline wait made to run out (1 ms, an arrival that never comes): the status
    tells, later calls write nothing until it is read, then calls work again."""
    q, scale, wq, wscale = operands(200, 1024, 1, 256, 4)
    want = mr.moe_expert_matmul(q, scale, wq, wscale)
    torch.cuda.synchronize()
    assert mr.moe_expert_device_status() == 0
    native_lib.moe_set_wait_timeout_ns(1_000_000)
    native_lib.moe_set_unreachable_barriers(1)
    try:
        mr.moe_expert_matmul(q, scale, wq, wscale)
        torch.cuda.synchronize()
    finally:
        native_lib.moe_set_unreachable_barriers(0)
        native_lib.moe_set_wait_timeout_ns(0)
    out = torch.full((200, 256), 5.0, dtype=torch.bfloat16, device="cuda")
    mr.moe_expert_matmul(q, scale, wq, wscale, out=out)
    assert (out == 5).all()
    assert mr.moe_expert_device_status() == 2
    assert mr.moe_expert_device_status() == 0
    assert torch.equal(mr.moe_expert_matmul(q, scale, wq, wscale, out=out), want)


def test_an_expired_wait_of_the_weight_gradient(mr, native_lib):
    """As above for the kernel that copies scales beside the operands."""
    counts = [900, 0, 300]
    offsets, kept, _ = split(counts, counts)
    gen = torch.Generator().manual_seed(8)
    x = torch.randn(1200, 512, generator=gen).to(torch.bfloat16).cuda()
    dy = torch.randn(1200, 256, generator=gen).to(torch.bfloat16).cuda()
    a, b = mr.moe_quantize_cols(dy, offsets, kept), mr.moe_quantize_cols(x, offsets, kept)
    args = (a["q"], a["scale"], b["q"], b["scale"], kept)
    want = mr.moe_expert_wgrad(*args)
    torch.cuda.synchronize()
    native_lib.moe_set_wait_timeout_ns(1_000_000)
    native_lib.moe_set_unreachable_barriers(1)
    try:
        mr.moe_expert_wgrad(*args)
        torch.cuda.synchronize()
    finally:
        native_lib.moe_set_unreachable_barriers(0)
        native_lib.moe_set_wait_timeout_ns(0)
    assert mr.moe_expert_device_status() == 2
    assert torch.equal(mr.moe_expert_wgrad(*args), want)
    assert mr.moe_expert_device_status() == 0


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("K", [2048, 1040])
def test_cols_of_many_tiles(mr, K, dtype):
    """More tiles than CTAs at once.  Columns in blocks of 128 rows are the rows, in blocks of 128, of
    the transposed matrix that has each expert's rows filled up with zeros."""
    counts, kept_counts, k = [9000, 0, 127, 4000, 1, 7000], [9000, 0, 100, 3900, 1, 0], 2
    offsets, kept, _ = split(counts, kept_counts)
    M = sum(counts)
    gen = torch.Generator().manual_seed(K)
    x = (torch.randn(M // k + 1, K, generator=gen) * 3).to(dtype).cuda()
    perm = torch.randint(0, x.shape[0] * k, (M,), generator=gen).int().cuda()
    out = {"q": torch.full((K, mr.moe_quantize_cols_width(M, len(counts))), 77, dtype=torch.uint8, device="cuda").view(torch.float8_e4m3fn),
           "scale": torch.full((mr.moe_quantize_cols_width(M, len(counts)) // 128, K), 7.0, device="cuda")}
    mr.moe_quantize_cols(x, offsets, kept, perm=perm, k=k, out=out)
    parts, at = [], 0
    for c, n in zip(counts, kept_counts):
        rows = x[(perm[at:at + n].long() // k)]
        parts += [rows, rows.new_zeros(-n % 128, K)]
        at += c
    filled = torch.cat(parts)
    W = filled.shape[0]
    want = mr.moe_quantize_rows(filled.T.contiguous())
    assert torch.equal(out["q"][:, :W].view(torch.uint8), want["q"].view(torch.uint8))
    assert torch.equal(out["scale"][: W // 128], want["scale"])
    assert (out["q"][:, W:].view(torch.uint8) == 77).all() and (out["scale"][W // 128:] == 7).all()


def test_wgrad_of_many_tiles_is_exact_for_whole_numbers(mr):
    """More tiles than CTAs and more blocks than the pipeline holds, scales that differ from block to
    block: every sum is a multiple of 1/4 below 2^22, so fp32 holds it exactly in any order."""
    counts = [1000, 130, 0, 1664]
    offsets, kept, _ = split(counts, counts)
    M, N, K = sum(counts), 2064, 1808
    gen = torch.Generator().manual_seed(3)

    def whole(C):
        v = torch.randint(-4, 5, (M, C), generator=gen).double()
        return (v * 2.0 ** torch.randint(-1, 2, ((M + 99) // 100, C), generator=gen).repeat_interleave(100, 0)[:M]).cuda()

    dy, x = whole(N), whole(K)
    a, b = (mr.moe_quantize_cols(t.to(torch.bfloat16), offsets, kept) for t in (dy, x))
    got = mr.moe_expert_wgrad(a["q"], a["scale"], b["q"], b["scale"], kept)
    at = 0
    for e, n in enumerate(counts):
        assert torch.equal(got[e].double(), dy[at:at + n].T @ x[at:at + n]), e
        at += n


TINY = 2.0 ** -149                                               # fp32's smallest step: half of it is a rounding there


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("M,K,E,N", [(150, 640, 2, 304), (900, 400, 2, 288), (5, 128, 1, 16)])
def test_scales_whose_product_leaves_fp32(mr, M, K, E, N, dtype):
    """Row scales by which the product of two scales is past 2^128 or far below 2^-126, or a scale is 0,
    while the results are ordinary numbers; rows of codes 0 give 0, not 0 times infinity.  Rows of
    ordinary scales keep their bits beside them."""
    g = torch.Generator().manual_seed(M)
    blocks = -(-K // 128)
    wq = (torch.randn(E, N, K, generator=g) * 0.03).clamp(-2.0 ** -4, 2.0 ** -4).to(F8).cuda()
    wscale = ((1 + torch.rand(E, -(-N // 128), blocks, generator=g)) * 2.0 ** torch.tensor([20.0, -40.0, 20.0, -45.0, -38.0])[:blocks]).cuda()
    up, down, no = 2.0 ** 112, 1.3 * 2.0 ** -106, 1.0             # beside 2^20: 2^132; beside 2^-40: 2^-146
    kind = torch.arange(M) % 4
    codes = torch.randn(M, K, generator=g)
    q, scale = torch.zeros(M, K), torch.ones(blocks, M)
    for b in range(blocks):
        at = slice(128 * b, 128 * (b + 1))
        big = b in (0, 2)                                         # the blocks of large weight scales
        q[:, at] = torch.where(kind[:, None] == 0, (codes[:, at] * 2.0 ** -9).clamp(-2.0 ** -8, 2.0 ** -8) if big else torch.zeros(()),
                               torch.where(kind[:, None] == 1, (codes[:, at] * 200).clamp(-448, 448) if not big else torch.zeros(()),
                                           codes[:, at] * 60)).clamp(-448, 448)
        scale[b] = torch.where(kind == 0, up, torch.where(kind == 1, down, torch.where(kind == 2, no, 0.0))) * (1 + torch.rand(M, generator=g) / 8)
    q, scale = q.to(F8).cuda(), scale.cuda()
    q.view(torch.uint8)[8::16] = 0
    offsets, _, rows = split([M // E] * (E - 1) + [M - M // E * (E - 1)])
    got = mr.moe_expert_matmul(q, scale, wq, wscale, offsets, out_dtype=dtype)
    want, size = ref.matmul(wide(q), wide(scale), wide(wq), wide(wscale), rows)
    bound = (256 + 3 * blocks) * ref.U32 * size + blocks * TINY
    if dtype == torch.bfloat16:
        bound = bound * (1 + ref.U16) + ref.U16 * np.abs(want) + 2.0 ** -134
    assert np.abs(want).max() > 2.0 ** 110 and np.isfinite(wide(got)).all() and not wide(got)[3::4].any()
    ref.assert_near("out", wide(got), want, bound)
    alone = scale.clone()
    alone[:, kind.cuda() != 2] = 1
    assert torch.equal(mr.moe_expert_matmul(q, alone, wq, wscale, offsets, out_dtype=dtype)[2::4], got[2::4])


def test_wgrad_scales_whose_product_leaves_fp32(mr):
    """The same for both sides' scales of a weight gradient, which meet in every element."""
    g = torch.Generator().manual_seed(5)
    N, K, counts = 272, 304, [300, 0, 128, 17]
    rows = ref.expert_rows(np.concatenate([[0], np.cumsum(counts)]), None, sum(counts))
    width = mr.moe_quantize_cols_width(sum(counts), len(counts))
    dq, xq = ((torch.randn(n, width, generator=g) * 100).clamp(-448, 448).to(F8).cuda() for n in (N, K))
    ds, xs = ((1 + torch.rand(width // 128, n, generator=g)).cuda() for n in (N, K))
    ds[:, 1::8] *= 2.0 ** 110
    ds[:, 2::8] *= 2.0 ** -145                                    # small sums times these hold few digits in fp32
    ds[:, 3::8] *= 2.0 ** -120
    ds[:, 5::8] = 0
    xs[:, 0::4] *= 2.0 ** -100
    xs[:, 1::4] *= 2.0 ** 75
    xs[:, 2::4] *= 2.0 ** -60
    xs[:, 3::4] *= 2.0 ** -70
    dq[2::8] = (torch.randn(dq[2::8].shape, generator=g) * 2.0 ** -8).to(F8).cuda()
    dq.view(torch.uint8)[9] = 0
    got = mr.moe_expert_wgrad(dq, ds, xq, xs, i32(counts))
    want, size = ref.wgrad(wide(dq), wide(ds), wide(xq), wide(xs), rows)
    over = size > 2.0 ** 127                                      # 2^110 times 2^75: infinite, or 0
    assert (~np.isfinite(wide(got))[over]).all() and np.isfinite(wide(got))[~over].all()
    bound = (256 + 3 * 3) * ref.U32 * size + 3 * TINY
    ref.assert_near("dw", np.where(over, 0, wide(got)), np.where(over, 0, want), np.where(over, 0, bound))


def test_a_call_beside_the_status_is_reported_or_right(mr, native_lib):
    """An error is read while another call is queued behind the read: that call either is covered by
    what was read or does its work."""
    import threading
    import time

    q, scale, wq, wscale = operands(200, 1024, 1, 256, 4)
    want = mr.moe_expert_matmul(q, scale, wq, wscale)
    out = torch.full_like(want, 5.0)
    s = torch.cuda.Stream()
    torch.cuda.synchronize()
    native_lib.moe_set_wait_timeout_ns(1_000_000)
    native_lib.moe_set_unreachable_barriers(1)
    try:
        mr.moe_expert_matmul(q, scale, wq, wscale)
        torch.cuda.synchronize()
    finally:
        native_lib.moe_set_unreachable_barriers(0)
        native_lib.moe_set_wait_timeout_ns(0)
    with torch.cuda.stream(s):
        torch.cuda._sleep(200_000_000)                           # some 0.1 s, in which both are queued
    read = []
    reader = threading.Thread(target=lambda: read.append(mr.moe_expert_device_status(stream=s)))
    reader.start()
    time.sleep(0.02)
    mr.moe_expert_matmul(q, scale, wq, wscale, out=out, stream=s)
    reader.join()
    s.synchronize()
    assert read == [2] and torch.equal(out, want)
    assert mr.moe_expert_device_status() == 0


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("value", [float("nan"), -float("nan"), float("inf"), -float("inf")])
def test_not_finite_blocks_of_columns_and_weights(mr, value, dtype):
    """One value that is not finite makes its block's scale NaN, whichever lane, warp and half of a
    word meets it, and no other block's."""
    counts = [130, 0, 300]
    offsets, _, rows = split(counts)
    M, K = sum(counts), 272
    clean = values((M, K), 6, dtype)
    q, scale = ref.quantize_cols(wide(clean), rows)
    first = {0: 0, 130: 2}                                       # an expert's first row: its first block
    for r, c in ((0, 0), (1, 1), (129, 271), (130, 128), (257, 127), (258, 8), (429, 143), (300, 200)):
        x = clean.clone()
        x[r, c] = value
        got = mr.moe_quantize_cols(x.cuda(), offsets)
        at = 0 if r < 130 else 130
        b = first[at] + (r - at) // 128
        bad = np.zeros_like(scale, bool)
        bad[b, c] = True
        s = wide(got["scale"])[:len(scale)]
        assert np.array_equal(np.isnan(s), bad) and np.array_equal(s[~bad], scale[~bad])
        same = np.ones_like(q, bool)
        same[c, 128 * b:128 * (b + 1)] = False
        assert np.array_equal(wide(got["q"])[:, :q.shape[1]][same], q[same])
    clean = values((2, 144, 272), 7, dtype)
    q, scale = ref.quantize_weights(wide(clean))
    for e, n, c in ((0, 0, 0), (0, 127, 127), (1, 128, 3), (1, 143, 271), (0, 77, 130), (1, 16, 129)):
        w = clean.clone()
        w[e, n, c] = value
        got = mr.moe_quantize_weights(w.cuda(), transposed=True)
        bad = np.zeros_like(scale, bool)
        bad[e, n // 128, c // 128] = True
        s = wide(got["scale"])
        assert np.array_equal(np.isnan(s), bad) and np.array_equal(s[~bad], scale[~bad])
        assert np.array_equal(wide(got["scalet"]).transpose(0, 2, 1), s, equal_nan=True)
        same = ~ref.spread(bad, q.shape)
        assert np.array_equal(wide(got["q"])[same], q[same]) and np.array_equal(wide(got["qt"]).transpose(0, 2, 1)[same], q[same])


@pytest.mark.parametrize("form", ["rows", "weights", "cols"])
def test_every_product_with_a_block_that_is_not_finite_is_nan(mr, form):
    """The NaN scale reaches every result that the block is part of, and no other."""
    M, K, N = 200, 272, 144
    x, w = values((M, K), 8, torch.float32), values((1, N, K), 9, torch.float32)
    if form == "rows":
        x[17, 200] = float("inf")
    elif form == "weights":
        w[0, 130, 5] = float("nan")
    else:
        x[150, 33] = -float("inf")
    a, b = mr.moe_quantize_rows(x.cuda()), mr.moe_quantize_weights(w.cuda())
    bad = np.zeros((M, N), bool)
    if form == "cols":
        offsets, kept, _ = split([M], [M])
        dy = values((M, N), 10, torch.float32)
        d, c = mr.moe_quantize_cols(dy.cuda(), offsets, kept), mr.moe_quantize_cols(x.cuda(), offsets, kept)
        got = mr.moe_expert_wgrad(d["q"], d["scale"], c["q"], c["scale"], kept)[0]
        bad = np.zeros((N, K), bool)
        bad[:, 33] = True
    else:
        got = mr.moe_expert_matmul(a["q"], a["scale"], b["q"], b["scale"], out_dtype=torch.float32)
        if form == "rows":
            bad[17] = True
        else:
            bad[:, 128:] = True
    assert np.array_equal(np.isnan(wide(got)), bad)


@pytest.mark.parametrize("case", [
    {"op": "route", "T": 300, "E": 96, "k": 4, "dtype": "bf16", "score": "sigmoid", "bias": True, "groups": 4, "keep": 2, "group_score": "top2",
     "renorm": True, "scale": 2.5, "bwd": True},
    {"op": "route", "T": 77, "E": 33, "k": 3, "dtype": "fp32", "score": "softmax", "bias": False, "groups": 3, "keep": 2, "group_score": "max",
     "renorm": False, "scale": 1.0, "bwd": True},
    {"op": "quantize", "form": "rows", "T": 50, "k": 2, "E": 8, "K": 272, "dtype": "bf16", "gather": True, "cf": 1.25},
    {"op": "quantize", "form": "cols", "T": 150, "k": 2, "E": 4, "K": 144, "dtype": "fp32", "gather": False, "cf": 1.0},
    {"op": "quantize", "form": "weights", "T": 1, "k": 1, "E": 2, "K": 272, "N": 144, "dtype": "bf16", "gather": False, "cf": 1.0},
    {"op": "matmul", "T": 90, "k": 2, "E": 4, "K": 400, "N": 144, "out": "bf16", "cf": 1.0},
    {"op": "wgrad", "T": 130, "k": 2, "E": 4, "K": 144, "N": 272, "cf": 1.25},
    {"op": "combine", "T": 40, "k": 4, "E": 8, "H": 264, "dtype": "bf16", "cf": 1.0, "bwd": True},
], ids=lambda c: "-".join(str(c[k]) for k in ("op", "form") if k in c))
def test_measured_calls_against_their_plain_and_exact_forms(mr, monkeypatch, case):
    """What perf/operators.py times: the calls, their plain torch forms and the definitions in 64 bits
    agree.  Whole numbers, codes and scales are equal; a number is off by half a step of its type
    and the sums' rounding, 1e-5 of the output's largest covers hundreds of 2^-24."""
    import importlib.util
    from pathlib import Path
    spec = importlib.util.spec_from_file_location("operators", Path(__file__).resolve().parents[1] / "perf" / "operators.py")
    ops = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(ops)

    def flat(o):
        return dict(o) if isinstance(o, dict) else {"out": o}

    plain = {n: v.clone() for n, v in flat(ops.run(ops.prepare(case, 3))).items()}
    monkeypatch.setattr(ops, "own", True)
    got = flat(ops.run(ops.prepare(case, 3)))
    want = flat(ops.exact(case, 3))
    assert set(plain) == set(got) == set(want)
    for name, w in want.items():
        w = torch.as_tensor(w).double().cpu()
        for side in (plain[name], got[name]):
            v = side.double().cpu()
            if not side.is_floating_point() or case["op"] == "quantize":
                assert torch.equal(v, w), name
            else:
                step = 2.0 ** -8 if side.dtype == torch.bfloat16 else 0.0
                assert ((v - w).abs() <= step * w.abs() + 1e-5 * w.abs().max()).all(), name


@pytest.mark.parametrize("share", [0.02, 0.4, 0.6, 1.0])
@pytest.mark.parametrize("M,K,N", [(75, 208, 48), (517, 1040, 272), (333, 16, 16)])
def test_few_and_many_rows_of_extreme_scales(mr, M, K, N, share):
    """One row of a tile, more than half of its rows and all of them: those have scales whose product
    fp32 holds no digits of, the others keep the bits that they have alone."""
    g = torch.Generator().manual_seed(M)
    blocks = -(-K // 128)
    for dtype in (torch.bfloat16, torch.float32):
        q, scale, wq, wscale = operands(M, K, 1, N, M)
        wscale *= 2.0 ** -40
        base = mr.moe_expert_matmul(q, scale, wq, wscale, out_dtype=dtype)
        far = torch.rand(M, generator=g) < share
        far[M // 2] = True
        at = far.nonzero()[:, 0].cuda()
        scale[:, at] *= 2.0 ** -95
        scale[0, at[::2]] = 0
        got = mr.moe_expert_matmul(q, scale, wq, wscale, out_dtype=dtype)
        want, size = ref.matmul(wide(q), wide(scale), wide(wq), wide(wscale), [(0, M)])
        u = ref.U16 if dtype == torch.bfloat16 else 0.0
        tiny = blocks * TINY * 2 + (2.0 ** -134 if u else 0.0)
        ref.assert_near("out", wide(got), want, (256 + 3 * blocks) * ref.U32 * size * (1 + u) + u * np.abs(want) + tiny)
        assert torch.equal(got[~far.cuda()], base[~far.cuda()])
        few = M - 20                                              # rows behind the kept ones stay
        out = torch.full_like(got, 7.0)
        mr.moe_expert_matmul(q, scale, wq, wscale, i32([0, M]), i32([few]), out=out)
        assert torch.equal(out[:few], got[:few]) and (out[few:] == 7).all()


@pytest.mark.parametrize("share", [0.02, 0.6, 1.0])
def test_few_and_many_rows_of_extreme_scales_of_a_weight_gradient(mr, share):
    g = torch.Generator().manual_seed(7)
    N, K, counts = 304, 336, [150, 1, 0, 400]
    rows = ref.expert_rows(np.concatenate([[0], np.cumsum(counts)]), None, sum(counts))
    width = mr.moe_quantize_cols_width(sum(counts), len(counts))
    dq, xq = ((torch.randn(n, width, generator=g) * 3).to(F8).cuda() for n in (N, K))
    ds, xs = (torch.exp(torch.randn(width // 128, n, generator=g)).cuda() for n in (N, K))
    base = mr.moe_expert_wgrad(dq, ds, xq, xs, i32(counts))
    far = torch.rand(N, generator=g) < share
    far[100] = True
    at = far.nonzero()[:, 0].cuda()
    ds[:, at] *= 2.0 ** -143                                      # a few bits of the scale and fewer of a product
    xs2 = xs * 2.0 ** 90
    got = mr.moe_expert_wgrad(dq, ds, xq, xs2, i32(counts))
    want, size = ref.wgrad(wide(dq), wide(ds), wide(xq), wide(xs2), rows)
    ref.assert_near("dw", wide(got), want, (256 + 3 * 4) * ref.U32 * size + 8 * TINY)
    assert torch.equal(mr.moe_expert_wgrad(dq, ds, xq, xs, i32(counts))[:, ~far.cuda()], base[:, ~far.cuda()])
