"""GPU parity of the experts' 4-bit products against float64.

Bound, against the sum S of the sizes of an element's terms: the tensor core adds 64 products at a
time to the sum in fp32; each of those 65 addends may lose what lies 2^-25 below the largest, and
the sum is cut to fp32 (2^-23): (65 * 2^-25 + 2^-23) * S for every 64 of K, which is less than
2^-24 * K * 0.54 + 2^-23 * K / 64 < K * 2^-24 * S.  A bf16 result adds half a step, 2^-8 of the value.
Where every sum is a whole number below 2^24 times one power of two the result has to be exact.
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


def i32(a):
    return torch.as_tensor(np.asarray(a), dtype=torch.int32).cuda()


def split(counts, kept=None):
    offsets = np.concatenate([[0], np.cumsum(counts)])
    return i32(offsets), None if kept is None else i32(kept), experts_ref.expert_rows(offsets, kept, int(offsets[-1]))


def codes(rows, K, seed, spread=6, middle=127):
    """Random codes and exponents of rows: ([rows, K/2], [ceil(K/128), rows, 4]); the bytes behind K are 255."""
    rng = np.random.default_rng(seed)
    q = rng.integers(0, 256, (rows, K // 2), dtype=np.uint8)
    n = rng.integers(middle - spread, middle + spread + 1, (rows, K // 32))
    s = ref.fold(n)
    b = np.moveaxis(s, 0, 1).reshape(rows, -1)
    b[:, K // 32:] = 255
    return q, np.ascontiguousarray(b.reshape(rows, -1, 4).transpose(1, 0, 2))


def operands(M, K, E, N, seed, **kw):
    q, s = codes(M, K, seed, **kw)
    wq, ws = codes(E * N, K, seed + 1000, **kw)
    return (torch.from_numpy(q).cuda(), torch.from_numpy(s).cuda(), torch.from_numpy(wq).view(E, N, K // 2).cuda(),
            torch.from_numpy(ws).view(-1, E, N, 4).cuda())


def expected(q, scale, wq, wscale, rows):
    return ref.products(ref.read(q.cpu().numpy(), scale.cpu().numpy()), ref.read(wq.cpu().numpy(), wscale.cpu().numpy()), rows)


def check(got, want, size, K, before=None):
    """Rows of no expert hold what they held before."""
    live = ~np.isnan(want)
    bound = K * ref.U32 * size
    if got.dtype is torch.bfloat16:
        bound = bound * (1 + ref.U16) + np.abs(np.where(live, want, 0.0)) * ref.U16
    g = wide(got)
    experts_ref.assert_near("out", g[live], want[live], bound[live])
    if before is not None:
        assert np.array_equal(g[~live], wide(before)[~live])


SHAPES = [([1], None, 32, 16), ([128], None, 64, 128), ([129], None, 96, 272), ([5, 0, 300, 129], None, 160, 144), ([260, 70, 600], [200, 70, 513], 544, 304),
          ([40] * 20, None, 320, 64), ([1, 2, 3, 0, 700], [1, 1, 3, 0, 650], 1440, 1040), ([31, 33], [0, 33], 4096, 48), ([1100], None, 256, 528)]


# Enough tiles for the wide ones, and for several rounds of the narrow ones; ragged rows, columns and ends of the contraction.
MANY = [([700, 300, 900, 513], None, 96, 1552), ([2413], None, 544, 1552), ([900, 0, 1501, 70, 2600], [900, 0, 1300, 70, 2555], 288, 2064),
        ([75] * 16, [75, 3] * 8, 320, 2064), ([5000, 1, 129], None, 1184, 272), ([1024] * 3, None, 768, 2048),
        ([1, 0, 2, 0] * 256, [1, 0, 1, 0] * 256, 64, 32), ([0] * 1023 + [140], None, 96, 144)]


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("counts,kept,K,N", SHAPES + MANY)
def test_products(mr, counts, kept, K, N, dtype):
    M, E = sum(counts), len(counts)
    ops = operands(M, K, E, N, M + K)
    offsets, kt, rows = split(counts, kept)
    before = torch.full((M, N), 7.0, dtype=dtype, device="cuda")
    got = mr.moe_expert_matmul_fp4(*ops, offsets, kt, out=before.clone())
    check(got, *expected(*ops, rows), K, before)


def test_scales_at_any_word(mr):
    """The rows' scales begin anywhere in 4 bytes; the weights' in 16, or the call is refused."""
    counts, K, N = [3, 150, 61], 160, 144
    offsets, _, rows = split(counts)
    q, s, wq, ws = operands(sum(counts), K, len(counts), N, 9)
    want = mr.moe_expert_matmul_fp4(q, s, wq, ws, offsets)
    for words in (1, 2, 3):
        moved = [torch.cat([t.flatten().new_zeros(4 * words), t.flatten()])[4 * words:].view(t.shape) for t in (s, ws)]
        assert torch.equal(mr.moe_expert_matmul_fp4(q, moved[0], wq, ws, offsets), want)
        with pytest.raises(mr._native.MoeRouterError, match="aligned"):
            mr.moe_expert_matmul_fp4(q, s, wq, moved[1], offsets)


@pytest.mark.parametrize("K", [32, 64, 96, 128, 160, 224, 256, 288, 352, 480, 512, 544])
def test_every_end_of_a_stage(mr, K):
    """Lengths that end at each block of a stage of 256, with whole-number sums: exact."""
    M, N = 150, 272
    ops = operands(M, K, 1, N, K, spread=2)
    got = mr.moe_expert_matmul_fp4(*ops, out_dtype=torch.float32)
    want, size = expected(*ops, [(0, M)])
    assert size.max() < 2.0 ** 24 * 2.0 ** -6                     # terms are multiples of 2^-6
    assert np.array_equal(wide(got), want)


def test_a_scale_reaches_its_block_alone(mr):
    """Ones times one block's scale at a time: which block, of which row and column, each result shows."""
    K, M, N = 512, 200, 288
    one = np.full((max(M, N), K // 2), 0x22, dtype=np.uint8)      # codes of 1
    n = np.full((M, K // 32), 127)
    n[np.arange(M), np.arange(M) % 16] = 127 + 1 + np.arange(M) // 16 % 8
    m = np.full((N, K // 32), 127)
    m[np.arange(N), (np.arange(N) * 5 + 3) % 16] = 127 - 1 - np.arange(N) // 16 % 5
    ops = [torch.from_numpy(a).cuda() for a in (one[:M], ref.fold(n), one[None, :N], ref.fold(m)[:, None])]
    got = mr.moe_expert_matmul_fp4(*ops, out_dtype=torch.float32)
    want = 32.0 * (2.0 ** (n - 127.0)) @ (2.0 ** (m - 127.0)).T
    assert np.array_equal(wide(got), want)


def test_without_offsets_is_one_expert(mr):
    ops = operands(77, 288, 1, 80, 3)
    got = mr.moe_expert_matmul_fp4(*ops)
    assert got.dtype is torch.bfloat16 and torch.equal(got, mr.moe_expert_matmul_fp4(*ops, i32([0, 77])))


@pytest.mark.parametrize("a,w", [(20, 234), (234, 20), (1, 253), (253, 1), (100, 127), (60, 80), (200, 150)])
def test_scales_far_apart(mr, a, w):
    """Exponents whose product is an ordinary number, though neither is."""
    M, K, N = 40, 256, 32
    q, s, wq, ws = operands(M, K, 1, N, a, spread=0)
    s.fill_(a)
    ws.fill_(w)
    got = mr.moe_expert_matmul_fp4(q, s, wq, ws, out_dtype=torch.float32)
    want, size = expected(q, s, wq, ws, [(0, M)])
    check(got, want, size, K)


def test_scales_past_fp32(mr):
    """Sums above the largest number are infinite, or a NaN where such terms of both signs meet; those below the smallest are 0 to within it."""
    M, K, N = 8, 64, 16
    one = lambda r: torch.full((r, K // 2), 0x22, dtype=torch.uint8, device="cuda")  # noqa: E731
    s = torch.full((1, M, 4), 1, dtype=torch.uint8, device="cuda")
    w = torch.full((1, 1, N, 4), 1, dtype=torch.uint8, device="cuda")
    got = mr.moe_expert_matmul_fp4(one(M), s, one(N)[None], w, out_dtype=torch.float32)
    assert bool((got.abs() <= 2.0 ** -126).all())
    got = mr.moe_expert_matmul_fp4(one(M), s.fill_(254), one(N)[None], w.fill_(254), out_dtype=torch.float32)
    assert bool(torch.isinf(got).all())


def test_not_a_number_scales(mr):
    """A row's and a column's own; no other result changes."""
    M, K, N, E = 300, 288, 144, 2
    q, s, wq, ws = operands(M, K, E, N, 11)
    offsets, _, rows = split([170, 130])
    base = mr.moe_expert_matmul_fp4(q, s, wq, ws, offsets, out_dtype=torch.float32)
    s2, ws2 = s.clone(), ws.clone()
    s2[1, 7, 2], s2[2, 299, 0], ws2[0, 1, 20, 3] = 255, 255, 255
    got = mr.moe_expert_matmul_fp4(q, s2, wq, ws2, offsets, out_dtype=torch.float32)
    bad = torch.zeros(M, N, dtype=torch.bool, device="cuda")
    bad[7] = bad[299] = True
    bad[170:, 20] = True
    assert bool(got[bad].isnan().all()) and torch.equal(got[~bad], base[~bad])


def test_rows_do_not_depend_on_one_another(mr):
    """A row alone and among others: the same bits."""
    K, N, E = 512, 384, 2
    q, s, wq, ws = operands(600, K, E, N, 9)
    offsets, kept, _ = split([300, 300], [250, 300])
    base = mr.moe_expert_matmul_fp4(q, s, wq, ws, offsets, kept, out_dtype=torch.float32)
    for r in (0, 249, 300, 599):
        one = mr.moe_expert_matmul_fp4(q[r:r + 1].contiguous(), s[:, r:r + 1].contiguous(), wq, ws, i32([0, 1, 1] if r < 300 else [0, 0, 1]), out_dtype=torch.float32)
        assert torch.equal(one[0], base[r])


def test_rows_alike_in_tiles_of_either_width(mr):
    """Rows of a call with many, and alone in a small one: the same bits, of sums that are rounded at every step."""
    M, K, N = 2413, 1184, 1552
    q, s, wq, ws = operands(M, K, 1, N, 4, spread=12)
    many = mr.moe_expert_matmul_fp4(q, s, wq, ws, out_dtype=torch.float32)
    for at in (slice(0, 40), slice(1201, 1330), slice(2412, 2413)):
        assert torch.equal(mr.moe_expert_matmul_fp4(q[at].contiguous(), s[:, at].contiguous(), wq, ws, out_dtype=torch.float32), many[at])


def test_positions_outside_the_arrays_stay_inside(mr):
    ops = operands(64, 128, 3, 64, 2)
    for offsets, kept in (([0, 900, 64, 64], [9, 9, 9]), ([-5, 30, 20, 1 << 30], None), ([64, 64, 64, 64], None), ([0, 10, 20, 30], [-3, 1 << 30, 5])):
        mr.moe_expert_matmul_fp4(*ops, i32(offsets), None if kept is None else i32(kept))
    torch.cuda.synchronize()


def test_results_past_32_bit_offsets(mr):
    """Operand and result positions past 2^31; rows at both ends are compared with a small call's."""
    M, K, N = 2 ** 31 // 4096 + 300, 8192, 4112
    part, ps, wq, ws = operands(300, K, 1, N, 1)
    q = torch.zeros(M, K // 2, dtype=torch.uint8, device="cuda")
    s = torch.full((K // 128, M, 4), 127, dtype=torch.uint8, device="cuda")
    for at in (slice(0, 300), slice(M - 300, M)):
        q[at], s[:, at] = part, ps
    got = mr.moe_expert_matmul_fp4(q, s, wq, ws)
    want = mr.moe_expert_matmul_fp4(part, ps, wq, ws)
    assert torch.equal(got[:300], want) and torch.equal(got[-300:], want) and not bool(got[300:-300].any())


def test_from_quantised_values(mr):
    """What moe_quantize_fp4 gives, through the product: the product of the values that it stands for."""
    g = torch.Generator().manual_seed(0)
    x, w = torch.randn(90, 416, generator=g).cuda(), torch.randn(2, 48, 416, generator=g).cuda()
    a, b = mr.moe_quantize_fp4(x), mr.moe_quantize_fp4(w)
    offsets, _, rows = split([50, 40])
    got = mr.moe_expert_matmul_fp4(a["q"], a["scale"], b["q"], b["scale"], offsets, out_dtype=torch.float32)
    xv, wv = (wide(mr.moe_dequantize_fp4(t["q"], t["scale"])) for t in (a, b))
    check(got, *ref.products(xv, wv, rows), 416)


def test_captured_and_concurrent_calls(mr):
    """Two graphs on two streams at once, and eager calls beside them: no state is shared."""
    sets, streams, graphs = [], [torch.cuda.Stream() for _ in range(2)], []
    offsets, kept, _ = split([100, 0, 150, 50], [90, 0, 150, 50])
    for i in range(2):
        ops = operands(300, 512, 4, 256, 20 + i)
        out = torch.zeros(300, 256, dtype=torch.bfloat16, device="cuda")
        sets.append((ops, out, mr.moe_expert_matmul_fp4(*ops, offsets, kept, out=torch.zeros_like(out))))
    torch.cuda.synchronize()
    for s, (ops, out, _) in zip(streams, sets):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, stream=s):
            for _ in range(3):
                mr.moe_expert_matmul_fp4(*ops, offsets, kept, out=out, stream=s)
        graphs.append(g)
    for _ in range(5):
        for s, g in zip(streams, graphs):
            with torch.cuda.stream(s):
                g.replay()
        mr.moe_expert_matmul_fp4(*sets[0][0], offsets, kept, out=torch.zeros_like(sets[0][1]))
    torch.cuda.synchronize()
    for _, out, want in sets:
        assert torch.equal(out, want)


def test_an_expired_wait_is_reported(mr, native_lib):
    """A pipeline wait made to run out (1 ms, an arrival that never comes): the status tells, later calls write nothing
    until it is read, then calls work again."""
    ops = operands(200, 1024, 1, 256, 4)
    want = mr.moe_expert_matmul_fp4(*ops)
    torch.cuda.synchronize()
    native_lib.moe_set_wait_timeout_ns(1_000_000)
    native_lib.moe_set_unreachable_barriers(1)
    try:
        mr.moe_expert_matmul_fp4(*ops)
        torch.cuda.synchronize()
    finally:
        native_lib.moe_set_unreachable_barriers(0)
        native_lib.moe_set_wait_timeout_ns(0)
    out = torch.full((200, 256), 3.0, dtype=torch.bfloat16, device="cuda")
    mr.moe_expert_matmul_fp4(*ops, out=out)
    torch.cuda.synchronize()
    assert bool((out == 3.0).all())
    assert mr.moe_expert_device_status() & 2
    assert mr.moe_expert_device_status() == 0
    assert torch.equal(mr.moe_expert_matmul_fp4(*ops), want)


def test_refusals(mr):
    q, s, wq, ws = operands(8, 64, 2, 32, 1)
    o = i32([0, 4, 8])
    for call in (lambda: mr.moe_expert_matmul_fp4(q, s, wq[:, :, :16].contiguous(), ws, o), lambda: mr.moe_expert_matmul_fp4(q, s[:, :4].contiguous(), wq, ws, o),
                 lambda: mr.moe_expert_matmul_fp4(q, s, wq, ws[:, :1].contiguous(), o), lambda: mr.moe_expert_matmul_fp4(q, s, wq, ws, o[:2]),
                 lambda: mr.moe_expert_matmul_fp4(q, s, wq, ws, o, kept=o), lambda: mr.moe_expert_matmul_fp4(q, s, wq, ws, o, out_dtype=torch.float16),
                 lambda: mr.moe_expert_matmul_fp4(q.int(), s, wq, ws, o), lambda: mr.moe_expert_matmul_fp4(q, s, wq, ws, o, out=torch.zeros(8, 16, device="cuda"))):
        with pytest.raises(ValueError):
            call()
    with pytest.raises(mr._native.MoeRouterError):
        mr.moe_expert_matmul_fp4(q, s, wq, ws)                    # two experts without offsets
    with pytest.raises(mr._native.MoeRouterError):
        mr.moe_expert_matmul_fp4(q, s, wq[:, :24].contiguous(), ws[:, :, :24].contiguous(), o)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("offsets,kept", [([0, 900, 64, 64], [9, 9, 9]), ([-5, 30, 20, 1 << 30], None), ([64, 64, 64, 64], None), ([0, 10, 20, 30], [-3, 1 << 30, 5]),
                                          ([40, 64, 1 << 30, 1 << 30], [1 << 30, 7, 7]), ([-100, -5, 3, 50], None)])
def test_positions_outside_the_arrays_write_nothing_beside_them(mr, offsets, kept, dtype):
    """In front of the result and behind it, and in rows of no expert, what was there stays; the other rows are right."""
    M, K, N, E, margin = 64, 128, 64, 3, 300
    ops = operands(M, K, E, N, 2)
    inside = np.clip(offsets, 0, M)
    ends = np.maximum(inside[1:], inside[:-1])
    number = ends - inside[:-1] if kept is None else np.minimum(ends - inside[:-1], np.maximum(kept, 0))
    rows = [(int(a), int(n)) for a, n in zip(inside[:-1], number)]
    owners = np.zeros(M, dtype=int)
    for at, n in rows:
        owners[at:at + n] += 1
    whole = torch.full((M + 2 * margin, N), 7.0, dtype=dtype, device="cuda")
    before = whole[margin:margin + M].clone()
    got = mr.moe_expert_matmul_fp4(*ops, i32(offsets), None if kept is None else i32(kept), out=whole[margin:margin + M])
    torch.cuda.synchronize()
    assert bool((whole[:margin] == 7.0).all()) and bool((whole[margin + M:] == 7.0).all())
    once = owners < 2                                            # a row of two experts has the result of either
    want, size = expected(*ops, rows)
    check(got[torch.from_numpy(once).cuda()], want[once], size[once], K, before[torch.from_numpy(once).cuda()])
