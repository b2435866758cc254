"""GPU parity of the 4-bit quantisation and its values against float64: codes, scales and values are compared exactly."""

import numpy as np
import pytest
import torch

import layer_reference as ref

pytestmark = pytest.mark.gpu
DTYPES = [torch.bfloat16, torch.float32]


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
    return t.double().cpu().numpy()


def i32(a):
    return torch.as_tensor(np.asarray(a), dtype=torch.int32).cuda()


def check(got, x):
    code, n = ref.quantize_fp4(wide(x))
    assert np.array_equal(got["scale"].cpu().numpy(), ref.fold(n))
    assert np.array_equal(ref.unpack(got["q"].cpu().numpy()), code)


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("M,K", [(1, 32), (1, 128), (33, 160), (100, 512), (7, 1056), (65, 2080)])
def test_rows(mr, M, K, dtype):
    x = values((M, K), M + K, dtype)
    x[0, :32] = 0                                                # a block of zeros
    x[-1, -3:] = -0.0
    got = mr.moe_quantize_fp4(x.cuda())
    check(got, x)
    for to in DTYPES:
        back = mr.moe_dequantize_fp4(got["q"], got["scale"], dtype=to)
        assert back.dtype is to and np.array_equal(wide(back), ref.read(got["q"].cpu().numpy(), got["scale"].cpu().numpy()))


def test_rows_gathered(mr):
    T, k, K = 70, 3, 288
    perm = np.random.default_rng(0).permutation(T * k)
    x = values((T, K), 1)
    check(mr.moe_quantize_fp4(x.cuda(), perm=i32(perm), k=k), x[torch.from_numpy(perm // k)])
    bad = perm.copy()
    bad[5], bad[6] = -1, T * k                                   # outside x: zeros
    got = mr.moe_quantize_fp4(x.cuda(), perm=i32(bad), k=k)
    assert not got["q"][5:7].any() and (got["scale"][:, 5:7] == 127).all()
    few = i32([3, 3, 0])                                         # fewer rows than x has, the same one twice
    check(mr.moe_quantize_fp4(x.cuda(), perm=few, k=k), x[[1, 1, 0]])


def test_weights(mr):
    w = values((3, 48, 416), 2, torch.float32)
    got = mr.moe_quantize_fp4(w.cuda())
    assert got["q"].shape == (3, 48, 208) and got["scale"].shape == (4, 3, 48, 4)
    check({"q": got["q"].view(144, 208), "scale": got["scale"].view(4, 144, 4)}, w.view(144, 416))
    back = mr.moe_dequantize_fp4(got["q"], got["scale"])
    assert back.shape == w.shape and np.array_equal(wide(back), ref.read(got["q"].cpu().numpy(), got["scale"].cpu().numpy()))


@pytest.mark.parametrize("dtype", DTYPES)
def test_every_rounding_and_scale(mr, dtype):
    """Halves between codes, values next to them, blocks whose largest value is at each end of its scale's range."""
    top = torch.tensor([6.0, 5.96875, 6.03125, 3.0, 3.015625, 2.0 ** -133, 2.0 ** -126, 6 * 2.0 ** -126, 6.03125 * 2.0 ** -126, 3.0e38, 1.0, 4.0])
    near = torch.cat([torch.tensor([0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0]) * f for f in (1.0, 1.0 + 2.0 ** -7, 1.0 - 2.0 ** -8)] + [torch.tensor([0.0, 0.5, 1.5, 2.0, 3.0, 4.0, 6.0, 1.0, -0.0, 0.1])])
    x = torch.zeros(2 * len(top), 64)
    for i, t in enumerate(top):
        for sign in (0, 1):
            row = x[2 * i + sign]
            row[:31] = near * (t / 6)
            row[31] = t
            row[32:] = row[:32] * 2.0 ** -3
            if sign:
                row.neg_()
    x = x.to(dtype)
    check(mr.moe_quantize_fp4(x.cuda()), x)


@pytest.mark.parametrize("dtype", DTYPES)
def test_not_finite(mr, dtype):
    """Their block alone has the scale NaN, and its values read back as NaN."""
    x = values((4, 160), 5, dtype)
    x[0, 3], x[1, 40], x[2, 159] = float("inf"), float("nan"), float("-inf")
    got = mr.moe_quantize_fp4(x.cuda())
    n = ref.unfold(got["scale"].cpu().numpy(), 160)
    want = np.zeros((4, 5), dtype=bool)
    want[0, 0] = want[1, 1] = want[2, 4] = True
    assert np.array_equal(n == 255, want)
    clean = x.clone()
    clean[0, :32], clean[1, 32:64], clean[2, 128:] = 0, 0, 0
    code, m = ref.quantize_fp4(wide(clean))
    keep = np.repeat(~want, 32, axis=1)
    assert np.array_equal(n[~want], m[~want]) and np.array_equal(ref.unpack(got["q"].cpu().numpy())[keep], code[keep])
    back = wide(mr.moe_dequantize_fp4(got["q"], got["scale"]))
    assert np.array_equal(np.isnan(back), ~keep)


@pytest.mark.parametrize("dtype", DTYPES)
def test_values_of_any_scale(mr, dtype):
    """Every exponent byte times every code, with their overflow to infinity."""
    code = np.tile(np.arange(32, dtype=np.uint8) % 16, (256, 1))
    scale = np.zeros((1, 256, 4), dtype=np.uint8)
    scale[0, :, 0] = np.arange(256)
    y = mr.moe_dequantize_fp4(torch.from_numpy(ref.pack(code)).cuda(), torch.from_numpy(scale).cuda(), dtype=dtype)
    want = ref.read(ref.pack(code), scale)
    want = torch.from_numpy(want).to(dtype).double().numpy()     # only sizes from 2^128 on change
    assert np.array_equal(wide(y), want, equal_nan=True)


def test_rows_past_32_bits(mr):
    """More than 2^31 values (and 2^32 bytes): the last rows are theirs."""
    M, K = 70_000, 32_768
    x = torch.zeros(M, K, dtype=torch.bfloat16, device="cuda")
    tail = values((3, K), 9)
    x[-3:] = tail.cuda()
    got = mr.moe_quantize_fp4(x)
    check({"q": got["q"][-3:], "scale": got["scale"][:, -3:]}, tail)
    back = mr.moe_dequantize_fp4(got["q"], got["scale"])
    assert not bool(back[:-3].any())
    assert np.array_equal(wide(back[-3:]), ref.read(got["q"][-3:].cpu().numpy(), got["scale"][:, -3:].cpu().numpy()))


def test_refusals(mr):
    x = torch.zeros(4, 64, device="cuda")
    for bad in (torch.zeros(4, 48, device="cuda"), torch.zeros(4, 2, 2, 32, device="cuda"), x.half(), x[:, ::2], torch.zeros(0, 64, device="cuda")):
        with pytest.raises((ValueError, mr._native.MoeRouterError)):
            mr.moe_quantize_fp4(bad)
    with pytest.raises(ValueError):
        mr.moe_quantize_fp4(torch.zeros(2, 2, 64, device="cuda"), perm=i32([0]))
    with pytest.raises(ValueError):
        mr.moe_quantize_fp4(x, out={"q": torch.zeros(4, 64, dtype=torch.uint8, device="cuda")})
    q = mr.moe_quantize_fp4(x)
    with pytest.raises(ValueError):
        mr.moe_dequantize_fp4(q["q"], q["scale"], dtype=torch.float16)
    with pytest.raises(ValueError):
        mr.moe_dequantize_fp4(q["q"], q["scale"][:, :2])
