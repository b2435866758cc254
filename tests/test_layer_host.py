"""The 4-bit path, the gated activation and the layer for few tokens on the host: refusals before anything is queued, and
the float64 forms that the GPU tests compare with against independent ones."""

import numpy as np
import pytest
import torch

import layer_reference as ref
import moe_expert_routing_router_gb300 as mr
from moe_expert_routing_router_gb300 import layer

FAKE, BIG = 0x10000, 1 << 31                                     # FAKE is never dereferenced

GOOD = {
    "moe_quantize_fp4": [FAKE, 1, 16, 64, 128, FAKE, 4, FAKE, FAKE, None],
    "moe_dequantize_fp4": [FAKE, FAKE, 64, 128, 1, FAKE, None],
    "moe_expert_matmul_fp4": [FAKE, FAKE, 64, 128, FAKE, FAKE, 8, 64, FAKE, FAKE, 1, FAKE, None],
    "moe_expert_glu": [FAKE, 1, 64, 128, 2, FAKE, FAKE, None],
    "moe_expert_glu_bwd": [FAKE, FAKE, 1, 64, 128, FAKE, None],
    "moe_layer_small": [FAKE, 4, 128, 64, 8, 2, FAKE, FAKE, 1, FAKE, FAKE, 0, FAKE, FAKE, FAKE, FAKE, 1 << 20, None],
}
BAD = [("moe_quantize_fp4", p, v, w) for p, v, w in [
    (0, None, 1), (0, FAKE + 8, 1), (1, 3, 2), (2, 0, 1), (2, BIG, 1), (3, 0, 1), (3, BIG, 1), (4, 0, 1), (4, 16, 1), (4, 144, 1), (4, 1 << 21, 1),
    (5, None, 1), (5, FAKE + 2, 1), (6, 0, 1), (6, 9, 1), (7, None, 1), (7, FAKE + 8, 1), (8, None, 1), (8, FAKE + 2, 1)]]
BAD += [("moe_dequantize_fp4", p, v, w) for p, v, w in [
    (0, None, 1), (0, FAKE + 8, 1), (1, None, 1), (1, FAKE + 1, 1), (2, 0, 1), (2, BIG, 1), (3, 48, 1), (3, 0, 1), (4, 2, 2), (5, None, 1), (5, FAKE + 4, 1)]]
BAD += [("moe_expert_matmul_fp4", p, v, w) for p, v, w in [
    (0, None, 1), (0, FAKE + 8, 1), (1, None, 1), (1, FAKE + 2, 1), (2, 0, 1), (2, BIG, 1), (3, 0, 1), (3, 16, 1), (3, 112, 1), (3, 1 << 21, 1), (4, None, 1),
    (4, FAKE + 4, 1), (5, None, 1), (5, FAKE + 1, 1), (5, FAKE + 8, 1), (6, 0, 1), (6, 1025, 1), (7, 40, 1), (7, 0, 1), (8, None, 1), (8, FAKE + 2, 1), (9, FAKE + 2, 1),
    (10, 2, 2), (11, None, 1), (11, FAKE + 8, 1)]]
BAD += [("moe_expert_glu", p, v, w) for p, v, w in [
    (0, None, 1), (0, FAKE + 8, 1), (1, 2, 2), (2, 0, 1), (2, BIG, 1), (3, 0, 1), (3, 16, 1), (3, 1 << 21, 1), (4, 3, 1), (4, -1, 1), (4, 0, 1), (5, None, 1),
    (5, FAKE + 8, 1), (6, None, 1), (6, FAKE + 2, 1)]]
BAD += [("moe_expert_glu_bwd", p, v, w) for p, v, w in [
    (0, None, 1), (0, FAKE + 8, 1), (1, None, 1), (1, FAKE + 4, 1), (2, 2, 2), (3, 0, 1), (4, 8, 1), (4, 24, 1), (5, None, 1), (5, FAKE + 8, 1)]]

BAD += [("moe_layer_small", p, v, w) for p, v, w in [
    (0, None, 1), (0, FAKE + 8, 1), (1, 0, 1), (1, 65, 1), (1, BIG, 1), (2, 0, 1), (2, 112, 1), (2, 16416, 1), (3, 0, 1), (3, 24, 1), (3, 16400, 1), (4, 0, 1),
    (4, 1025, 1), (5, 0, 1), (5, 9, 1), (6, None, 1), (6, FAKE + 2, 1), (7, None, 1), (7, FAKE + 1, 1), (8, 2, 1), (8, -1, 1), (9, None, 1), (9, FAKE + 8, 1),
    (10, None, 1), (10, FAKE + 2, 1), (11, 3, 1), (12, None, 1), (12, FAKE + 4, 1), (13, None, 1), (13, FAKE + 1, 1), (14, None, 1), (14, FAKE + 2, 1),
    (15, None, 1), (15, FAKE + 8, 1), (16, 0, 5), (16, 100, 5)]]


@pytest.mark.parametrize("name,pos,value,status", BAD)
def test_bad_arguments_are_refused(native_lib, name, pos, value, status):
    args = list(GOOD[name])
    args[pos] = value
    assert getattr(native_lib, name)(*args) == status, (name, pos, value)
    assert native_lib.moe_last_error()


def test_refusals_of_combinations(native_lib):
    m = list(GOOD["moe_expert_matmul_fp4"])
    m[6], m[8] = 1, None                                         # no offsets, but counts
    assert native_lib.moe_expert_matmul_fp4(*m) == 1
    m[9], m[6] = None, 2                                         # no offsets for two experts
    assert native_lib.moe_expert_matmul_fp4(*m) == 1
    m = list(GOOD["moe_expert_matmul_fp4"])
    m[2], m[6], m[7] = BIG - 1, 1024, 1 << 20                    # E * N fills 2^30 rows; M rows make too many tiles
    assert native_lib.moe_expert_matmul_fp4(*m) == 1
    d = list(GOOD["moe_dequantize_fp4"])
    d[2], d[3] = BIG - 1, 1 << 20                                # more pieces than a grid has
    assert native_lib.moe_dequantize_fp4(*d) == 1
    a = list(GOOD["moe_expert_glu"])
    a[3], a[4] = 24, 1                                           # e4m3 takes multiples of 16
    assert native_lib.moe_expert_glu(*a) == 1
    a[2], a[3], a[4], a[6] = BIG - 1, 1 << 20, 0, None           # more pieces than a grid has
    assert native_lib.moe_expert_glu(*a) == 1


def test_small_layer_work_size(native_lib):
    size = native_lib.moe_layer_small_work_size
    assert size(4, 128, 64, 2) >= 4 * 2 * (128 + 64) * 4 and size(4, 128, 64, 2) % 256 == 0
    for bad in ((0, 128, 64, 2), (65, 128, 64, 2), (4, 8, 64, 2), (4, 16400, 64, 2), (4, 128, 0, 2), (4, 128, 64, 0), (4, 128, 64, 9)):
        assert size(*bad) == 0


M, K = 8, 64
u8 = torch.zeros(M, K // 2, dtype=torch.uint8)
sc = torch.zeros(1, M, 4, dtype=torch.uint8)
HOST = {
    "moe_quantize_fp4": lambda **a: mr.moe_quantize_fp4(torch.zeros(M, K), **a),
    "moe_dequantize_fp4": lambda **a: mr.moe_dequantize_fp4(u8, sc, **a),
    "moe_expert_matmul_fp4": lambda **a: mr.moe_expert_matmul_fp4(u8, sc, u8[None], sc[:, None], **a),
    "moe_expert_glu": lambda **a: mr.moe_expert_glu(torch.zeros(M, K), **a),
    "moe_expert_glu_bwd": lambda **a: mr.moe_expert_glu_bwd(torch.zeros(M, K), torch.zeros(M, K // 2), **a),
    "moe_layer_small": lambda **a: mr.moe_layer_small(torch.zeros(M, K, dtype=torch.bfloat16), torch.zeros(M, 2, dtype=torch.int32), torch.zeros(M, 2),
                                                      {"q": u8[None], "scale": sc[:, None]}, {"q": u8[None], "scale": sc[:, None]}, **a),
}


def test_every_entry_point_is_listed():
    assert set(HOST) == set(layer.__all__)
    assert set(layer.__all__) <= set(mr.__all__) and all(getattr(mr, n) is getattr(layer, n) for n in layer.__all__)


@pytest.mark.parametrize("name", sorted(HOST))
def test_host_tensors_are_refused_before_the_library(name, monkeypatch):
    def reached():
        raise AssertionError("a call with host tensors reached the library")
    monkeypatch.setattr(layer, "lib", reached)
    with pytest.raises(ValueError, match="CUDA tensor"):
        HOST[name]()


def test_perf_cases_make_public_calls():
    import re
    from pathlib import Path
    text = (Path(__file__).resolve().parents[1] / "perf" / "more_operators.py").read_text()
    assert set(re.findall(r"\bmr\.(\w+)\(", text)) <= set(mr.__all__)


# -- the reference forms against independent ones ----------------------------------------

def test_reference_rounding_by_the_nearest():
    x = np.concatenate([np.linspace(-6, 6, 4001), (ref.FP4[1:] + ref.FP4[:-1]) / 2])
    got = ref.values(ref.round_fp4(x))
    every = np.concatenate([ref.FP4, -ref.FP4])
    assert np.array_equal(np.abs(got - x), np.abs(every[:, None] - x).min(axis=0))
    # half-way: 1/4 3/4 5/4 7/4 5/2 7/2 5 go to the even code
    assert np.array_equal(got[-7:], [0.0, 1.0, 1.0, 2.0, 2.0, 4.0, 4.0])


def test_reference_exponent():
    a = np.array([0.0, 6.0, 6.0001, 3.0, 3.001, 1.0, 2.0 ** -133, 3e38, np.inf, np.nan])
    assert np.array_equal(ref.fp4_exponent(a)[:5], [127, 127, 128, 126, 127])
    assert np.array_equal(ref.fp4_exponent(a)[6:], [1, 253, 255, 255])


def test_reference_layout_round_trip():
    rng = np.random.default_rng(0)
    x = rng.standard_normal((5, 160))
    code, n = ref.quantize_fp4(x)
    assert np.array_equal(ref.unpack(ref.pack(code)), code)
    assert np.array_equal(ref.unfold(ref.fold(n), 160), n) and ref.fold(n).shape == (2, 5, 4)
    back = ref.read(ref.pack(code), ref.fold(n))
    assert np.array_equal(back, ref.values(code) * np.repeat(2.0 ** (n - 127.0), 32, axis=1))
    assert (np.abs(back - x) <= np.maximum(np.abs(x) / 5, np.repeat(2.0 ** (n - 127.0), 32, axis=1) / 4)).all()


def test_reference_glu_gradient_against_differences_and_autograd():
    rng = np.random.default_rng(0)
    h, dy = 3 * rng.standard_normal((4, 12)), rng.standard_normal((4, 6))
    got, step = ref.glu_bwd(h, dy), 1e-6
    for i in np.ndindex(4, 12):
        d = np.zeros_like(h)
        d[i] = step
        assert abs(((ref.glu(h + d) - ref.glu(h - d)) * dy).sum() / (2 * step) - got[i]) < 1e-7
    t = torch.from_numpy(h).requires_grad_()
    (torch.nn.functional.silu(t[:, :6]) * t[:, 6:]).backward(torch.from_numpy(dy))
    assert np.allclose(t.grad.numpy(), got, rtol=1e-12, atol=1e-14)
