"""The expert side on the host: its C ABI loads and refuses bad arguments before anything is
queued, the binding refuses host tensors and tensors that do not belong together, and the
float64 forms that the GPU tests compare with agree with independent ones."""

import ctypes as C
import re
import subprocess
from pathlib import Path

import numpy as np
import pytest
import torch

import experts_reference as ref
import moe_expert_routing_router_gb300 as mr
from moe_expert_routing_router_gb300 import _native, experts

HEADER = Path(__file__).resolve().parents[1] / "include" / "moe_experts.h"
FAKE = 0x10000                                                   # never dereferenced


def test_header_binding_and_library_agree(native_lib):
    text = re.sub(r"/\*.*?\*/", "", HEADER.read_text(), flags=re.S)
    names = set(re.findall(r"^MOE_API [a-z_][\w \*]*?\b(moe_\w+)\s*\(", text, flags=re.M))
    assert names == set(_native.EXPERT_SIGNATURES)
    out = subprocess.run(["nm", "-D", "--defined-only", str(_native.LIB_PATH)], capture_output=True, text=True).stdout
    assert names <= {ln.split()[-1] for ln in out.splitlines() if ln.strip()}
    assert native_lib.moe_experts_abi_version() == 1
    assert set(experts.__all__) <= set(mr.__all__) and all(getattr(mr, n) is getattr(experts, n) for n in experts.__all__)


def test_header_compiles_as_c(tmp_path):
    src = tmp_path / "t.c"
    src.write_text('#include "moe_experts.h"\nint main(void) { return MOE_SCORE_SOFTMAX - 1; }\n')
    subprocess.run(["gcc", "-std=c99", "-Wall", "-Werror", "-fsyntax-only", f"-I{HEADER.parent}", str(src)], check=True)


GOOD = {
    "moe_route_fwd": [FAKE, 1, 16, 64, 4, 0, 8, 4, 1, FAKE, 1, 1.0, 0.0, None, FAKE, FAKE, FAKE, None],
    "moe_route_bwd": [FAKE, 1, 16, 64, 4, 0, 1, 1.0, FAKE, FAKE, FAKE, None],
    "moe_quantize_rows": [FAKE, 1, 16, 64, 128, FAKE, 4, FAKE, FAKE, None],
    "moe_quantize_cols": [FAKE, 1, 16, 64, 128, 8, FAKE, FAKE, FAKE, 4, FAKE, FAKE, None],
    "moe_quantize_weights": [FAKE, 1, 4, 64, 128, FAKE, FAKE, FAKE, FAKE, None],
    "moe_expert_matmul": [FAKE, FAKE, 64, 128, FAKE, FAKE, 8, 64, FAKE, FAKE, 1, FAKE, None],
    "moe_expert_wgrad": [FAKE, FAKE, FAKE, FAKE, 1024, 64, 128, 8, FAKE, FAKE, None],
    "moe_expert_combine": [FAKE, 1, 64, 128, 16, 4, 8, FAKE, FAKE, FAKE, FAKE, FAKE, None],
    "moe_expert_combine_bwd": [FAKE, FAKE, 1, 64, 128, 16, 4, 8, FAKE, FAKE, FAKE, FAKE, FAKE, FAKE, None],
}
NAN, INF, BIG = float("nan"), float("inf"), 1 << 31
BAD = [("moe_route_fwd", p, v, w) for p, v, w in [
    (0, None, 1), (0, FAKE + 1, 1), (1, 7, 2), (2, 0, 1), (2, BIG, 1), (2, 1 << 29, 1), (3, 0, 1), (3, 1025, 1), (4, 0, 1), (4, 9, 1),
    (5, 2, 1), (6, 0, 1), (6, 33, 1), (6, 7, 1), (7, 0, 1), (7, 9, 1), (8, 2, 1), (8, -1, 1), (9, FAKE + 2, 1), (10, 2, 1), (10, -2, 1),
    (11, NAN, 1), (14, None, 1), (15, None, 1), (16, None, 1), (14, FAKE + 2, 1), (16, FAKE + 1, 1)]]
BAD += [("moe_route_bwd", p, v, w) for p, v, w in [
    (0, None, 1), (1, 2, 2), (2, 0, 1), (3, 1025, 1), (4, 9, 1), (5, 2, 1), (6, 2, 1), (7, INF, 1), (8, None, 1), (9, None, 1), (10, None, 1), (10, FAKE + 2, 1)]]
BAD += [("moe_quantize_rows", p, v, w) for p, v, w in [
    (0, None, 1), (0, FAKE + 8, 1), (1, 3, 2), (2, 0, 1), (3, 0, 1), (3, BIG, 1), (4, 0, 1), (4, 136, 1), (4, 1 << 21, 1), (5, None, 1), (5, FAKE + 2, 1),
    (6, 0, 1), (6, 9, 1), (7, None, 1), (7, FAKE + 8, 1), (8, None, 1)]]
BAD += [("moe_quantize_cols", p, v, w) for p, v, w in [
    (0, None, 1), (1, 3, 2), (2, 0, 1), (3, 0, 1), (4, 24, 1), (5, 0, 1), (5, 1025, 1), (6, None, 1), (6, FAKE + 1, 1), (7, FAKE + 2, 1), (8, None, 1),
    (9, 0, 1), (10, FAKE + 4, 1), (10, None, 1), (11, None, 1), (11, FAKE + 4, 1), (3, BIG - 1, 1)]]
BAD += [("moe_quantize_weights", p, v, w) for p, v, w in [
    (0, None, 1), (0, FAKE + 2, 1), (1, 5, 2), (2, 0, 1), (3, 8, 1), (4, 72, 1), (5, None, 1), (6, None, 1), (7, None, 1), (8, None, 1), (5, FAKE + 4, 1)]]
BAD += [("moe_expert_matmul", p, v, w) for p, v, w in [
    (0, None, 1), (0, FAKE + 8, 1), (1, None, 1), (2, 0, 1), (2, BIG, 1), (3, 8, 1), (3, 120, 1), (4, None, 1), (4, FAKE + 4, 1), (5, None, 1), (6, 0, 1),
    (6, 1025, 1), (7, 40, 1), (8, None, 1), (8, FAKE + 2, 1), (9, FAKE + 2, 1), (10, 2, 2), (11, None, 1), (11, FAKE + 8, 1)]]
BAD += [("moe_expert_wgrad", p, v, w) for p, v, w in [
    (0, None, 1), (1, None, 1), (2, None, 1), (3, None, 1), (2, FAKE + 8, 1), (4, 0, 1), (4, 1000, 1), (4, BIG, 1), (5, 24, 1), (6, 0, 1), (7, 0, 1), (8, None, 1),
    (8, FAKE + 2, 1), (9, None, 1), (9, FAKE + 4, 1), (1, FAKE + 4, 1), (3, FAKE + 8, 1)]]
BAD += [("moe_expert_combine", p, v, w) for p, v, w in [
    (0, None, 1), (0, FAKE + 1, 1), (1, 4, 2), (2, 0, 1), (3, 0, 1), (3, 1 << 21, 1), (4, 0, 1), (5, 9, 1), (6, 0, 1), (7, None, 1), (8, None, 1), (9, None, 1),
    (10, FAKE + 2, 1), (11, None, 1)]]
BAD += [("moe_expert_combine_bwd", p, v, w) for p, v, w in [
    (0, None, 1), (1, None, 1), (2, 4, 2), (3, 0, 1), (4, 0, 1), (5, 0, 1), (6, 9, 1), (7, 0, 1), (8, None, 1), (9, None, 1), (10, None, 1), (11, None, 1),
    (12, None, 1), (13, None, 1), (13, FAKE + 2, 1)]]


@pytest.mark.parametrize("name,pos,value,status", BAD)
def test_bad_arguments_are_refused(native_lib, name, pos, value, status):
    args = list(GOOD[name])
    args[pos] = value
    assert getattr(native_lib, name)(*args) == status, (name, pos, value)
    assert native_lib.moe_last_error()


def test_refusals_of_combinations(native_lib):
    f = native_lib.moe_route_fwd
    a = list(GOOD["moe_route_fwd"])
    a[4], a[6], a[7] = 8, 32, 2                                  # 2 groups of 2 experts hold no 8 picks
    assert f(*a) == 1
    a = list(GOOD["moe_route_fwd"])
    a[12], a[13] = INF, FAKE                                     # an update by an infinite step
    assert f(*a) == 1
    m = list(GOOD["moe_expert_matmul"])
    m[6], m[8] = 1, None                                         # no offsets, but counts
    assert native_lib.moe_expert_matmul(*m) == 1
    m = list(GOOD["moe_expert_matmul"])
    m[6], m[7] = 1024, 1 << 20                                   # E * N fills 2^30 rows; M rows make too many tiles
    m[2] = BIG - 1
    assert native_lib.moe_expert_matmul(*m) == 1
    assert native_lib.moe_expert_device_status(None, None) == 1


def test_column_width(native_lib):
    w = native_lib.moe_quantize_cols_width
    assert w(1, 1) == 128 and w(128, 1) == 128 and w(129, 1) == 256
    for counts in ([1] * 5, [128, 1, 129], [0, 0, 256], [127] * 9):
        assert w(max(sum(counts), 1), len(counts)) >= 128 * sum(-(-c // 128) for c in counts)
    assert w(0, 1) == -1 and w(5, 0) == -1 and w(BIG, 1) == -1
    with pytest.raises(ValueError):
        mr.moe_quantize_cols_width(0, 4)


T, E, k, K = 8, 16, 2, 32
F8 = torch.float8_e4m3fn
z = torch.zeros(T, E, dtype=torch.bfloat16)
i32 = torch.zeros(T, k, dtype=torch.int32)
one = torch.zeros(E + 1, dtype=torch.int32)
HOST = {
    "moe_route_fwd": lambda **a: mr.moe_route_fwd(z, k, **a),
    "moe_route_bwd": lambda **a: mr.moe_route_bwd(z, i32, torch.zeros(T, k), **a),
    "moe_quantize_rows": lambda **a: mr.moe_quantize_rows(torch.zeros(T, K), **a),
    "moe_quantize_cols": lambda **a: mr.moe_quantize_cols(torch.zeros(T, K), one, **a),
    "moe_quantize_weights": lambda **a: mr.moe_quantize_weights(torch.zeros(E, K, K), **a),
    "moe_expert_matmul": lambda **a: mr.moe_expert_matmul(torch.zeros(T, K).to(F8), torch.ones(1, T), torch.zeros(1, K, K).to(F8), torch.ones(1, 1, 1), **a),
    "moe_expert_wgrad": lambda **a: mr.moe_expert_wgrad(torch.zeros(K, 128).to(F8), torch.ones(1, K), torch.zeros(K, 128).to(F8), torch.ones(1, K), one, **a),
    "moe_expert_combine": lambda **a: mr.moe_expert_combine(torch.zeros(T * k, K), i32, i32.view(-1), one, **a),
    "moe_expert_combine_bwd": lambda **a: mr.moe_expert_combine_bwd(torch.zeros(T, K), torch.zeros(T * k, K), i32, i32.view(-1), one, torch.zeros(T, k), **a),
}


@pytest.mark.parametrize("name", sorted(HOST))
def test_host_tensors_are_refused_before_the_library(name, monkeypatch):
    def reached():
        raise AssertionError("a call with host tensors reached the library")
    monkeypatch.setattr(experts, "lib", reached)
    with pytest.raises(ValueError, match="CUDA tensor"):
        HOST[name]()


def test_a_given_stream_is_current_while_the_call_allocates(monkeypatch):
    import contextlib
    entered = []

    @contextlib.contextmanager
    def fake(stream):
        entered.append(stream)
        yield

    monkeypatch.setattr(torch.cuda, "stream", fake)
    s = object()
    for name in sorted(HOST):
        with pytest.raises(ValueError):
            HOST[name](stream=s)
        with pytest.raises(ValueError):
            HOST[name]()
    assert entered == [s] * len(HOST)
    assert set(HOST) == set(experts.__all__) - {"moe_quantize_cols_width", "moe_expert_device_status"}


# -- the reference forms against independent ones ----------------------------------------

def test_reference_e4m3_agrees_with_torch():
    v = ref.e4m3_values()
    codes = torch.arange(127, dtype=torch.uint8).view(F8).double().numpy()
    assert np.array_equal(v, codes)
    x = np.concatenate([v, (v[:-1] + v[1:]) / 2, np.random.default_rng(0).uniform(0, 448, 20000), np.random.default_rng(1).uniform(0, 0.1, 5000)])
    x = np.concatenate([x, -x]).astype(np.float32)
    assert np.array_equal(ref.round_e4m3(x.astype(np.float64)), torch.from_numpy(x).to(F8).double().numpy())


def test_reference_block_scale():
    a = np.array([0.0, 448.0, 448.0001, 224.0, 224.001, 1.0, 2.0 ** -133, 3e38])
    s = ref.block_scale(a)
    assert np.array_equal(s[:5], [1.0, 1.0, 2.0, 0.5, 1.0])
    ok = a > 2.0 ** -117
    assert ((a / s)[ok] <= 448).all() and ((a / s)[ok] > 224).all() and s[6] == 2.0 ** -126


@pytest.mark.parametrize("score", ["sigmoid", "softmax"])
@pytest.mark.parametrize("renorm", [True, False])
def test_reference_route_gradient_against_differences(score, renorm):
    rng = np.random.default_rng(0)
    z, dg = rng.standard_normal((3, 9)), rng.standard_normal((3, 4))
    idx = ref.choose(z, 4, score)
    loss = lambda q: (1.5 * ref.pick_weights(q, idx, score, renorm) * dg).sum()  # noqa: E731
    got = ref.route_grad(z, idx, dg, score, renorm, 1.5)
    h = 1e-5
    for t in range(3):
        for e in range(9):
            d = np.zeros_like(z)
            d[t, e] = h
            assert abs((loss(z + d) - loss(z - d)) / (2 * h) - got[t, e]) < 1e-8


def test_reference_choice_by_brute_force():
    from itertools import combinations
    rng = np.random.default_rng(3)
    for trial in range(20):
        zz = rng.integers(-2, 3, (1, 12)).astype(np.float64)
        bias = (rng.integers(-2, 3, 12) * 0.25).astype(np.float32)
        c = 1 / (1 + np.exp(-zz[0])) + bias
        groups = [sum(sorted(c[g * 3:g * 3 + 3])[-2:]) for g in range(4)]
        best = max(combinations(range(4), 2), key=lambda s: (sum(groups[g] for g in s), tuple(-g for g in s)))
        cand = [e for g in best for e in range(3 * g, 3 * g + 3)]
        top = max(combinations(cand, 3), key=lambda s: (round(sum(c[e] for e in s), 12), tuple(-e for e in s)))
        assert sorted(ref.choose(zz, 3, "sigmoid", bias, 4, 2, "top2")[0]) == sorted(top)


def test_perf_cases_run_their_plain_forms_from_the_public_names():
    """Every call that the measured cases make is a public one."""
    text = (HEADER.parents[1] / "perf" / "operators.py").read_text()
    assert set(re.findall(r"\bmr\.(\w+)\(", text)) <= set(experts.__all__)
