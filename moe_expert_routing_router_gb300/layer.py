"""Python binding of what include/moe_experts.h has around the experts' 8-bit operators: 4-bit quantisation, the experts'
products on it, the gated activation between two products, and the experts of a layer for few tokens.  Argument
marshalling only, by the rules of ``experts``.
"""

from __future__ import annotations

import torch

from ._native import check, lib
from .api import _DTYPES, _out, _ptr
from .experts import _F8, _I32, _VALUES, _blocks, _choice, _entry, _gathered, _need, _need_dims, _stream

__all__ = ["moe_quantize_fp4", "moe_dequantize_fp4", "moe_expert_matmul_fp4", "moe_expert_glu", "moe_expert_glu_bwd", "moe_layer_small"]

_U8 = (torch.uint8,)                           # 4-bit codes, two in a byte, and their scales' exponents
_GLU_FORMS = {"plain": 0, "e4m3": 1, "fp4": 2}


@_entry
def moe_quantize_fp4(x: torch.Tensor, perm: torch.Tensor | None = None, k: int = 1, out: dict | None = None,
                     stream: torch.cuda.Stream | None = None) -> dict:
    """4-bit codes of blocks of 32 of the rows of x [rows, K], or of rows perm[r] // k of x: q [M, K/2] uint8 (two codes a
    byte) and scale [ceil(K/128), M, 4] uint8 (exponents).  Weights x [E, N, K] give q [E, N, K/2] and scale
    [ceil(K/128), E, N, 4] (C: moe_quantize_fp4)."""
    if isinstance(x, torch.Tensor) and x.dim() == 3:
        if perm is not None:
            raise ValueError("weights [E, N, K] are quantised as they are, without perm")
        shape = _need_dims("x", x, 3, _VALUES)
        rows, K = shape[0] * shape[1], shape[2]
        M, lead = rows, shape[:2]
    else:
        rows, K = _need_dims("x", x, 2, _VALUES)
        M = _gathered(x, perm)
        lead = (M,)
    o = {"q": _out(out, "q", (*lead, K // 2), torch.uint8, x.device),
         "scale": _out(out, "scale", (_blocks(K), *lead, 4), torch.uint8, x.device)}
    check(lib().moe_quantize_fp4(_ptr(x), _DTYPES[x.dtype], rows, M, K, _ptr(perm), int(k), _ptr(o["q"]), _ptr(o["scale"]),
                                 _stream()), "moe_quantize_fp4")
    return o


@_entry
def moe_dequantize_fp4(q: torch.Tensor, scale: torch.Tensor, dtype: torch.dtype = torch.bfloat16,
                       out: torch.Tensor | None = None, stream: torch.cuda.Stream | None = None) -> torch.Tensor:
    """The values [M, K] (weights: [E, N, K]) that moe_quantize_fp4's codes stand for, exact in fp32 and bf16; ``out``, when
    given, decides the type (C: moe_dequantize_fp4)."""
    lead = _need_dims("q", q, 3 if isinstance(q, torch.Tensor) and q.dim() == 3 else 2, _U8)[:-1]
    K = 2 * q.shape[-1]
    _need("scale", scale, q.get_device(), torch.uint8, (_blocks(K), *lead, 4))
    if out is not None:
        dtype = out.dtype
    if dtype not in _DTYPES:
        raise ValueError("the result must be float32 or bfloat16")
    y = _out({"out": out}, "out", (*lead, K), dtype, q.device)
    check(lib().moe_dequantize_fp4(_ptr(q), _ptr(scale), lead.numel(), K, _DTYPES[dtype], _ptr(y), _stream()), "moe_dequantize_fp4")
    return y


@_entry
def moe_expert_matmul_fp4(q: torch.Tensor, scale: torch.Tensor, wq: torch.Tensor, wscale: torch.Tensor,
                          offsets: torch.Tensor | None = None, kept: torch.Tensor | None = None,
                          out_dtype: torch.dtype = torch.bfloat16, out: torch.Tensor | None = None,
                          stream: torch.cuda.Stream | None = None) -> torch.Tensor:
    """out [M, N]: the rows offsets[e] .. offsets[e] + kept[e] of moe_quantize_fp4's q [M, K/2] times expert e's weights
    wq [E, N, K/2], transposed, each with its scales (C: moe_expert_matmul_fp4).  Other rows of ``out`` are left as they
    are.  Without offsets, one expert takes all rows.  ``out``, when given, decides the type."""
    M, half = _need_dims("q", q, 2, _U8)
    at = q.get_device()
    E, N, _ = _need_dims("wq", wq, 3, _U8, at)
    _need("wq", wq, at, torch.uint8, (E, N, half))
    _need("scale", scale, at, torch.uint8, (_blocks(2 * half), M, 4))
    _need("wscale", wscale, at, torch.uint8, (_blocks(2 * half), E, N, 4))
    if offsets is not None:
        _need("offsets", offsets, at, torch.int32, (E + 1,))
    if kept is not None:
        _need("kept", kept, at, torch.int32, (E,))
    if out is not None:
        out_dtype = out.dtype
    if out_dtype not in _DTYPES:
        raise ValueError("the result must be float32 or bfloat16")
    y = _out({"out": out}, "out", (M, N), out_dtype, q.device)
    check(lib().moe_expert_matmul_fp4(_ptr(q), _ptr(scale), M, 2 * half, _ptr(wq), _ptr(wscale), E, N, _ptr(offsets), _ptr(kept),
                                      _DTYPES[out_dtype], _ptr(y), _stream()), "moe_expert_matmul_fp4")
    return y


@_entry
def moe_expert_glu(h: torch.Tensor, form: str = "plain", out: dict | torch.Tensor | None = None,
                   stream: torch.cuda.Stream | None = None) -> torch.Tensor | dict:
    """silu(h[:, :I]) * h[:, I:] of h [M, 2I]: a tensor [M, I] of h's type, or with another form the next product's operand,
    {"q", "scale"} as moe_quantize_rows ("e4m3") or moe_quantize_fp4 ("fp4") give them; ``out`` is a tensor or a dict
    accordingly (C: moe_expert_glu)."""
    M, width = _need_dims("h", h, 2, _VALUES)
    if width % 2 != 0:
        raise ValueError(f"h must be [M, 2I], got {tuple(h.shape)}")
    f, I, dev = _choice("form", form, _GLU_FORMS), width // 2, h.device
    if f == 0:
        if isinstance(out, dict):
            raise ValueError("of plain values, out is a tensor")
        o = {"q": _out({"out": out}, "out", (M, I), h.dtype, dev), "scale": None}
    else:
        if out is not None and not isinstance(out, dict):
            raise ValueError("of a quantised form, out is a dict of q and scale")
        o = {"q": _out(out, "q", (M, I), _F8, dev) if f == 1 else _out(out, "q", (M, I // 2), torch.uint8, dev),
             "scale": _out(out, "scale", (_blocks(I), M), torch.float32, dev) if f == 1 else
             _out(out, "scale", (_blocks(I), M, 4), torch.uint8, dev)}
    check(lib().moe_expert_glu(_ptr(h), _DTYPES[h.dtype], M, I, f, _ptr(o["q"]), _ptr(o["scale"]), _stream()), "moe_expert_glu")
    return o if f else o["q"]


@_entry
def moe_expert_glu_bwd(h: torch.Tensor, dy: torch.Tensor, out: torch.Tensor | None = None,
                       stream: torch.cuda.Stream | None = None) -> torch.Tensor:
    """dh [M, 2I] from dy [M, I], the gradient of moe_expert_glu's value, in h's type (C: moe_expert_glu_bwd)."""
    M, width = _need_dims("h", h, 2, _VALUES)
    if width % 2 != 0:
        raise ValueError(f"h must be [M, 2I], got {tuple(h.shape)}")
    _need("dy", dy, h.get_device(), h.dtype, (M, width // 2))
    dh = _out({"out": out}, "out", (M, width), h.dtype, h.device)
    check(lib().moe_expert_glu_bwd(_ptr(h), _ptr(dy), _DTYPES[h.dtype], M, width // 2, _ptr(dh), _stream()), "moe_expert_glu_bwd")
    return dh


def _weights(name: str, w: dict, E: int | None, N: int | None, K: int | None, at: int) -> tuple[int, int, int, int, torch.Tensor, torch.Tensor]:
    """(kind, E, N, K, codes, scales) of quantised weights, whose sizes are as given where they are."""
    if not isinstance(w, dict) or "q" not in w or "scale" not in w:
        raise ValueError(f"{name} must be a dict of q and scale, as moe_quantize_weights or moe_quantize_fp4 give it")
    q, scale = w["q"], w["scale"]
    e, n, width = _need_dims(f"{name}['q']", q, 3, (_F8, torch.uint8), at)
    fp4 = q.dtype is torch.uint8
    k = 2 * width if fp4 else width
    if (E is not None and e != E) or (N is not None and n != N) or (K is not None and k != K):
        raise ValueError(f"{name} must hold weights {(E, N, K)}, got {(e, n, k)}")
    if fp4:
        _need(f"{name}['scale']", scale, at, torch.uint8, (_blocks(k), e, n, 4))
    else:
        _need(f"{name}['scale']", scale, at, torch.float32, (e, _blocks(n), _blocks(k)))
    return int(fp4), e, n, k, q, scale


@_entry
def moe_layer_small(x: torch.Tensor, idx: torch.Tensor, gate: torch.Tensor, w1: dict, w2: dict, out: torch.Tensor | None = None,
                    stream: torch.cuda.Stream | None = None) -> torch.Tensor:
    """out [T, H] bf16 = sum_j gate[t, j] * W2_e silu(G_e x_t) * (U_e x_t), e = idx[t, j], for up to 64 tokens x [T, H] bf16:
    what follows moe_route_fwd in a layer, in three kernels.  w1 holds the weights [E, 2I, H] (G's rows, then U's) and w2
    [E, H, I], each as moe_quantize_weights or moe_quantize_fp4 gives them; idx and gate are [T, k], and an idx outside
    [0, E) adds nothing (C: moe_layer_small)."""
    T, H = _need_dims("x", x, 2, (torch.bfloat16,))
    at = x.get_device()
    k = _need_dims("idx", idx, 2, _I32, at)[1]
    _need("idx", idx, at, torch.int32, (T, k))
    _need("gate", gate, at, torch.float32, (T, k))
    kind1, E, N1, _, q1, s1 = _weights("w1", w1, None, None, H, at)
    if N1 % 2 != 0:
        raise ValueError(f"w1 must hold weights [E, 2I, H], got {N1} rows")
    kind2, _, _, I, q2, s2 = _weights("w2", w2, E, H, N1 // 2, at)
    o = _out({"out": out}, "out", (T, H), torch.bfloat16, x.device)
    need = int(lib().moe_layer_small_work_size(T, H, I, k))
    work = torch.empty(max(need, 1), dtype=torch.uint8, device=x.device)
    check(lib().moe_layer_small(_ptr(x), T, H, I, E, k, _ptr(idx), _ptr(gate), kind1, _ptr(q1), _ptr(s1), kind2, _ptr(q2), _ptr(s2),
                                _ptr(o), _ptr(work), need, _stream()), "moe_layer_small")
    return o
