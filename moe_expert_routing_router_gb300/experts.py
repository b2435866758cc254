"""Python binding of the expert side's C ABI (include/moe_experts.h): argument marshalling only.

Scored group-limited routing, block-scaled 8-bit quantisation, the experts'
matrix products and the gated combine, each with its gradient.  As in ``api``,
every function takes CUDA tensors, allocates its outputs with torch (on
``stream`` when one is given), passes raw pointers to the library and checks the
returned status.  The tensors of a call lie on one device; it need not be the
current one.
"""

from __future__ import annotations

import contextlib
import ctypes as C
import functools
import inspect

import torch

from ._native import check, lib
from .api import _DTYPES, _need_cuda, _on, _out, _ptr

__all__ = [
    "moe_route_fwd", "moe_route_bwd", "moe_quantize_rows", "moe_quantize_cols", "moe_quantize_cols_width",
    "moe_quantize_weights", "moe_expert_matmul", "moe_expert_wgrad", "moe_expert_device_status", "moe_expert_combine",
    "moe_expert_combine_bwd",
]

_VALUES = tuple(_DTYPES)                       # fp32 and bf16
_I32, _F32 = (torch.int32,), (torch.float32,)
_SCORES = {"sigmoid": 0, "softmax": 1}
_GROUP_SCORES = {"max": 0, "top2": 1}
_F8 = torch.float8_e4m3fn
_CODES = (_F8,)
_BLOCK = 128


# The current device and its current stream's handle, without the stream object around it (a call's
# arguments are checked and its outputs allocated in some 10 us; the object alone takes 3).
_device = torch._C._cuda_getDevice if hasattr(torch._C, "_cuda_getDevice") else torch.cuda.current_device


def _stream() -> int:
    return torch._C._cuda_getCurrentRawStream(_device())


def _entry(fn):
    """Runs an entry point on the device of its first argument, with its `stream`
    argument, when given, as torch's current stream (see ``api._on_stream``)."""
    pos = list(inspect.signature(fn).parameters).index("stream")
    first = next(iter(inspect.signature(fn).parameters))

    @functools.wraps(fn)
    def call(*args, **kwargs):
        stream = args[pos] if len(args) > pos else kwargs.get("stream")
        t = args[0] if args else kwargs.get(first)
        on = isinstance(t, torch.Tensor) and t.is_cuda
        if stream is None and (not on or t.get_device() == _device()):
            return fn(*args, **kwargs)
        if on and stream is not None and stream.device != t.device:
            raise ValueError(f"the stream is on {stream.device}, {first} on {t.device}")
        with torch.cuda.device(t.device) if on else contextlib.nullcontext(), _on(stream):
            return fn(*args, **kwargs)
    return call


def _fault(name: str, t, index: int | None, dtypes, shape) -> None:
    """Says what is wrong with an argument that `_ok` has refused."""
    _need_cuda(name, t)
    if t.dtype not in dtypes:
        raise ValueError(f"{name} must be {' or '.join(str(d) for d in dtypes)}, got {t.dtype}")
    if index is not None and t.get_device() != index:
        raise ValueError(f"{name} is on {t.device}, the call's tensors on cuda:{index}")
    raise ValueError(f"{name} must be {shape}, got {tuple(t.shape)}")


def _need(name: str, t: torch.Tensor, index: int, dtype: torch.dtype, shape: tuple) -> None:
    """A contiguous CUDA tensor on device `index`, of `dtype` and `shape`."""
    if not (isinstance(t, torch.Tensor) and t.get_device() == index and t.dtype is dtype and t.shape == shape and t.is_contiguous()):
        _fault(name, t, index, (dtype,), shape)


def _need_dims(name: str, t: torch.Tensor, dims: int, dtypes, index: int | None = None) -> torch.Size:
    """As `_need` for a tensor whose lengths the call takes from it; returns them.  Without an index the tensor
    decides the call's device."""
    if not (isinstance(t, torch.Tensor) and t.is_cuda and t.dtype in dtypes and t.dim() == dims and t.is_contiguous()
            and (index is None or t.get_device() == index)):
        _fault(name, t, index, dtypes, f"{dims}-D")
    return t.shape


def _choice(name: str, value, table: dict) -> int:
    if value not in table:
        raise ValueError(f"{name} must be one of {sorted(table)}, got {value!r}")
    return table[value]


def _blocks(n: int) -> int:
    return (n + _BLOCK - 1) // _BLOCK


@_entry
def moe_route_fwd(logits: torch.Tensor, k: int, score: str = "sigmoid", bias: torch.Tensor | None = None,
                  n_groups: int = 1, topk_groups: int = 1, group_score: str = "top2", renorm: int = -1,
                  scale: float = 1.0, bias_gamma: float = 0.0, bias_out: torch.Tensor | bool | None = None,
                  out: dict | None = None, stream: torch.cuda.Stream | None = None) -> dict:
    """Scored, group-limited routing of logits [T, E] (C: moe_route_fwd).

    Returns idx [T, k] int32 (largest choice value first), gate [T, k] fp32 and
    counts [E] int32; and ``bias_out`` when an update is asked for: a tensor to
    receive it (it may be ``bias`` itself), or True for a new one."""
    T, E = _need_dims("logits", logits, 2, _VALUES)
    dev, at = logits.device, logits.get_device()
    if bias is not None:
        _need("bias", bias, at, torch.float32, (E,))
    if bias_out is True:
        bias_out = torch.empty(E, dtype=torch.float32, device=dev)
    elif bias_out is False:
        bias_out = None
    if bias_out is not None:
        _need("bias_out", bias_out, at, torch.float32, (E,))
    sc, gs = _choice("score", score, _SCORES), _choice("group_score", group_score, _GROUP_SCORES)
    k = int(k)
    o = {"idx": _out(out, "idx", (T, max(k, 0)), torch.int32, dev),
         "gate": _out(out, "gate", (T, max(k, 0)), torch.float32, dev),
         "counts": _out(out, "counts", (E,), torch.int32, dev)}
    check(lib().moe_route_fwd(_ptr(logits), _DTYPES[logits.dtype], T, E, k, sc, int(n_groups), int(topk_groups), gs,
                              _ptr(bias), int(renorm), float(scale), float(bias_gamma), _ptr(bias_out),
                              _ptr(o["idx"]), _ptr(o["gate"]), _ptr(o["counts"]), _stream()), "moe_route_fwd")
    if bias_out is not None:
        o["bias_out"] = bias_out
    return o


@_entry
def moe_route_bwd(logits: torch.Tensor, idx: torch.Tensor, dgate: torch.Tensor, score: str = "sigmoid",
                  renorm: int = -1, scale: float = 1.0, dlogits: torch.Tensor | None = None,
                  stream: torch.cuda.Stream | None = None) -> torch.Tensor:
    """dL/dlogits [T, E] fp32 from the gates' gradient dgate [T, k], picks held constant (C: moe_route_bwd)."""
    T, E = _need_dims("logits", logits, 2, _VALUES)
    dev, at = logits.device, logits.get_device()
    k = _need_dims("idx", idx, 2, _I32, at)[1]
    _need("idx", idx, at, torch.int32, (T, k))
    _need("dgate", dgate, at, torch.float32, (T, k))
    sc = _choice("score", score, _SCORES)
    dl = _out({"dlogits": dlogits}, "dlogits", (T, E), torch.float32, dev)
    check(lib().moe_route_bwd(_ptr(logits), _DTYPES[logits.dtype], T, E, k, sc, int(renorm), float(scale),
                              _ptr(idx), _ptr(dgate), _ptr(dl), _stream()), "moe_route_bwd")
    return dl


def _gathered(x: torch.Tensor, perm: torch.Tensor | None) -> int:
    """Rows of the quantised output."""
    if perm is None:
        return x.shape[0]
    return _need_dims("perm", perm, 1, _I32, x.get_device())[0]


@_entry
def moe_quantize_rows(x: torch.Tensor, perm: torch.Tensor | None = None, k: int = 1, out: dict | None = None,
                      stream: torch.cuda.Stream | None = None) -> dict:
    """q [M, K] e4m3 and scale [ceil(K/128), M] of the rows of x, or of rows perm[r] // k of x: the token rows in
    dispatch order (C: moe_quantize_rows)."""
    rows, K = _need_dims("x", x, 2, _VALUES)
    M = _gathered(x, perm)
    o = {"q": _out(out, "q", (M, K), _F8, x.device),
         "scale": _out(out, "scale", (_blocks(K), M), torch.float32, x.device)}
    check(lib().moe_quantize_rows(_ptr(x), _DTYPES[x.dtype], rows, M, K, _ptr(perm), int(k), _ptr(o["q"]),
                                  _ptr(o["scale"]), _stream()), "moe_quantize_rows")
    return o


def moe_quantize_cols_width(M: int, E: int) -> int:
    """Columns of moe_quantize_cols's output for M rows of E experts (C: moe_quantize_cols_width)."""
    w = int(lib().moe_quantize_cols_width(int(M), int(E)))
    if w < 0:
        raise ValueError(f"invalid sizes for quantised columns: M={M}, E={E}")
    return w


@_entry
def moe_quantize_cols(x: torch.Tensor, offsets: torch.Tensor, kept: torch.Tensor | None = None,
                      perm: torch.Tensor | None = None, k: int = 1, out: dict | None = None,
                      stream: torch.cuda.Stream | None = None) -> dict:
    """q [K, width] e4m3 and scale [width/128, K]: every expert's rows of x (or of rows perm[r] // k of x) in blocks of
    128 rows by one column, transposed, as moe_expert_wgrad takes them (C: moe_quantize_cols)."""
    rows, K = _need_dims("x", x, 2, _VALUES)
    dev, at = x.device, x.get_device()
    M = _gathered(x, perm)
    E = _need_dims("offsets", offsets, 1, _I32, at)[0] - 1
    if kept is not None:
        _need("kept", kept, at, torch.int32, (E,))
    width = moe_quantize_cols_width(M, E)
    o = {"q": _out(out, "q", (K, width), _F8, dev),
         "scale": _out(out, "scale", (width // _BLOCK, K), torch.float32, dev)}
    check(lib().moe_quantize_cols(_ptr(x), _DTYPES[x.dtype], rows, M, K, E, _ptr(offsets), _ptr(kept), _ptr(perm), int(k),
                                  _ptr(o["q"]), _ptr(o["scale"]), _stream()), "moe_quantize_cols")
    return o


@_entry
def moe_quantize_weights(w: torch.Tensor, transposed: bool = False, out: dict | None = None,
                         stream: torch.cuda.Stream | None = None) -> dict:
    """q [E, N, K] e4m3 and scale [E, ceil(N/128), ceil(K/128)] of w [E, N, K]; with ``transposed`` also qt [E, K, N] and
    scalet [E, ceil(K/128), ceil(N/128)], the weights of the data gradient (C: moe_quantize_weights)."""
    E, N, K = _need_dims("w", w, 3, _VALUES)
    dev = w.device
    o = {"q": _out(out, "q", (E, N, K), _F8, dev),
         "scale": _out(out, "scale", (E, _blocks(N), _blocks(K)), torch.float32, dev)}
    if transposed:
        o["qt"] = _out(out, "qt", (E, K, N), _F8, dev)
        o["scalet"] = _out(out, "scalet", (E, _blocks(K), _blocks(N)), torch.float32, dev)
    check(lib().moe_quantize_weights(_ptr(w), _DTYPES[w.dtype], E, N, K, _ptr(o["q"]), _ptr(o["scale"]),
                                     _ptr(o.get("qt")), _ptr(o.get("scalet")), _stream()), "moe_quantize_weights")
    return o


@_entry
def moe_expert_matmul(q: torch.Tensor, scale: torch.Tensor, wq: torch.Tensor, wscale: torch.Tensor,
                      offsets: torch.Tensor | None = None, kept: torch.Tensor | None = None,
                      out_dtype: torch.dtype = torch.bfloat16, out: torch.Tensor | None = None,
                      stream: torch.cuda.Stream | None = None) -> torch.Tensor:
    """out [M, N]: the rows offsets[e] .. offsets[e] + kept[e] of q (scaled) times expert e's weights wq [E, N, K]
    (scaled), transposed (C: moe_expert_matmul).  Other rows of ``out`` are left as they are.  Without offsets, one
    expert takes all rows.  ``out``, when given, decides the type."""
    M, K = _need_dims("q", q, 2, _CODES)
    at = q.get_device()
    E, N, _ = _need_dims("wq", wq, 3, _CODES, at)
    _need("wq", wq, at, _F8, (E, N, K))
    _need("scale", scale, at, torch.float32, (_blocks(K), M))
    _need("wscale", wscale, at, torch.float32, (E, _blocks(N), _blocks(K)))
    if offsets is not None:
        _need("offsets", offsets, at, torch.int32, (E + 1,))
    if kept is not None:
        _need("kept", kept, at, torch.int32, (E,))
    if out is not None:
        out_dtype = out.dtype
    if out_dtype not in _DTYPES:
        raise ValueError("the result must be float32 or bfloat16")
    y = _out({"out": out}, "out", (M, N), out_dtype, q.device)
    check(lib().moe_expert_matmul(_ptr(q), _ptr(scale), M, K, _ptr(wq), _ptr(wscale), E, N, _ptr(offsets), _ptr(kept),
                                  _DTYPES[out_dtype], _ptr(y), _stream()), "moe_expert_matmul")
    return y


@_entry
def moe_expert_wgrad(dyq: torch.Tensor, dyscale: torch.Tensor, xq: torch.Tensor, xscale: torch.Tensor, kept: torch.Tensor,
                     out: torch.Tensor | None = None, stream: torch.cuda.Stream | None = None) -> torch.Tensor:
    """dw [E, N, K] fp32 = sum over every expert's rows of dy^T x, from moe_quantize_cols of dy and x (C: moe_expert_wgrad)."""
    N, width = _need_dims("dyq", dyq, 2, _CODES)
    at = dyq.get_device()
    if width % _BLOCK != 0:
        raise ValueError("the columns of dyq must be whole blocks of 128")
    K = _need_dims("xq", xq, 2, _CODES, at)[0]
    _need("xq", xq, at, _F8, (K, width))
    _need("dyscale", dyscale, at, torch.float32, (width // _BLOCK, N))
    _need("xscale", xscale, at, torch.float32, (width // _BLOCK, K))
    E = _need_dims("kept", kept, 1, _I32, at)[0]
    dw = _out({"out": out}, "out", (E, N, K), torch.float32, dyq.device)
    check(lib().moe_expert_wgrad(_ptr(dyq), _ptr(dyscale), _ptr(xq), _ptr(xscale), width, N, K, E, _ptr(kept), _ptr(dw),
                                 _stream()), "moe_expert_wgrad")
    return dw


def moe_expert_device_status(stream: torch.cuda.Stream | None = None) -> int:
    """Reads and clears the error bits that the expert products have left on the current device (synchronises)."""
    flags = C.c_int32(0)
    with _on(stream):
        st = lib().moe_expert_device_status(_stream(), C.byref(flags))
    if flags.value == 0:
        check(st, "moe_expert_device_status")
    return int(flags.value)


def _assignments(idx, slot, offsets, gate, at: int) -> tuple[int, int, int]:
    T, k = _need_dims("idx", idx, 2, _I32, at)
    if not isinstance(slot, torch.Tensor) or slot.numel() != T * k:
        _need_cuda("slot", slot)
        raise ValueError("slot must have T*k elements")
    _need("slot", slot, at, torch.int32, slot.shape)
    E = _need_dims("offsets", offsets, 1, _I32, at)[0] - 1
    if gate is not None:
        _need("gate", gate, at, torch.float32, (T, k))
    return T, k, E


@_entry
def moe_expert_combine(y: torch.Tensor, idx: torch.Tensor, slot: torch.Tensor, offsets: torch.Tensor,
                       gate: torch.Tensor | None = None, out: torch.Tensor | None = None,
                       stream: torch.cuda.Stream | None = None) -> torch.Tensor:
    """out [T, H]: every token's kept rows of y [M, H], summed by gate, or plainly without one (C: moe_expert_combine)."""
    M, H = _need_dims("y", y, 2, _VALUES)
    T, k, E = _assignments(idx, slot, offsets, gate, y.get_device())
    o = _out({"out": out}, "out", (T, H), y.dtype, y.device)
    check(lib().moe_expert_combine(_ptr(y), _DTYPES[y.dtype], M, H, T, k, E, _ptr(idx), _ptr(slot), _ptr(offsets),
                                   _ptr(gate), _ptr(o), _stream()), "moe_expert_combine")
    return o


@_entry
def moe_expert_combine_bwd(dout: torch.Tensor, y: torch.Tensor, idx: torch.Tensor, slot: torch.Tensor,
                           offsets: torch.Tensor, gate: torch.Tensor, out: dict | None = None,
                           stream: torch.cuda.Stream | None = None) -> dict:
    """dy [M, H] (rows of kept assignments; others are left as they are) and dgate [T, k] fp32 of
    moe_expert_combine (C: moe_expert_combine_bwd)."""
    _need_dims("dout", dout, 2, _VALUES)
    dev, at = dout.device, dout.get_device()
    M, H = _need_dims("y", y, 2, (dout.dtype,), at)
    if gate is None:
        raise ValueError("gate must be a CUDA tensor")
    T, k, E = _assignments(idx, slot, offsets, gate, at)
    _need("dout", dout, at, y.dtype, (T, H))
    o = {"dy": _out(out, "dy", (M, H), y.dtype, dev), "dgate": _out(out, "dgate", (T, k), torch.float32, dev)}
    check(lib().moe_expert_combine_bwd(_ptr(dout), _ptr(y), _DTYPES[y.dtype], M, H, T, k, E, _ptr(idx), _ptr(slot),
                                       _ptr(offsets), _ptr(gate), _ptr(o["dy"]), _ptr(o["dgate"]), _stream()),
          "moe_expert_combine_bwd")
    return o
