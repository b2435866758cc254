"""Plain float64 (numpy) forms of the 4-bit path, the gated activation and the layer for few tokens, from
their formulas, for the tests.  Nothing here is shared with the package.  U32 and U16 are the
relative errors of one rounding to fp32 and to bf16."""

from __future__ import annotations

import numpy as np

U32, U16 = 2.0 ** -24, 2.0 ** -8
FP4 = np.array([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0])         # a code's size; the index is the code
BLOCK = 32


def round_fp4(x: np.ndarray) -> np.ndarray:
    """Codes (with bit 3 for the sign, that of a zero too) of the nearest sizes, ties to the even code."""
    a = np.abs(x)
    hi = np.clip(np.searchsorted(FP4, a, side="left"), 1, 7)
    lo = hi - 1
    dl, dh = a - FP4[lo], FP4[hi] - a
    code = np.where(dl < dh, lo, np.where(dh < dl, hi, np.where(lo % 2 == 0, lo, hi)))
    return np.where(np.signbit(x), code + 8, code).astype(np.uint8)


def values(code: np.ndarray) -> np.ndarray:
    return np.where(code >= 8, -FP4[code % 8], FP4[code % 8])


def fp4_exponent(amax: np.ndarray) -> np.ndarray:
    """The least n >= -126 with amax <= 6 * 2^n, as the byte n + 127; 127 for 0, 255 where it is not finite."""
    out = np.full(amax.shape, 127, dtype=np.int64)
    for i, a in np.ndenumerate(amax):
        if not np.isfinite(a):
            out[i] = 255
        elif a > 0:
            n = -126
            while a > 6 * 2.0 ** n:
                n += 1
            out[i] = n + 127
    return out


def quantize_fp4(x: np.ndarray):
    """(codes [M, K], exponent bytes [M, K/32])."""
    M, K = x.shape
    v = x.reshape(M, K // BLOCK, BLOCK)
    n = fp4_exponent(np.abs(v).max(axis=2))
    return round_fp4(v / 2.0 ** (n[:, :, None] - 127.0)).reshape(M, K), n


def unpack(q: np.ndarray) -> np.ndarray:
    """Codes [.., K] of bytes [.., K/2]: the even column in the low four bits."""
    return np.stack([q & 15, q >> 4], axis=-1).reshape(*q.shape[:-1], 2 * q.shape[-1])


def pack(code: np.ndarray) -> np.ndarray:
    return (code[..., 0::2] | code[..., 1::2] << 4).astype(np.uint8)


def unfold(scale: np.ndarray, K: int) -> np.ndarray:
    """Exponent bytes [.., K/32] of the stored [ceil(K/128), .., 4]."""
    s = np.moveaxis(scale, 0, -2)
    return s.reshape(*s.shape[:-2], -1)[..., :K // BLOCK]


def fold(n: np.ndarray) -> np.ndarray:
    """Exponent bytes [M, K/32] as they are stored, [ceil(K/128), M, 4]; 127 behind the last."""
    M, b = n.shape
    s = np.full((M, -(-b // 4) * 4), 127, dtype=np.uint8)
    s[:, :b] = n
    return np.ascontiguousarray(s.reshape(M, -1, 4).transpose(1, 0, 2))


def read(q: np.ndarray, scale: np.ndarray) -> np.ndarray:
    """float64 values [.., K] of codes in bytes and stored exponents; a NaN where a scale is one."""
    code = unpack(q)
    n = unfold(scale, code.shape[-1]).astype(np.float64)
    s = np.where(n == 255, np.nan, 2.0 ** (n - 127))
    return values(code) * np.repeat(s, BLOCK, axis=-1)


def sigmoid(g: np.ndarray) -> np.ndarray:
    t = np.exp(-np.abs(g))
    return np.where(g >= 0, 1.0, t) / (1.0 + t)


def glu(h: np.ndarray) -> np.ndarray:
    g, u = np.split(h, 2, axis=-1)
    return g * sigmoid(g) * u


def glu_bwd(h: np.ndarray, dy: np.ndarray) -> np.ndarray:
    g, u = np.split(h, 2, axis=-1)
    s = sigmoid(g)
    return np.concatenate([dy * u * s * (1 + g * sigmoid(-g)), dy * g * s], axis=-1)


def products(a: np.ndarray, w: np.ndarray, rows):
    """([M, N] products of the experts' rows with their weights, the sums of the products' sizes); NaN where no
    expert has the row.  rows: (first, number) of each expert."""
    out, size = np.full((a.shape[0], w.shape[1]), np.nan), np.zeros((a.shape[0], w.shape[1]))
    for e, (at, n) in enumerate(rows):
        out[at:at + n] = a[at:at + n] @ w[e].T
        size[at:at + n] = np.abs(a[at:at + n]) @ np.abs(w[e]).T
    return out, size


def layer(x, idx, gate, w1, w2):
    """([T, H], the sums of the sizes of what is added, [T, H]) of sum_j gate_j W2 glu(W1 x); an idx outside the
    experts adds nothing."""
    T, k = idx.shape
    out, size = np.zeros((T, w2.shape[1])), np.zeros((T, w2.shape[1]))
    for t in range(T):
        for j in range(k):
            e = idx[t, j]
            if 0 <= e < w1.shape[0]:
                act = glu(w1[e] @ x[t])
                out[t] += gate[t, j] * (w2[e] @ act)
                size[t] += abs(gate[t, j]) * (np.abs(w2[e]) @ np.abs(act))
    return out, size
