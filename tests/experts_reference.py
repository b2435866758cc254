"""Plain float64 (numpy) forms of the expert side's operators, from their formulas, for the tests.

Nothing here is shared with the package: rounding to e4m3, the block scales, the
choice of experts and every sum are written out.  Bounds of the comparisons:
U32 = 2^-24 and U16 = 2^-8 are the relative errors of one rounding to fp32 and
to bf16.
"""

from __future__ import annotations

import numpy as np

U32, U16 = 2.0 ** -24, 2.0 ** -8
BLOCK = 128


# -- routing -------------------------------------------------------------------

def scores(z: np.ndarray, score: str) -> np.ndarray:
    """sigmoid or softmax of float64 logits; a masked logit (-inf or NaN) scores 0."""
    masked = ~(z > -np.inf)
    if score == "sigmoid":
        with np.errstate(over="ignore", invalid="ignore"):
            s = np.where(z >= 0, 1.0, np.exp(np.minimum(z, 0.0))) / (1.0 + np.exp(-np.abs(z)))
    else:
        zz = np.where(masked, -np.inf, z)
        m = zz.max(axis=1, keepdims=True)
        e = np.where(masked, 0.0, np.exp(np.where(masked, 0.0, zz - np.where(m > -np.inf, m, 0.0))))
        total = e.sum(axis=1, keepdims=True)
        s = e / np.where(total > 0, total, 1.0)
    return np.where(masked, 0.0, s)


def choose(z, k, score, bias=None, n_groups=1, topk_groups=1, group_score="top2") -> np.ndarray:
    """The picks [T, k]: k largest choice values of the best groups, ties to the lower index."""
    T, E = z.shape
    masked = ~(z > -np.inf)
    choice = np.where(masked, -np.inf, scores(z, score) + (0.0 if bias is None else bias.astype(np.float64)))
    order = choice if bias is not None else np.where(masked, -np.inf, z)
    idx = np.empty((T, k), dtype=np.int64)
    size = E // n_groups
    for t in range(T):
        value = []
        for g in range(n_groups):
            at = slice(g * size, (g + 1) * size)
            if group_score == "max":
                value.append(order[t, at].max())
            else:
                top = sorted(choice[t, at], reverse=True)[:2]
                value.append(sum(v for v in top if v > -np.inf) if top[0] > -np.inf else -np.inf)
        best = sorted(range(n_groups), key=lambda g: (-value[g], g))[:topk_groups]
        cand = [e for g in best for e in range(g * size, (g + 1) * size)]
        idx[t] = sorted(cand, key=lambda e: (-order[t, e], e))[:k]
    return idx


def pick_weights(z, idx, score, renorm) -> np.ndarray:
    """The picks' scores [T, k], or their shares of the row's sum: there scores carry a
    common factor exp(m), so that they do not underflow."""
    zp = np.take_along_axis(z, idx, 1)
    live = zp > -np.inf
    if not renorm:
        return np.take_along_axis(scores(z, score), idx, 1)
    m = np.where(live, zp, -np.inf).max(axis=1, keepdims=True)
    m = np.where(m > -np.inf, m if score == "softmax" else np.minimum(m, 0.0), 0.0)
    zz = np.where(live, zp, 0.0)
    if score == "softmax":
        w = np.exp(np.where(live, zz - m, 0.0))
    else:
        w = np.exp(np.where(live, np.minimum(zz, 0.0) - m, 0.0)) / (1.0 + np.exp(-np.abs(zz)))
    w = np.where(live, w, 0.0)
    total = w.sum(axis=1, keepdims=True)
    return w / np.where(total > 0, total, 1.0)


def route_grad(z, idx, dgate, score, renorm, scale) -> np.ndarray:
    """dL/dz [T, E] of sum(dgate * gate), from the Jacobian of the gates, pick by pick."""
    T, E = z.shape
    s = scores(z, score)
    out = np.zeros((T, E))
    live = (idx >= 0) & (idx < E)
    safe = np.where(live, idx, 0)
    dg = np.where(live, dgate.astype(np.float64), 0.0) * scale
    if renorm:
        zz = np.where(live, np.take_along_axis(z, safe, 1), -np.inf)
        rows = np.arange(idx.shape[1])[None, :].repeat(T, 0)
        w = pick_weights(zz, rows, score, True)
        d = w * (dg - (w * dg).sum(axis=1, keepdims=True))
        if score == "sigmoid":
            d = d * (1.0 - np.take_along_axis(s, safe, 1))
        for j in range(idx.shape[1]):
            np.add.at(out, (np.arange(T), safe[:, j]), np.where(live[:, j], d[:, j], 0.0))
        return out
    dp = np.zeros((T, E))
    for j in range(idx.shape[1]):
        np.add.at(dp, (np.arange(T), safe[:, j]), dg[:, j])
    if score == "sigmoid":
        return dp * s * (1.0 - s)
    return s * (dp - (s * dp).sum(axis=1, keepdims=True))


# -- quantisation ---------------------------------------------------------------

def e4m3_values() -> np.ndarray:
    """The non-negative numbers of e4m3 (4 exponent bits, bias 7, 3 fraction bits; 448 the largest)."""
    v = [m / 8.0 * 2.0 ** -6 for m in range(8)]
    v += [(1 + m / 8.0) * 2.0 ** (e - 7) for e in range(1, 16) for m in range(8) if not (e == 15 and m == 7)]
    return np.array(v)


def round_e4m3(x: np.ndarray) -> np.ndarray:
    """x (|x| <= 448) to the nearest e4m3 number, ties to the even code."""
    v = e4m3_values()
    a = np.abs(x)
    hi = np.clip(np.searchsorted(v, a, side="left"), 1, len(v) - 1)
    lo = hi - 1
    dl, dh = a - v[lo], v[hi] - a
    code = np.where(dl < dh, lo, np.where(dh < dl, hi, np.where(lo % 2 == 0, lo, hi)))
    return np.sign(x) * v[code]


def block_scale(amax: np.ndarray) -> np.ndarray:
    """The power of two s with 224 < amax / s <= 448, at least 2^-126; 1 for 0."""
    s = np.ones_like(amax)
    for i, a in np.ndenumerate(amax):
        if a > 0:
            n = -126
            while a > 448 * 2.0 ** n:
                n += 1
            s[i] = 2.0 ** n
    return s


def quantize_rows(x: np.ndarray):
    """(values of the codes [M, K], scale [ceil(K/128), M])."""
    M, K = x.shape
    nb = -(-K // BLOCK)
    q, scale = np.empty((M, K)), np.empty((nb, M))
    for b in range(nb):
        at = slice(b * BLOCK, (b + 1) * BLOCK)
        scale[b] = block_scale(np.abs(x[:, at]).max(axis=1))
        q[:, at] = round_e4m3(x[:, at] / scale[b][:, None])
    return q, scale


def quantize_weights(w: np.ndarray):
    E, N, K = w.shape
    q, scale = np.empty_like(w), np.empty((E, -(-N // BLOCK), -(-K // BLOCK)))
    for i in range(scale.shape[1]):
        for j in range(scale.shape[2]):
            at = np.s_[:, i * BLOCK:(i + 1) * BLOCK, j * BLOCK:(j + 1) * BLOCK]
            scale[:, i, j] = block_scale(np.abs(w[at]).max(axis=(1, 2)))
            q[at] = round_e4m3(w[at] / scale[:, i, j][:, None, None])
    return q, scale


def expert_rows(offsets, kept, M):
    """(first row, rows) of every expert."""
    n = [int(offsets[e + 1]) - int(offsets[e]) for e in range(len(offsets) - 1)]
    if kept is not None:
        n = [min(a, int(b)) for a, b in zip(n, kept)]
    return [(int(offsets[e]), n[e]) for e in range(len(n))]


def quantize_cols(x: np.ndarray, rows):
    """(codes' values [K, total], scale [blocks, K]) of every expert's rows in blocks of 128, as far as they reach."""
    q, scale = [], []
    for at, n in rows:
        for i in range(0, n, BLOCK):
            v = np.zeros((BLOCK, x.shape[1]))
            part = x[at + i:at + min(n, i + BLOCK)]
            v[:len(part)] = part
            s = block_scale(np.abs(v).max(axis=0))
            scale.append(s)
            q.append(round_e4m3(v / s).T)
    K = x.shape[1]
    return (np.concatenate(q, axis=1) if q else np.zeros((K, 0))), (np.stack(scale) if scale else np.zeros((0, K)))


# -- products --------------------------------------------------------------------

def spread(scale, shape):
    """A block scale laid over the values that it stands for (last axes of `shape`)."""
    for axis in (-1, -2):
        if scale.shape[axis] != shape[axis]:
            scale = np.repeat(scale, BLOCK, axis=axis)
    return scale[..., :shape[-2], :shape[-1]]


def matmul(q, scale, wq, wscale, rows):
    """([M, N] products, [M, N] sums of the products' sizes); NaN where no expert has the row."""
    M, K = q.shape
    a = q * np.repeat(scale.T, BLOCK, axis=1)[:, :K]
    out = np.full((M, wq.shape[1]), np.nan)
    size = np.zeros((M, wq.shape[1]))
    for e, (at, n) in enumerate(rows):
        w = wq[e] * spread(wscale[e], wq[e].shape)
        out[at:at + n] = a[at:at + n] @ w.T
        size[at:at + n] = np.abs(a[at:at + n]) @ np.abs(w).T
    return out, size


def wgrad(dq, dscale, xq, xscale, rows):
    """([E, N, K], the sums of the products' sizes) from column-quantised operands."""
    out = np.zeros((len(rows), dq.shape[0], xq.shape[0]))
    size = np.zeros_like(out)
    b = 0
    for e, (_, n) in enumerate(rows):
        for _ in range(-(-n // BLOCK)):
            at = slice(b * BLOCK, (b + 1) * BLOCK)
            d, x = dq[:, at] * dscale[b][:, None], xq[:, at] * xscale[b][:, None]
            out[e] += d @ x.T
            size[e] += np.abs(d) @ np.abs(x).T
            b += 1
    return out, size


# -- dispatch and combine -----------------------------------------------------------

def dispatch(idx: np.ndarray, E: int, capacity: int):
    """The stable counting sort of moe_dispatch: perm, slot, offsets, kept."""
    flat = idx.ravel()
    perm = np.argsort(flat, kind="stable")
    counts = np.bincount(flat, minlength=E)
    offsets = np.concatenate([[0], np.cumsum(counts)])
    slot = np.empty(len(flat), dtype=np.int64)
    slot[perm] = np.arange(len(flat)) - offsets[flat[perm]]
    slot = np.where(slot < capacity, slot, -1)
    return perm, slot, offsets, np.minimum(counts, capacity)


def combine(y, idx, slot, offsets, gate):
    """([T, H] sums, sums of sizes)."""
    T, k = idx.shape
    out, size = np.zeros((T, y.shape[1])), np.zeros((T, y.shape[1]))
    for t in range(T):
        for j in range(k):
            s = slot[t * k + j]
            if s >= 0:
                v = (1.0 if gate is None else float(gate[t, j])) * y[offsets[idx[t, j]] + s]
                out[t] += v
                size[t] += np.abs(v)
    return out, size


def assert_near(name, got, want, bound):
    """|got - want| <= bound elementwise; not-a-number in the same places."""
    got, want = np.asarray(got, dtype=np.float64), np.asarray(want, dtype=np.float64)
    assert got.shape == want.shape, (name, got.shape, want.shape)
    assert np.array_equal(np.isnan(got), np.isnan(want)), f"{name}: not-a-number in other places"
    bad = np.abs(got - want) > bound
    if bad.any():
        err = np.where(bad, np.abs(got - want) - bound, 0.0)
        i = np.unravel_index(np.argmax(err), err.shape)
        raise AssertionError(f"{name}: {int(bad.sum())} of {bad.size} outside the bound; worst at {i}: got {got[i]!r}, "
                             f"want {want[i]!r}, bound {np.broadcast_to(bound, got.shape)[i]:.3e}")
