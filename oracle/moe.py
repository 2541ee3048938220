"""Expert-layer operators in 64 bits: routing and its gradient, the order of
rows, the weighted sum back and its gradient, the experts' products and
weight gradients over ragged rows, the gated activation and its gradient.

Plain numpy, from the formulas; index results are exact, float results are
float64.  Pinned in tests/test_oracle_moe.py by differences, brute force and
closed forms.
"""
from __future__ import annotations

import numpy as np


def scores(x, sigmoid: bool) -> np.ndarray:
    """p [T, E]; a row of -inf alone has scores of zero."""
    x = np.asarray(x, np.float64)
    with np.errstate(over="ignore", invalid="ignore", divide="ignore"):
        if sigmoid:
            return 1.0 / (1.0 + np.exp(-x))
        top = x.max(1, keepdims=True)
        p = np.exp(x - np.where(np.isfinite(top), top, 0.0))
        total = p.sum(1, keepdims=True)
        return np.where(total > 0, p / np.where(total > 0, total, 1.0), 0.0)


def shares(x, on, sigmoid: bool) -> np.ndarray:
    """p / sum of p over the logits [T, k] that are `on`: of e^x or
    1 / (1 + e^-x) times a power of e that makes the row's largest ordinary, so
    that no row of finite logits is lost to underflow; zeros for a row of -inf."""
    x = np.where(on, np.asarray(x, np.float64), -np.inf)
    with np.errstate(over="ignore", invalid="ignore"):
        m = x.max(1, keepdims=True)
        m = np.minimum(m, 0.0) if sigmoid else m
        m = np.where(m == -np.inf, 0.0, m)
        a = np.exp(np.minimum(x, 0.0) - m) / (1.0 + np.exp(-np.abs(x))) if sigmoid else np.exp(x - m)
        total = a.sum(1, keepdims=True)
    return np.where(total == 0, 0.0, a / np.where(total == 0, 1.0, total))


def route(x, k, bias=None, groups=1, top_groups=1, group_top=1, sigmoid=False, renorm=True, scale=1.0):
    """(ids [T, k], weights [T, k], p [T, E])."""
    p = scores(x, sigmoid)
    T, E = p.shape
    c = p + (0.0 if bias is None else np.asarray(bias, np.float64))
    ids = np.zeros((T, k), np.int32)
    for t in range(T):
        left = c[t].copy()
        if groups > 1:
            by = c[t].reshape(groups, E // groups)
            worth = np.sort(by, axis=1)[:, ::-1][:, :group_top].sum(1)
            best = sorted(range(groups), key=lambda g: (-worth[g], g))[:top_groups]
            keep = np.isin(np.arange(groups), best).repeat(E // groups)
            left = np.where(keep, left, -np.inf)
        ids[t] = sorted(range(E), key=lambda e: (-left[e], e))[:k]
    w = np.take_along_axis(p, ids.astype(np.int64), 1)
    if renorm:
        w = shares(np.take_along_axis(np.asarray(x, np.float64), ids.astype(np.int64), 1), True, sigmoid)
    return ids, w * scale, p


def route_backward(x, ids, dw, ds=None, sigmoid=False, renorm=True, scale=1.0):
    """dlogits [T, E] and a bound's size: the same sums of absolute values."""
    p = scores(x, sigmoid)
    T, E = p.shape
    ids = np.asarray(ids, np.int64)
    on = (ids >= 0) & (ids < E)
    at = np.where(on, ids, 0)
    pc = np.where(on, np.take_along_axis(p, at, 1), 0.0)
    d = np.where(on, np.asarray(dw, np.float64) * scale, 0.0)
    m = np.abs(d)
    if renorm:
        # of w = p / sum: w (d - sum w d) = p dp, the factor 1 - p of a sigmoid aside
        w = shares(np.take_along_axis(np.asarray(x, np.float64), at, 1), on, sigmoid)
        d, m = w * (d - (w * d).sum(1, keepdims=True)), w * (m + (w * m).sum(1, keepdims=True))
    else:
        d, m = d * pc, m * pc
    c, mc = np.zeros((T, E)), np.zeros((T, E))  # p dp of the choices
    for t in range(T):
        for j in range(ids.shape[1]):
            if on[t, j]:
                c[t, ids[t, j]] += d[t, j]
                mc[t, ids[t, j]] += m[t, j]
    if ds is not None:
        c += p * ds
        mc += p * np.abs(ds)
    if sigmoid:
        q = scores(-np.asarray(x, np.float64), True)
        return c * q, mc * q
    return c - p * c.sum(1, keepdims=True), mc + p * mc.sum(1, keepdims=True)


def plan(ids, E, align, cap):
    """(offsets [E + 1], counts [E], rows [cap], pos like ids)."""
    flat = np.asarray(ids).reshape(-1)
    rows = np.full(cap, -1, np.int32)
    pos = np.full(flat.size, -1, np.int32)
    offsets, counts, at = [0], [], 0
    for e in range(E):
        mine = np.nonzero(flat == e)[0]
        for i, c in enumerate(mine):
            rows[at + i] = c
            pos[c] = at + i
        at += -(-mine.size // align) * align
        counts.append(mine.size)
        offsets.append(at)
    return np.array(offsets, np.int32), np.array(counts, np.int32), rows, pos.reshape(np.shape(ids))


def gather(x, rows, k, weights=None):
    """float32 [cap, H] in the order of rows; the product with a weight is
    one float32 multiplication."""
    x = np.asarray(x, np.float32)
    out = np.zeros((len(rows), x.shape[1]), np.float32)
    for r, c in enumerate(rows):
        if 0 <= c < x.shape[0] * k:
            out[r] = x[c // k]
            if weights is not None:
                out[r] = x[c // k] * np.float32(weights.reshape(-1)[c])
    return out


def combine(y, pos, weights=None):
    """(out [T, H], the same sum of absolute values)."""
    y = np.asarray(y, np.float64)
    T, k = pos.shape
    out, size = np.zeros((T, y.shape[1])), np.zeros((T, y.shape[1]))
    for t in range(T):
        for j in range(k):
            r = pos[t, j]
            if 0 <= r < y.shape[0]:
                w = 1.0 if weights is None else float(weights[t, j])
                out[t] += w * y[r]
                size[t] += np.abs(w * y[r])
    return out, size


def combine_backward(y, pos, dout):
    y, dout = np.asarray(y, np.float64), np.asarray(dout, np.float64)
    ok = (pos >= 0) & (pos < y.shape[0])
    if y.shape[0] == 0:
        return np.zeros(pos.shape), np.zeros(pos.shape)
    v = y[np.where(ok, pos, 0)] * dout[:, None, :]
    return np.where(ok, v.sum(2), 0.0), np.where(ok, np.abs(v).sum(2), 0.0)


def _group_max(a):
    """Maxima of |a| over 8 neighbours along the last axis."""
    return np.abs(a).reshape(*a.shape[:-1], -1, 8).max(-1)


def product(a, b, offsets, cap, rows=None, k=1):
    """(out, sum of |products|, sum over 8-groups of max|a| max|b|), each
    [cap, N], of operands already decoded to values."""
    a, b = np.asarray(a, np.float64), np.asarray(b, np.float64)
    N = b.shape[1]
    res = [np.zeros((cap, N)) for _ in range(3)]
    for e in range(b.shape[0]):
        for r in range(offsets[e], offsets[e + 1]):
            c = r if rows is None else (rows[r] // k if rows[r] >= 0 else -1)
            if 0 <= c < a.shape[0]:
                res[0][r] = b[e] @ a[c]
                res[1][r] = np.abs(b[e]) @ np.abs(a[c])
                res[2][r] = _group_max(b[e]) @ _group_max(a[c])
    return res


def wgrad(dyt, xt, offsets):
    dyt, xt = np.asarray(dyt, np.float64), np.asarray(xt, np.float64)
    res = [[], [], []]
    for lo, hi in zip(offsets[:-1], offsets[1:]):
        d, x = dyt[:, lo:hi], xt[:, lo:hi]
        res[0].append(d @ x.T)
        res[1].append(np.abs(d) @ np.abs(x).T)
        res[2].append(_group_max(d) @ _group_max(x).T if hi > lo else np.zeros((d.shape[0], x.shape[0])))
    return [np.stack(r) for r in res]


def swiglu(g, u):
    g, u = np.asarray(g, np.float64), np.asarray(u, np.float64)
    return g * scores(g, True) * u


def swiglu_backward(g, u, dh):
    """(dg, du)."""
    g, u, dh = (np.asarray(v, np.float64) for v in (g, u, dh))
    s, q = scores(g, True), scores(-g, True)
    return dh * u * s * (1.0 + g * q), dh * g * s
