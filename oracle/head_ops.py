"""Plain float64 NumPy forms of the operators around the head (8-bit groups,
the final norm and its gradient).  Test infrastructure: written from the
definitions in ``include/cce.h``."""

from __future__ import annotations

import numpy as np

GROUP = 128
TINY = np.float32(2.0 ** -90)


def groups(n: int) -> int:
    return -(-n // GROUP)


def e4m3_round(v):
    """Nearest e4m3 value (ties to even), saturated at 448; float64."""
    v = np.asarray(v, np.float64)
    with np.errstate(all="ignore"):
        a = np.minimum(np.abs(v), 448.0)
        _, e = np.frexp(np.maximum(a, 2.0 ** -6))
        step = np.ldexp(1.0, e - 4)
        q = np.minimum(np.rint(a / step) * step, 448.0)
        return np.where(np.isnan(v), np.nan, np.copysign(q, v))


def _codes(x, m):
    """(values of the codes, scale) of x with group maxima m, the quotients and
    products rounded in fp32 as the format defines them."""
    with np.errstate(all="ignore"):
        inv = np.float32(448.0) * (np.float32(1.0) / m)
        return e4m3_round((x * inv).astype(np.float32)), m * (np.float32(1.0) / np.float32(448.0))


def _amax(x, axis):
    """Largest magnitude; NaN does not count."""
    a = np.where(np.isnan(x), np.float32(0), np.abs(x))
    return np.maximum(a.max(axis=axis, keepdims=True), TINY)


def quant_rows(x):
    """x float32 [M, D] -> code values float64 [M, D], scales float32 [M, G]."""
    x = np.asarray(x, np.float32)
    M, D = x.shape
    G = groups(D)
    p = np.zeros((M, G * GROUP), np.float32)
    p[:, :D] = x
    p = p.reshape(M, G, GROUP)
    q, s = _codes(p, _amax(p, 2))
    return q.reshape(M, -1)[:, :D], s[..., 0]


def quant_blocks(w):
    """w float32 [N, K] -> code values float64 [N, K], scales float32 [R, G]."""
    w = np.asarray(w, np.float32)
    N, K = w.shape
    R, G = groups(N), groups(K)
    p = np.zeros((R * GROUP, G * GROUP), np.float32)
    p[:N, :K] = w
    p = p.reshape(R, GROUP, G, GROUP)
    q, s = _codes(p, _amax(p, (1, 3)))
    return q.reshape(R * GROUP, -1)[:N, :K], s[:, 0, :, 0]


def rows_values(q, s):
    """Values of row-wise codes; float64."""
    return np.asarray(q, np.float64) * np.repeat(np.asarray(s, np.float64), GROUP, 1)[:, :q.shape[1]]


def blocks_values(q, s):
    big = np.repeat(np.repeat(np.asarray(s, np.float64), GROUP, 0), GROUP, 1)
    return np.asarray(q, np.float64) * big[:q.shape[0], :q.shape[1]]


def norm_forward(x, w, eps):
    """(H, rstd) in float64."""
    x = np.asarray(x, np.float64)
    rstd = 1.0 / np.sqrt((x * x).mean(1) + eps)
    return x * rstd[:, None] * np.asarray(w, np.float64), rstd


def norm_backward(n, rstd, w, dh):
    """(dX, dW) from the normalised rows n = x * rstd; float64."""
    g = dh * np.asarray(w, np.float64)
    dx = rstd[:, None] * (g - n * (g * n).mean(1, keepdims=True))
    return dx, (dh * n).sum(0)


def sample_row(logits, temperature, top_k, top_p, min_p, u):
    """(token, logp, ranked ids that stay) of one row; (-1, 0.0, []) for a row
    without live logits."""
    l = np.asarray(logits, np.float64)
    ids = np.flatnonzero(l > -np.inf)
    if ids.size == 0:
        return -1, 0.0, ids
    l = l[ids]
    top = l.max()
    with np.errstate(invalid="ignore", divide="ignore", over="ignore"):
        d = np.where(l == top, 0.0, l - top)
        order = np.argsort(-l, kind="stable")
        n = order.size
        if not temperature > 0:
            n, w = 1, np.ones(1)
        else:
            e = np.where(d[order] == 0, 0.0, d[order] / np.float64(temperature))
            w = np.exp(e)
            if top_k > 0:
                n = min(n, int(top_k))
            if top_p < 1:
                c = np.cumsum(w[:n])
                n = min(n, max(1, int((c < float(top_p) * c[-1]).sum()) + 1))
            if min_p > 0:
                n = min(n, max(1, int((w[:n] >= float(min_p)).sum())))
        c = np.cumsum(w[:n])
        u = min(max(float(u), 0.0), 1.0 - 2.0 ** -24)
        at = order[min(n - 1, int((c <= u * c[-1]).sum()))]
        logp = d[at] - np.log1p(np.exp(np.delete(d, int(np.argmax(l)))).sum())
    return int(ids[at]), float(logp), ids[order[:n]]
