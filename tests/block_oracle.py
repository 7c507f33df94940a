"""Plain 64-bit forms of a feed-forward block's operators, written from their definitions in
include/sgemm.h with numpy, and the magnitudes that the results' errors are measured against."""
from __future__ import annotations

import math

import numpy as np

F32, F64 = np.float32, np.float64
erf = np.vectorize(math.erf, otypes=[F64])
erfc = np.vectorize(math.erfc, otypes=[F64])
C = 2.0 * math.sqrt(2.0 / math.pi)


def logistic(u):
    e = np.exp(-np.abs(u))
    return np.where(u < 0, e / (1.0 + e), 1.0 / (1.0 + e))


def act(kind, g):
    """(the activation, what its error in 32 bits is measured against)."""
    g = np.asarray(g, F64)
    at = np.maximum(g, -1e300)  # the limit at -infinity
    with np.errstate(invalid="ignore", over="ignore"):
        if kind == 0:
            a = at * logistic(at)
            return a, np.abs(a)
        if kind == 1:
            a = 0.5 * at * erfc(-at / math.sqrt(2.0))
            # an argument off by 2^-23 moves erfc by up to g^2 + 1 of it
            return a, np.abs(a) * (2.0 + np.minimum(g * g, 1e4) * (g < 0))
        b = np.clip(at, -40.0, 40.0)
        u = C * (b + 0.044715 * b ** 3)
        a = at * logistic(u)
        return a, np.abs(a) * (1.0 + np.abs(u) * logistic(-u))


def slope(kind, g):
    """(the activation's derivative, its terms' magnitudes)."""
    g = np.asarray(g, F64)
    b = np.clip(g, -1e5, 1e5)
    if kind == 0:
        s, r = logistic(b), logistic(-b)
        return s * (1.0 + b * r), s * (1.0 + np.abs(b) * r)
    if kind == 1:
        phi = np.exp(-0.5 * b * b) / math.sqrt(2.0 * math.pi)
        return 0.5 * erfc(-b / math.sqrt(2.0)) + b * phi, 0.5 * erfc(-b / math.sqrt(2.0)) + np.abs(b) * phi * (1 + b * b)
    b = np.clip(g, -40.0, 40.0)
    u = C * (b + 0.044715 * b ** 3)
    s, r = logistic(u), logistic(-u)
    d = C * (1.0 + 0.134145 * b * b)
    return s + b * s * r * d, (s + np.abs(b) * s * r * d) * (1.0 + np.abs(u) * r)


def quantize(v):
    """(whole numbers, scales) of float32 rows."""
    v = np.asarray(v, F32)
    bits = v.view(np.uint32) & np.uint32(0x7fffffff)
    most = bits.max(1, initial=0).astype(np.uint32)
    finite = most < 0x7f800000
    top = np.where(finite, most, 0).astype(np.uint32).view(F32).astype(F64)
    per = 127.0 * np.divide(1.0, top, out=np.zeros_like(top), where=top > 0)
    q = np.where(finite[:, None], np.rint(np.where(finite[:, None], v, 0).astype(F64) * per[:, None]), 0)
    return q.astype(np.int8), np.where(finite, top / 127.0, np.nan).astype(F32)


def norm(x, residual, weight, eps):
    """(h rounded to 32 bits, y in 64 bits)."""
    with np.errstate(all="ignore"):
        h = np.asarray(x, F32) if residual is None else np.asarray(x, F32) + np.asarray(residual, F32)
        h64 = h.astype(F64)
        r = 1.0 / np.sqrt((h64 * h64).mean(1, keepdims=True) + F64(F32(eps))) if h.shape[1] else np.zeros((len(h), 1))
        y = h64 * r
        return h, y if weight is None else y * np.asarray(weight, F64)


def norm_grad(h, weight, eps, dy, dsum):
    """(dh, its terms' magnitudes, dweight, its)."""
    h, dy = np.asarray(h, F64), np.asarray(dy, F64)
    w = np.ones(h.shape[1]) if weight is None else np.asarray(weight, F64)
    r = 1.0 / np.sqrt((h * h).mean(1, keepdims=True) + F64(F32(eps)))
    g = dy * w
    back = h * r * r * (g * h).mean(1, keepdims=True)
    dh, size = r * (g - back), r * (np.abs(g) + np.abs(h) * r * r * np.abs(g * h).mean(1, keepdims=True))
    if dsum is not None:
        dh, size = dh + dsum, size + np.abs(dsum)
    return dh, size, (dy * h * r).sum(0), np.abs(dy * h * r).sum(0)


def i8(A, sa, B, sb, alpha, beta, C0):
    """(C, its terms' magnitudes)."""
    total = (A.astype(F64) @ B.astype(F64).T) * F64(F32(alpha))
    if sa is not None:
        total = total * np.asarray(sa, F64)[:, None]
    if sb is not None:
        total = total * np.asarray(sb, F64)[None, :]
    if beta == 0:
        return total, np.abs(total)
    old = F64(F32(beta)) * np.asarray(C0, F64)
    return total + old, np.abs(total) + np.abs(old)


def gated(kind, x, G, U):
    """(gate, its terms' magnitudes, up, its)."""
    x, G, U = (np.asarray(v, F64) for v in (x, G, U))
    return x @ G, np.abs(x) @ np.abs(G), x @ U, np.abs(x) @ np.abs(U)


def gated_grad(kind, x, G, U, gate, up, dy):
    """((dx, dG, dU), their terms' magnitudes)."""
    x, G, U, gate, up, dy = (np.asarray(v, F64) for v in (x, G, U, gate, up, dy))
    s, s_size = slope(kind, gate)
    a, a_size = act(kind, gate)
    dg, du = dy * up * s, dy * a
    dg_size, du_size = np.abs(dy * up) * s_size, np.abs(dy) * a_size
    xt = np.abs(x).T
    return ((dg @ G.T + du @ U.T, x.T @ dg, x.T @ du),
            (dg_size @ np.abs(G).T + du_size @ np.abs(U).T, xt @ dg_size, xt @ du_size))
