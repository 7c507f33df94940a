"""Plain 64-bit forms of the calls around products whose B is picked row by row, written from
their definitions in include/sgemm.h with numpy loops, and the magnitudes that the float32
results' errors are measured against."""
from __future__ import annotations

import math

import numpy as np


def scores(row, sigmoid):
    """The scores of one row of logits (float64), 0 for masked (-inf) and NaN entries."""
    live = row > -math.inf
    s = np.zeros(len(row))
    if not live.any():
        return s
    if sigmoid:
        s[live] = [1.0 / (1.0 + math.exp(-v)) if v > -700 else math.exp(v) for v in row[live]]
        return s
    m = row[live].max()
    e = np.array([1.0 if v == m else math.exp(v - m) for v in row[live]])
    s[live] = e / e.sum()
    return s


def route(logits, k, sigmoid=False, bias=None, groups=1, top_groups=1, best=1, renorm=False, scale=1.0):
    """ids (T x k) and weights (float64)."""
    T, E = logits.shape
    per = E // groups
    ids = np.full((T, k), -1, np.int32)
    weights = np.zeros((T, k))
    for t in range(T):
        row = logits[t].astype(np.float64)
        s = scores(row, sigmoid)
        if bias is None and not (groups > 1 and best == 2):
            key = row
        else:
            key = s + (0.0 if bias is None else bias.astype(np.float64))
        live = [e for e in range(E) if row[e] > -math.inf and key[e] > -math.inf]
        if groups > 1:
            worth = {}
            for g in range(groups):
                mine = sorted((key[e] for e in live if e // per == g), reverse=True)[:best]
                if mine:
                    worth[g] = sum(mine)
            kept = sorted(worth, key=lambda g: (-worth[g], g))[:top_groups]
            live = [e for e in live if e // per in kept]
        live.sort(key=lambda e: (-key[e], e))
        chosen = live[:k]
        if not chosen:
            continue
        ids[t, :len(chosen)] = chosen
        if renorm and not sigmoid:  # the softmax over the chosen alone
            w = scores(row[chosen], False)
        else:
            w = s[chosen]
            if renorm:
                w = w / w.sum() if w.sum() > 0 else np.zeros(len(w))
        weights[t, :len(chosen)] = math.nan if np.isnan(row).any() else w * scale
    return ids, weights


def route_grad(logits, ids, dweights, sigmoid=False, renorm=False, scale=1.0):
    """dlogits (float64), and per element the size of the terms it is made of."""
    T, E = logits.shape
    out, size = np.zeros((T, E)), np.zeros((T, E))
    for t in range(T):
        s = scores(logits[t].astype(np.float64), sigmoid)
        pick = [(int(i), float(d) * scale) for i, d in zip(ids[t], dweights[t]) if 0 <= i < E]
        if not pick:
            continue
        S = sum(s[i] for i, _ in pick)
        d = dict(pick)
        a = {i: abs(v) for i, v in pick}
        if renorm:
            if S == 0:
                continue
            mean = sum(v * s[i] for i, v in pick) / S
            amean = sum(abs(v) * s[i] for i, v in pick) / S
            d = {i: (v - mean) / S for i, v in pick}
            a = {i: (abs(v) + amean) / S for i, v in pick}
        q = 0.0 if sigmoid else sum(v * s[i] for i, v in d.items())
        aq = 0.0 if sigmoid else sum(v * s[i] for i, v in a.items())
        for e in range(E):
            f = s[e] * (1 - s[e]) if sigmoid else s[e]
            out[t, e] = f * (d.get(e, 0.0) - q)
            size[t, e] = f * (a.get(e, 0.0) + aq)
    return out, size


def group_rows(ids, G):
    flat = np.asarray(ids).reshape(-1)
    lists = [np.nonzero(flat == g)[0] for g in range(G)]
    offsets = np.concatenate([[0], np.cumsum([len(v) for v in lists])]).astype(np.int32)
    rows = np.concatenate(lists + [np.zeros(0, np.int64)]).astype(np.int32)
    return offsets, rows


def _at(rows, p, div):
    return p if div == 0 else int(rows[p]) // div


def grouped(offsets, rows, N, K, alpha, A, a_div, B, trans_b, beta, C, c_scatter):
    """C after the call and the size of its elements' terms (NaN where untouched)."""
    out, size = C.astype(np.float64), np.full(C.shape, np.nan)
    A, B = A.astype(np.float64), B.astype(np.float64)
    for g in range(len(offsets) - 1):
        b = B[g].T if trans_b else B[g]
        for p in range(offsets[g], offsets[g + 1]):
            a, c = _at(rows, p, a_div), _at(rows, p, 1 if c_scatter else 0)
            old = beta * out[c] if beta != 0 else 0.0
            out[c] = old + (alpha * (A[a] @ b) if alpha != 0 and K else 0.0)
            size[c] = abs(alpha) * (np.abs(A[a]) @ np.abs(b)) + np.abs(old)
    return out, size


def grouped_tn(offsets, rows, alpha, A, a_div, B, b_div, beta, C):
    out, size = np.zeros(C.shape), np.zeros(C.shape)
    A, B = A.astype(np.float64), B.astype(np.float64)
    for g in range(len(offsets) - 1):
        places = range(offsets[g], offsets[g + 1])
        a = A[[_at(rows, p, a_div) for p in places]]
        b = B[[_at(rows, p, b_div) for p in places]]
        old = beta * C[g].astype(np.float64) if beta != 0 else np.zeros(C[g].shape)
        out[g] = alpha * (a.T @ b) + old
        size[g] = abs(alpha) * (np.abs(a).T @ np.abs(b)) + np.abs(old)
    return out, size


def adapters(A, B, ids, ranks, scales, U, V, alpha, beta, C):
    A, B, U, V = (x.astype(np.float64) for x in (A, B, U, V))
    out = alpha * (A @ B) + (beta * C.astype(np.float64) if beta != 0 else 0.0)
    size = abs(alpha) * (np.abs(A) @ np.abs(B)) + (np.abs(beta * C.astype(np.float64)) if beta != 0 else 0.0)
    G = len(U)
    for m, g in enumerate(ids):
        if not 0 <= g < G:
            continue
        r = U.shape[2] if ranks is None else min(max(int(ranks[g]), 0), U.shape[2])
        s = alpha * (1.0 if scales is None else float(scales[g]))
        out[m] += s * ((A[m] @ U[g, :, :r]) @ V[g, :r])
        # two products one after the other: both round
        size[m] += 2 * abs(s) * ((np.abs(A[m]) @ np.abs(U[g, :, :r])) @ np.abs(V[g, :r]))
    return out, size


def adapters_grad(A, B, dC, ids, ranks, scales, U, V, alpha, beta, dU, dV):
    A, B, dC, U, V = (x.astype(np.float64) for x in (A, B, dC, U, V))
    ab = np.abs
    oa, sa = alpha * (dC @ B.T), abs(alpha) * (ab(dC) @ ab(B).T)
    ou = beta * dU.astype(np.float64) if beta != 0 else np.zeros(U.shape)
    ov = beta * dV.astype(np.float64) if beta != 0 else np.zeros(V.shape)
    su, sv = ab(ou), ab(ov)
    for g in range(len(U)):
        r = U.shape[2] if ranks is None else min(max(int(ranks[g]), 0), U.shape[2])
        m = np.nonzero(np.asarray(ids) == g)[0]
        s = alpha * (1.0 if scales is None else float(scales[g]))
        u, v = U[g, :, :r], V[g, :r]
        oa[m] += s * (dC[m] @ v.T) @ u.T
        sa[m] += 2 * abs(s) * (ab(dC[m]) @ ab(v).T) @ ab(u).T
        ou[g, :, :r] += s * A[m].T @ (dC[m] @ v.T)
        su[g, :, :r] += 2 * abs(s) * ab(A[m]).T @ (ab(dC[m]) @ ab(v).T)
        ov[g, :r] += s * (A[m] @ u).T @ dC[m]
        sv[g, :r] += 2 * abs(s) * (ab(A[m]) @ ab(u)).T @ ab(dC[m])
    return (oa, sa), (ou, su), (ov, sv)
