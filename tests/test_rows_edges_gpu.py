"""Corners of the router, the slots sorted by group, the products over groups of rows and the
adapters that their parametrised tests do not reach, against forms written from the
definitions in include/sgemm.h.

A rounding to float32 is off by at most 2^-24 of the value, and results that are computed in 64
bits and rounded once are held to that (with 1% for what 64 bits lose)."""
import numpy as np
import pytest
import torch

import fp32_gemm_03_amd as g
from tests import gpu_util as gu
from tests import rows_oracle as ro
from tests.test_rows_gpu import U24, Buffer, call_route, router_logits, within

pytestmark = pytest.mark.gpu
ONCE = 1.01 * U24  # one rounding


@pytest.fixture(autouse=True)
def _gpu_available():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")


def sigmoid(x):
    return 1.0 / (1.0 + np.exp(-x.astype(np.float64)))


# ---------------------------------------------------------------------------
# router
# ---------------------------------------------------------------------------
@pytest.mark.parametrize("best", [1, 2])
@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
def test_route_order_with_one_group(score, best):
    """Without a bias, group_best 1 orders by the logits and group_best 2 by the 64-bit scores, in
    which saturated sigmoids and vanished softmax scores tie, to the lowest index."""
    gu.say("route order", score, best)
    if score == "sigmoid":
        x = np.array([[40, 41, 60, 1, 39], [-3, 50, 38, 45, 90], [0, 1, 2, 3, 4]], np.float32)
        s = sigmoid(x)
        assert s[0, 0] == s[0, 2] == 1.0
    else:
        x = np.array([[0, -800, -790, -760, -1], [-900, -800, 5, -850, -860], [0, 1, 2, 3, 4]], np.float32)
        e = np.exp(x.astype(np.float64) - x.max(1, keepdims=True))
        s = e / e.sum(1, keepdims=True)
        assert s[0, 1] == s[0, 2] == 0.0
    key = s if best == 2 else x.astype(np.float64)
    want = np.argsort(-key, axis=1, kind="stable")[:, :4]
    ids, w = call_route(x, 4, dict(sigmoid=score == "sigmoid", best=best))
    assert np.array_equal(ids, want)
    within(w, np.take_along_axis(s, want, 1), np.take_along_axis(s, want, 1), 64 * U24, "weights")


@pytest.mark.parametrize("E", [5, 16, 64, 250, 1024])
def test_route_softmax_weights_are_rounded_once(E):
    """Softmax weights that are not renormalised: the row's sum is held in 64 bits too."""
    T, k = 300, min(E, 8)
    gu.say("route softmax weights", E)
    x = (np.random.default_rng(E).standard_normal((T, E)) * 2).astype(np.float32)
    for scale in (1.0, 2.5):
        ids, w = call_route(x, k, dict(scale=scale))
        want_ids, want = ro.route(x, k, scale=scale)
        assert np.array_equal(ids, want_ids)
        within(w, want, np.abs(want), ONCE, "weights")


def confident_rows(E, seed):
    """Rows whose highest logit is 0 to 60 above the next, the rest spread below it; one of two
    equal highest logits, one with a masked half, one of -infinity."""
    r = np.random.default_rng(seed)
    gaps = [0.0, 0.5, 3.0, 8.0, 10.0, 14.0, 16.0, 17.0, 18.0, 20.0, 25.0, 30.0, 36.0, 40.0, 60.0]
    x = (-np.abs(r.standard_normal((len(gaps) + 3, E))) * 2).astype(np.float32)
    for t, gap in enumerate(gaps):
        x[t, r.integers(E)] = gap
    x[-3, :2] = 20.0
    x[-2, E // 2:] = -np.inf
    x[-2, 0] = 18.0
    x[-1] = -np.inf
    return x


@pytest.mark.parametrize("score,renorm", [("softmax", False), ("softmax", True), ("sigmoid", True), ("sigmoid", False)])
@pytest.mark.parametrize("E,k", [(2, 1), (9, 1), (9, 2), (64, 1), (64, 6), (200, 8), (40, 33)])
def test_route_grad_of_confident_rows(E, k, score, renorm):
    """dl_j = p_j sum_i p_i (c_j - c_i), over the row (c_i = 0 where not chosen) or with renorm
    over the chosen: no term of it cancels.  64 bits are off by at most 2^-40 of the terms (sums of
    200 terms, each with a difference that has up to 400 times their size), then one rounding."""
    gu.say("route_grad confident", E, k, score, renorm)
    x = confident_rows(E, E + k)
    T = len(x)
    r = np.random.default_rng([E, k])
    ids, _ = ro.route(x, k, sigmoid=score == "sigmoid")
    if E > 9:
        ids[3, 0] = ids[8, k - 1] = -1  # the highest is not among the chosen; one choice less
    dw = r.standard_normal((T, k)).astype(np.float32)
    if k > 1:
        dw[5] = dw[5, 0]  # one gradient for all: with renorm nothing is left
    scale = np.float32(2.5)
    out = Buffer(np.full((T, E), 7.0, np.float32))
    X, I, D = Buffer(x), Buffer(ids.reshape(-1)), Buffer(dw.reshape(-1))
    g.sgemm_route_grad(T, E, k, 1 if score == "sigmoid" else 0, X.ptr, X.ld, renorm, float(scale), I.ptr, D.ptr,
                       out.ptr, out.ld)
    torch.cuda.synchronize()
    want, size = np.zeros((T, E)), np.zeros((T, E))
    for t in range(T):
        c, chosen = np.zeros(E), np.zeros(E, bool)
        for i, v in zip(ids[t], dw[t]):
            if i >= 0:
                c[i], chosen[i] = float(v) * float(scale), True
        row = x[t].astype(np.float64)
        over = chosen if renorm else np.ones(E, bool)
        over = over & (row > -np.inf)
        if not over.any():
            continue
        if score == "sigmoid":
            s, rest = 1.0 / (1.0 + np.exp(-row)), 1.0 / (1.0 + np.exp(row))
            if not renorm:
                want[t] = c * s * rest
                continue
        else:
            s, rest = np.exp(row - row[over].max()), 1.0
        p = np.where(over, s, 0.0)
        p = p / p.sum()
        terms = p[:, None] * (c[:, None] - c[None, :]) * p[None, :]
        want[t], size[t] = terms.sum(1) * rest, np.abs(terms).sum(1) * rest
    got = out.read().astype(np.float64)
    assert (np.abs(got - want) <= ONCE * np.abs(want) + 2.0 ** -40 * size + 1e-37).all(), \
        np.max(np.abs(got - want) / (ONCE * np.abs(want) + 2.0 ** -40 * size + 1e-37))
    if score == "softmax":  # a row's gradient sums to 0, but for the roundings of its elements
        assert (np.abs(got.sum(1)) <= ONCE * np.abs(got).sum(1) + 1e-36).all()


# groups of more than four experts per lane of a row, on 16 lanes and on 64
LONG_GROUPS = [
    (9, 256, 8, dict(groups=2)), (9, 130, 5, dict(groups=2, best=2, bias=True)), (8, 255, 8, dict(groups=3, top_groups=2, best=2)),
    (9, 200, 6, dict(groups=2, bias=True, sigmoid=True, renorm=True)), (7, 1024, 8, dict(groups=2, best=2, bias=True)),
    (9, 520, 20, dict(groups=2)), (8, 1023, 64, dict(groups=3, top_groups=2, best=2, sigmoid=True)),
    (9, 600, 9, dict(groups=2, top_groups=2, bias=True)),
]


@pytest.mark.parametrize("case", LONG_GROUPS, ids=lambda c: f"{c[1]}in{c[3]['groups']}k{c[2]}")
@pytest.mark.parametrize("special", [False, True])
def test_route_long_groups(case, special):
    T, E, k, o = case
    gu.say("route long groups", case, special)
    x = router_logits(T, E, 20 + k, special)
    o = dict(o)
    bias = (np.random.default_rng(E).standard_normal(E) * 0.2).astype(np.float32) if o.pop("bias", False) else None
    ids, w = call_route(x, k, o, ldl=E + 1, bias_values=bias)
    want_ids, want = ro.route(x, k, bias=bias, **o)
    assert np.array_equal(ids, want_ids)
    within(w, want, np.abs(np.nan_to_num(want)), 2 * U24, "weights")


# ---------------------------------------------------------------------------
# slots sorted by group
# ---------------------------------------------------------------------------
@pytest.mark.parametrize("R,G", [((1 << 20) + 4097, 16), ((1 << 20) + 1, 1500), ((1 << 21) + 12345, 256), (3 << 20, 5)])
def test_group_rows_of_several_turns(R, G):
    """So many slots that a workgroup takes several runs of 4096 one after the other."""
    gu.say("group_rows several turns", R, G)
    r = np.random.default_rng([R, G])
    ids = (r.integers(0, G, R) * r.random(R) ** 2).astype(np.int32)  # low ones often
    ids[r.random(R) < 0.05] = -1
    ids[9000:30000] = G - 1
    I, off = Buffer(ids), Buffer(np.full(G + 1, -9, np.int32))
    rows = Buffer(np.full(R, -9, np.int32))
    need = g.sgemm_group_rows_workspace_size(R, G)
    ws = torch.full((need + 256,), 0xAB, dtype=torch.uint8, device="cuda")
    placed = np.nonzero(ids >= 0)[0]
    want = placed[np.argsort(ids[placed], kind="stable")]
    begins = np.concatenate([[0], np.cumsum(np.bincount(ids[placed], minlength=G))])
    for _ in range(2):
        g.sgemm_group_rows(R, G, I.ptr, off.ptr, rows.ptr, ws, need)
        torch.cuda.synchronize()
        assert np.array_equal(off.read(), begins)
        got = rows.read()
        assert np.array_equal(got[:len(want)], want) and (got[len(want):] == -9).all()
    assert (ws[need:] == 0xAB).all()


# ---------------------------------------------------------------------------
# products over groups of rows
# ---------------------------------------------------------------------------
@pytest.mark.parametrize("div", [10, 2 ** 31 - 10, 2 ** 31 - 1])
@pytest.mark.parametrize("trans", [False, True], ids=["nn", "nt"])
def test_grouped_one_row_for_all_slots(trans, div):
    """a_div (b_div) at and beyond R, up to the largest int: every slot takes row 0."""
    gu.say("grouped one row", trans, div)
    G, R, N, K = 2, 10, 40, 24
    r = np.random.default_rng(3)
    a, b = (r.uniform(-1, 1, s).astype(np.float32) for s in ((1, K), (G, N, K) if trans else (G, K, N)))
    offsets, rows = np.array([0, 4, 10], np.int32), r.permutation(R).astype(np.int32)
    A, B, C, off, rw = Buffer(a), Buffer(b), Buffer(np.full((R, N), np.nan, np.float32)), Buffer(offsets), Buffer(rows)
    g.sgemm_grouped(G, R, N, K, 1.0, A.ptr, K, div, B.ptr, B.ld, N * K, trans, 0.0, C.ptr, N, True, off.ptr, rw.ptr)
    torch.cuda.synchronize()
    want, size = ro.grouped(offsets, rows, N, K, 1.0, a, div, b, trans, 0.0, np.full((R, N), np.nan), True)
    within(C.read(), want, size, 1e-5, "C")
    y = r.uniform(-1, 1, (R, N)).astype(np.float32)
    Y = Buffer(y)
    for swap in (False, True):
        if swap:
            D = Buffer(np.full((G, N, K), np.nan, np.float32))
            g.sgemm_grouped_tn(G, R, N, K, 1.0, Y.ptr, N, 1, A.ptr, K, div, 0.0, D.ptr, K, N * K, off.ptr, rw.ptr)
            want, size = ro.grouped_tn(offsets, rows, 1.0, y, 1, a, div, 0.0, np.zeros((G, N, K)))
        else:
            D = Buffer(np.full((G, K, N), np.nan, np.float32))
            g.sgemm_grouped_tn(G, R, K, N, 1.0, A.ptr, K, div, Y.ptr, N, 1, 0.0, D.ptr, N, N * K, off.ptr, rw.ptr)
            want, size = ro.grouped_tn(offsets, rows, 1.0, a, div, y, 1, 0.0, np.zeros((G, K, N)))
        torch.cuda.synchronize()
        within(D.read(), want, size, 1e-5, "C")
