"""The router, the slots sorted by group, the products over groups of rows, the weighted sums
and the low-rank adapters against their 64-bit plain forms (rows_oracle), through the public
binding.

Tolerances.  Products follow the library's rule, an error of at most 1e-5 of the sum of the
terms' magnitudes (rows_oracle gives it; twice that for two products one after the other): a
float32 sum of n products is off by at most (n + 1) 2^-24 of it, and rounding errors of a sum
of thousands of random terms stay far below that bound.  The weighted sum of k slots is off by
at most (k + 1) 2^-24 of its terms' magnitudes.  Router weights are computed in 64 bits and
rounded once (2^-24), except that a softmax row's sum may be taken in float32: at most 32
additions and one exp of 2 ulp each, 64 * 2^-24.  Its gradient is the product of at most five
such factors, one of them that sum: 128 * 2^-24 of its terms."""
import numpy as np
import pytest
import torch

import fp32_gemm_03_amd as g
from tests import gpu_util as gu
from tests import rows_oracle as ro

pytestmark = pytest.mark.gpu
U24 = 2.0 ** -24
NAN = float("nan")


@pytest.fixture(autouse=True)
def _gpu_available():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")


class Buffer:
    """rows x cols float32 (or ints) with a leading dimension, in a guard band of NaN (or of
    -77), the columns beyond cols filled the same way."""

    def __init__(self, data, ld=None, offset=0, groups=None, stride=None):
        data = np.asarray(data)
        self.kind = torch.int32 if data.dtype.kind == "i" else torch.float32
        self.fill = -77 if self.kind is torch.int32 else NAN
        self.shape = data.shape
        if data.ndim == 1:
            idx = np.arange(data.size)
        else:
            rows, cols = data.shape[-2:]
            ld = cols if ld is None else ld
            idx = np.arange(rows)[:, None] * ld + np.arange(cols)[None, :]
            if data.ndim == 3:
                stride = rows * ld if stride is None else stride
                idx = np.arange(data.shape[0])[:, None, None] * stride + idx[None]
        self.ld, self.stride = ld, stride
        self.index = gu.GUARD + offset + idx
        n = (int(self.index.max()) + 1 if idx.size else gu.GUARD) + gu.GUARD
        host = torch.full((n,), self.fill, dtype=self.kind)
        host[torch.from_numpy(self.index.reshape(-1).astype(np.int64))] = torch.from_numpy(
            np.ascontiguousarray(data.reshape(-1))).to(self.kind)
        self.owner = host.cuda()
        self.ptr = self.owner.data_ptr() + 4 * (gu.GUARD + offset)

    def read(self):
        """The data, after a check that nothing around it was written."""
        host = self.owner.cpu().numpy()
        outside = np.ones(len(host), bool)
        outside[self.index.reshape(-1)] = False
        rest = host[outside]
        assert np.isnan(rest).all() if self.kind is torch.float32 else (rest == -77).all(), "written outside"
        return host[self.index]


def rng_of(*key):
    return np.random.default_rng([abs(hash(str(k))) % (1 << 31) if isinstance(k, str) else int(k) for k in key])


def within(got, want, size, tol, what=""):
    got = np.asarray(got, np.float64)
    assert got.shape == want.shape
    assert np.array_equal(np.isnan(got), np.isnan(want)), f"{what}: NaN where none belongs, or the reverse"
    ok = ~np.isnan(want)
    err = np.abs(got[ok] - want[ok])
    lim = tol * size[ok] + 1e-37
    assert (err <= lim).all(), f"{what}: {np.max(err / lim):.3g} of what is allowed"


# ---------------------------------------------------------------------------
# router
# ---------------------------------------------------------------------------
def router_logits(T, E, seed, special=True):
    r = rng_of(1, T, E, seed)
    x = (r.standard_normal((T, E)) * 2).astype(np.float32)
    x[r.random((T, E)) < 0.1] = -np.inf
    if special:
        for t in range(0, T, 7):
            x[t] = -np.inf                          # nothing left
        for t in range(1, T, 7):
            x[t] = np.round(x[t])                   # ties, and -0.0 next to 0.0
        for t in range(2, T, 7):
            x[t] = np.finfo(np.float32).min         # the type's lowest value is no mask
        for t in range(3, T, 14):
            x[t, ::3] = np.inf
        for t in range(4, T, 14):
            x[t, E // 2] = np.nan
        for t in range(5, T, 14):
            x[t] = x[t] * 40                        # scores that vanish in 32 bits
    return x


ROUTES = [
    # T, E, k, options
    (1, 1, 1, {}), (1, 64, 4, dict(renorm=True)), (5, 3, 3, dict(sigmoid=True)), (40, 16, 16, {}),
    (33, 17, 2, dict(renorm=True, scale=2.5)), (64, 60, 6, dict(sigmoid=True, renorm=True)),
    (29, 64, 6, dict(bias=True)), (31, 128, 8, dict(bias=True, renorm=True)),
    (30, 256, 8, dict(sigmoid=True, bias=True, groups=8, top_groups=4, best=2, renorm=True, scale=2.5)),
    (30, 100, 5, dict(groups=4, top_groups=2)), (30, 96, 4, dict(groups=3, top_groups=2, best=2)),
    (28, 62, 7, dict(groups=31, top_groups=9, best=2, bias=True)), (22, 300, 10, dict(groups=2, top_groups=1)),
    (17, 1000, 17, dict(bias=True, sigmoid=True)), (15, 1024, 64, dict(groups=64, top_groups=13, best=2)),
    (16, 40, 33, {}), (18, 8, 8, dict(groups=8, top_groups=3, renorm=True)), (257, 64, 2, dict(bias=True)),
]


def call_route(x, k, o, ldl=None, **kw):
    T, E = x.shape
    X = Buffer(x, ldl)
    bias = kw.pop("bias_values", None)
    b = None if bias is None else Buffer(bias)
    ids, w = Buffer(np.full(T * k, -5, np.int32)), Buffer(np.full(T * k, 9.0, np.float32))
    g.sgemm_route(T, E, k, 1 if o.get("sigmoid") else 0, X.ptr, X.ld, None if b is None else b.ptr,
                  o.get("groups", 1), o.get("top_groups", 1), o.get("best", 1), o.get("renorm", False),
                  o.get("scale", 1.0), ids.ptr, w.ptr, **kw)
    torch.cuda.synchronize()
    return ids.read().reshape(T, k), w.read().reshape(T, k)


@pytest.mark.parametrize("case", ROUTES, ids=lambda c: f"{c[0]}x{c[1]}k{c[2]}")
@pytest.mark.parametrize("special", [False, True])
def test_route(case, special):
    T, E, k, o = case
    gu.say("route", case, special)
    x = router_logits(T, E, k, special)
    o = dict(o)
    bias = None
    if o.pop("bias", False):
        bias = (rng_of(2, T, E).standard_normal(E) * 0.2).astype(np.float32)
        if E > 4:
            bias[1], bias[2] = -np.inf, 3.0
    ids, w = call_route(x, k, o, ldl=E + 3, bias_values=bias)
    want_ids, want = ro.route(x, k, bias=bias, **o)
    assert np.array_equal(ids, want_ids)
    within(w, want, np.abs(np.nan_to_num(want)), 64 * U24, "weights")
    if o.get("renorm") or o.get("sigmoid"):
        # 64 bits rounded once, then the scale's own rounding in the oracle's order
        within(w, want, np.abs(np.nan_to_num(want)), 2 * U24, "weights")


@pytest.mark.parametrize("case", ROUTES, ids=lambda c: f"{c[0]}x{c[1]}k{c[2]}")
def test_route_grad(case):
    T, E, k, o = case
    gu.say("route_grad", case)
    o = {n: o[n] for n in ("sigmoid", "renorm", "scale") if n in o}
    x = router_logits(T, E, k, False)
    if T > 2:
        x[1] = -np.inf
    r = rng_of(3, T, E, k)
    ids = np.stack([r.permutation(E)[:k] for _ in range(T)]).astype(np.int32)
    ids[r.random((T, k)) < 0.1] = -1
    if T > 4:
        ids[2], ids[3, 0] = -1, E + 5
    # masked experts are never chosen
    ids[np.take_along_axis(x, np.clip(ids, 0, E - 1).astype(np.int64), 1) == -np.inf] = -1
    dw = r.standard_normal((T, k)).astype(np.float32)
    dw[ids < 0] = np.nan  # not read
    X, I, D = Buffer(x, E + 1), Buffer(ids.reshape(-1)), Buffer(dw.reshape(-1))
    out = Buffer(np.full((T, E), 7.0, np.float32), E + 2)
    g.sgemm_route_grad(T, E, k, 1 if o.get("sigmoid") else 0, X.ptr, X.ld, o.get("renorm", False),
                       o.get("scale", 1.0), I.ptr, D.ptr, out.ptr, out.ld)
    torch.cuda.synchronize()
    want, size = ro.route_grad(x, np.where(ids >= E, -1, ids), np.nan_to_num(dw), **o)
    within(out.read(), want, size, 128 * U24, "dlogits")


# ---------------------------------------------------------------------------
# slots sorted by group
# ---------------------------------------------------------------------------
@pytest.mark.parametrize("G", [1, 2, 7, 64, 1000, 1025, 4096])
@pytest.mark.parametrize("R", [0, 1, 63, 64, 65, 511, 513, 4096, 4097, 20001])
def test_group_rows(R, G):
    gu.say("group_rows", R, G)
    r = rng_of(4, R, G)
    ids = r.integers(0, G, R).astype(np.int32)
    if R > 3:
        ids[r.random(R) < 0.1] = -1
        ids[R // 2], ids[R // 3] = G, 1 << 30
    if G > 3:
        ids[ids == 2] = 1  # an empty group
    I, off, rows = Buffer(ids), Buffer(np.full(G + 1, -9, np.int32)), Buffer(np.full(R, -9, np.int32))
    need = g.sgemm_group_rows_workspace_size(R, G)
    ws = torch.full((need + 256,), 0xAB, dtype=torch.uint8, device="cuda")
    want_off, want_rows = ro.group_rows(ids, G)
    for _ in range(2):
        g.sgemm_group_rows(R, G, I.ptr, off.ptr, rows.ptr, ws, need)
        torch.cuda.synchronize()
        assert np.array_equal(off.read(), want_off)
        got = rows.read()
        assert np.array_equal(got[:len(want_rows)], want_rows)
        assert (got[len(want_rows):] == -9).all()  # left as they were
    assert (ws[need:] == 0xAB).all()


def test_group_rows_all_in_one_group_and_none():
    for value in (3, -1):
        R, G = 9000, 5
        ids = torch.full((R,), value, dtype=torch.int32, device="cuda")
        off, rows = (torch.full((n,), -9, dtype=torch.int32, device="cuda") for n in (G + 1, R))
        ws = torch.empty(g.sgemm_group_rows_workspace_size(R, G), dtype=torch.uint8, device="cuda")
        g.sgemm_group_rows(R, G, ids, off, rows, ws)
        if value == 3:
            assert off.tolist() == [0, 0, 0, 0, R, R] and torch.equal(rows.cpu(), torch.arange(R, dtype=torch.int32))
        else:
            assert off.tolist() == [0] * 6 and (rows == -9).all()


# ---------------------------------------------------------------------------
# products over groups of rows
# ---------------------------------------------------------------------------
def sizes_to_ids(sizes, extra, seed):
    """Slot ids with the given number of rows per group, shuffled, and `extra` placed nowhere."""
    ids = np.concatenate([np.full(n, i, np.int32) for i, n in enumerate(sizes)] + [np.full(extra, -1, np.int32)])
    rng_of(5, seed, len(ids)).shuffle(ids)
    return ids


GROUPED = [
    # rows per group, slots of none, N, K
    ([1], 0, 1, 1), ([0, 1, 0], 2, 5, 3), ([2, 0, 3], 1, 33, 17), ([1, 1, 1, 1], 0, 64, 64),
    ([16, 15, 17, 0], 3, 65, 63), ([31, 33], 0, 130, 40), ([64, 3, 0, 65], 5, 127, 129),
    ([130, 5], 1, 200, 96), ([7] * 70, 4, 36, 20), ([300, 0, 257], 2, 257, 132), ([1, 40, 2], 0, 96, 1030),
    ([5, 9], 0, 515, 260), ([128, 128], 0, 128, 128), ([600], 9, 140, 68),
    ([3, 2], 1, 1024, 16), ([2] * 9, 0, 17, 2050),
]
MODES = [(1, 1), (0, 0), (3, 1), (1, 0), (0, 1)]


def grouped_case(sizes, extra, N, K, a_div, c_scatter, seed=0):
    r = rng_of(6, N, K, seed)
    ids = sizes_to_ids(sizes, extra, N * 7 + K)
    R, G = len(ids), len(sizes)
    offsets, rows = ro.group_rows(ids, G)
    rows = np.concatenate([rows, np.full(R - len(rows), -1, np.int32)])
    ar = R if a_div <= 1 else -(-R // a_div)
    f = lambda *s: r.uniform(-1, 1, s).astype(np.float32)  # noqa: E731
    return R, G, offsets, rows, ar, f


@pytest.mark.parametrize("mode", MODES, ids=lambda m: f"div{m[0]}s{m[1]}")
@pytest.mark.parametrize("trans", [False, True], ids=["nn", "nt"])
@pytest.mark.parametrize("case", GROUPED, ids=lambda c: f"{len(c[0])}g{sum(c[0])}r{c[2]}x{c[3]}")
def test_grouped(case, trans, mode):
    sizes, extra, N, K = case
    a_div, scatter = mode
    gu.say("grouped", case, trans, mode)
    R, G, offsets, rows, ar, f = grouped_case(sizes, extra, N, K, a_div, scatter)
    a, c0 = f(ar, K), f(R, N)
    b = f(G, N, K) if trans else f(G, K, N)
    variants = [(1.0, 0.0, 0, 0, 0)] if mode != (1, 1) else [(1.0, 0.0, 0, 0, 0), (1.5, -0.5, 3, 1, 2), (-0.75, 1.0, 4, 0, 0)]
    for alpha, beta, pad, mis, extra_ld in variants:
        A, B = Buffer(a, K + pad, mis), Buffer(b, b.shape[2] + pad + extra_ld, mis, stride=b.shape[1] * (b.shape[2] + pad + extra_ld) + 7 * pad)
        C = Buffer(c0 if beta != 0 else np.full_like(c0, np.nan), N + pad, mis)
        if beta == 0:  # untouched rows keep what they hold
            want0 = np.full_like(c0, np.nan)
        off, rw = Buffer(offsets), Buffer(rows)
        g.sgemm_grouped(G, R, N, K, alpha, A.ptr, A.ld, a_div, B.ptr, B.ld, B.stride, trans, beta, C.ptr, C.ld,
                        scatter, off.ptr, rw.ptr)
        torch.cuda.synchronize()
        want, size = ro.grouped(offsets, rows, N, K, alpha, a, a_div, b, trans, beta, c0 if beta != 0 else want0, scatter)
        got = C.read()
        touched = ~np.isnan(size)
        assert np.array_equal(got[~touched], (c0 if beta != 0 else want0)[~touched], equal_nan=True)
        within(got[touched], want[touched], size[touched], 1e-5, "C")


@pytest.mark.parametrize("divs", [(0, 0), (1, 1), (2, 1), (1, 3), (0, 1)])
@pytest.mark.parametrize("case", GROUPED, ids=lambda c: f"{len(c[0])}g{sum(c[0])}r{c[2]}x{c[3]}")
def test_grouped_tn(case, divs):
    sizes, extra, N, M = case
    gu.say("grouped_tn", case, divs)
    R, G, offsets, rows, _, f = grouped_case(sizes, extra, N, M, 1, 1, 1)
    n_rows = lambda d: R if d <= 1 else -(-R // d)  # noqa: E731
    a, b, c0 = f(n_rows(divs[0]), M), f(n_rows(divs[1]), N), f(G, M, N)
    variants = [(1.0, 0.0, 0, 0)] if divs != (1, 1) else [(1.0, 0.0, 0, 0), (-1.5, 0.5, 3, 1), (0.5, 1.0, 4, 0)]
    for alpha, beta, pad, mis in variants:
        A, B = Buffer(a, M + pad, mis), Buffer(b, N + pad, mis)
        C = Buffer(c0 if beta != 0 else np.full_like(c0, np.nan), N + pad, mis, stride=M * (N + pad) + 5 * pad)
        off, rw = Buffer(offsets), Buffer(rows)
        g.sgemm_grouped_tn(G, R, M, N, alpha, A.ptr, A.ld, divs[0], B.ptr, B.ld, divs[1], beta, C.ptr, C.ld, C.stride,
                           off.ptr, rw.ptr)
        torch.cuda.synchronize()
        want, size = ro.grouped_tn(offsets, rows, alpha, a, divs[0], b, divs[1], beta, c0)
        within(C.read(), want, size, 1e-5, "C")


# tiles of every form the sums of outer products take: rows per group, M, N
OUTER = [
    ([1, 0, 3] * 43, 260, 300), ([90] * 7, 390, 321),  # 64 x 64 on one wave, on four
    ([40] * 9, 1000, 61), ([40] * 9, 61, 1000), ([300, 0] * 6, 643, 16), ([17] * 14, 7, 701),  # 64 x 16 on four
    ([1100], 1027, 250), ([1300, 700], 250, 515), ([0, 1600, 2], 64, 900),  # 64 x 16 on eight
    ([1, 50, 333], 130, 33), ([33, 2], 20, 515), ([700], 900, 3), ([0, 0], 70, 5),  # 32 x 16
    ([900], 33, 200), ([5, 0, 261], 65, 64), ([256], 100, 100),  # 16 x 16
]


@pytest.mark.parametrize("case", OUTER, ids=lambda c: f"{len(c[0])}g{sum(c[0])}r{c[1]}x{c[2]}")
def test_grouped_tn_tiles(case):
    sizes, M, N = case
    gu.say("grouped_tn tiles", case)
    R, G, offsets, rows, _, f = grouped_case(sizes, 3, N, M, 1, 1, 3)
    a, b, c0 = f(R, M), f(-(-R // 2), N), f(G, M, N)
    off, rw = Buffer(offsets), Buffer(rows)
    for alpha, beta, pad, mis in ((1.0, 0.0, 0, 0), (-1.5, 0.5, 3, 1)):
        A, B = Buffer(a, M + pad, mis), Buffer(b, N + pad, mis)
        C = Buffer(c0 if beta != 0 else np.full_like(c0, np.nan), N + pad, mis, stride=M * (N + pad) + 5 * pad)
        g.sgemm_grouped_tn(G, R, M, N, alpha, A.ptr, A.ld, 1, B.ptr, B.ld, 2, beta, C.ptr, C.ld, C.stride, off.ptr, rw.ptr)
        torch.cuda.synchronize()
        want, size = ro.grouped_tn(offsets, rows, alpha, a, 1, b, 2, beta, c0)
        within(C.read(), want, size, 1e-5, "C")


# and those of the products: rows per group, N, K
TILES = [
    ([33, 0, 50], 16, 400), ([200, 17], 40, 130), ([5] * 12, 64, 300),  # 16 x 16, 16 x 32
    ([2600, 1700], 16, 70), ([1500, 900], 64, 90),  # more of them, 32 x 32
    ([90, 0, 70] * 7, 700, 66), ([20] * 40, 450, 100), ([700] * 3, 1500, 80),  # 32 x 64, 64 rows
    ([9000, 200], 13, 70), ([8000, 500], 31, 70), ([16500, 90], 40, 70),  # many rows, few columns
]


@pytest.mark.parametrize("trans", [False, True], ids=["nn", "nt"])
@pytest.mark.parametrize("case", TILES, ids=lambda c: f"{len(c[0])}g{sum(c[0])}r{c[1]}x{c[2]}")
def test_grouped_tiles(case, trans):
    sizes, N, K = case
    gu.say("grouped tiles", case, trans)
    R, G, offsets, rows, ar, f = grouped_case(sizes, 2, N, K, 2, 1, 4)
    a, b, c0 = f(-(-R // 2), K), f(G, N, K) if trans else f(G, K, N), f(R, N)
    off, rw = Buffer(offsets), Buffer(rows)
    for alpha, beta, pad, mis in ((1.0, 1.0, 0, 0), (-1.5, 0.5, 3, 1)):
        A, B, C = Buffer(a, K + pad, mis), Buffer(b, b.shape[2] + pad, mis, stride=b.shape[1] * (b.shape[2] + pad) + pad), Buffer(c0, N + pad, mis)
        g.sgemm_grouped(G, R, N, K, alpha, A.ptr, A.ld, 2, B.ptr, B.ld, B.stride, trans, beta, C.ptr, C.ld, True, off.ptr, rw.ptr)
        torch.cuda.synchronize()
        want, size = ro.grouped(offsets, rows, N, K, alpha, a, 2, b, trans, beta, c0, True)
        got, touched = C.read(), ~np.isnan(size)
        assert np.array_equal(got[~touched], c0[~touched])
        within(got[touched], want[touched], size[touched], 1e-5, "C")


def test_grouped_without_a_product():
    """alpha 0 or K 0: C = beta C for the placed rows, A and B not read."""
    for K, alpha in ((0, 1.0), (4, 0.0)):
        offsets, rows = np.array([0, 1, 3], np.int32), np.array([4, 0, 2, -1, -1], np.int32)
        c = rng_of(8).uniform(-1, 1, (5, 6)).astype(np.float32)
        C, off, rw = Buffer(c, 7), Buffer(offsets), Buffer(rows)
        g.sgemm_grouped(2, 5, 6, K, alpha, 0, 4, 1, 0, 6, 0, False, 0.5, C.ptr, 7, True, off.ptr, rw.ptr)
        torch.cuda.synchronize()
        want = c.copy()
        want[[4, 0, 2]] *= np.float32(0.5)
        assert np.array_equal(C.read(), want)
        g.sgemm_grouped(2, 5, 6, K, alpha, 0, 4, 1, 0, 6, 0, True, 0.0, C.ptr, 7, False, off.ptr, rw.ptr)
        torch.cuda.synchronize()
        want[:3] = 0
        assert np.array_equal(C.read(), want)
    d = rng_of(9).uniform(-1, 1, (2, 5, 6)).astype(np.float32)
    D = Buffer(d, 8)
    g.sgemm_grouped_tn(2, 5, 5, 6, 0.0, 0, 5, 1, 0, 6, 1, 2.0, D.ptr, 8, D.stride, 0, 0)
    torch.cuda.synchronize()
    assert np.array_equal(D.read(), 2 * d)


def test_grouped_skips_values_outside_and_takes_offsets_within():
    """Offsets beyond R and rows outside [0, R) are taken as the documentation says."""
    R, N, K = 6, 40, 24
    r = rng_of(10)
    a, b = (r.uniform(-1, 1, s).astype(np.float32) for s in ((R, K), (2, K, N)))
    A, B, C = Buffer(a), Buffer(b), Buffer(np.full((R, N), 3.0, np.float32))
    off, rw = Buffer(np.array([-4, 3, 99], np.int32)), Buffer(np.array([5, -1, 0, 7, 2, 1 << 30], np.int32))
    g.sgemm_grouped(2, R, N, K, 1.0, A.ptr, K, 1, B.ptr, N, K * N, False, 0.0, C.ptr, N, True, off.ptr, rw.ptr)
    torch.cuda.synchronize()
    got = C.read()
    for s, e in ((5, 0), (0, 0), (2, 1)):
        within(got[s], a[s].astype(np.float64) @ b[e], np.abs(a[s]) @ np.abs(b[e]), 1e-5)
    assert (got[[1, 3, 4]] == 3.0).all()
    D = Buffer(np.full((2, K, N), np.nan, np.float32))
    y = r.uniform(-1, 1, (R, N)).astype(np.float32)
    Y = Buffer(y)
    g.sgemm_grouped_tn(2, R, K, N, 1.0, A.ptr, K, 1, Y.ptr, N, 1, 0.0, D.ptr, N, K * N, off.ptr, rw.ptr)
    torch.cuda.synchronize()
    got = D.read()
    for e, slots in ((0, [5, 0]), (1, [2])):
        within(got[e], a[slots].astype(np.float64).T @ y[slots], np.abs(a[slots]).T @ np.abs(y[slots]), 1e-5)


@pytest.mark.parametrize("R", [6, 500])
@pytest.mark.parametrize("trans", [False, True], ids=["nn", "nt"])
@pytest.mark.parametrize("a_div,scatter", [(1, 0), (2, 0), (2, 1), (0, 1), (0, 0)])
def test_grouped_leaves_out_a_place_without_a_slot(a_div, scatter, trans, R):
    """Places in order whose slot is outside [0, R): C's row is left as it was, unless no slot is asked for."""
    N, K = 40, 100
    gu.say("grouped without a slot", a_div, scatter, trans, R)
    r = rng_of(16, R)
    a = r.uniform(-1, 1, (-(-R // a_div) if a_div else R, K)).astype(np.float32)
    b = r.uniform(-1, 1, (2, N, K) if trans else (2, K, N)).astype(np.float32)
    rows = r.permutation(R).astype(np.int32)
    rows[[1, R // 2]] = -3, R
    offsets = np.array([0, R // 3, R], np.int32)
    A, B, C = Buffer(a), Buffer(b), Buffer(np.full((R, N), 3.0, np.float32))
    off, rw = Buffer(offsets), Buffer(rows)
    g.sgemm_grouped(2, R, N, K, 1.0, A.ptr, K, a_div, B.ptr, b.shape[2], N * K, trans, 0.5, C.ptr, N, scatter, off.ptr, rw.ptr)
    torch.cuda.synchronize()
    want, size = np.full((R, N), 3.0), np.full((R, N), 3.0)
    for p in range(R):
        if (a_div or scatter) and not 0 <= rows[p] < R:
            continue
        x = a[rows[p] // a_div if a_div else p].astype(np.float64)
        e = b[0 if p < offsets[1] else 1].astype(np.float64)
        c = rows[p] if scatter else p
        want[c] = x @ (e.T if trans else e) + 1.5
        size[c] = np.abs(x) @ np.abs(e.T if trans else e) + 1.5
    within(C.read(), want, size, 1e-5, "C")


@pytest.mark.parametrize("trans", [False, True], ids=["nn", "nt"])
def test_grouped_rows_beyond_4_gib(trans):
    """Rows 1.5 GiB apart: offsets beyond 32 bits in A and in C, gathered and scattered."""
    R, N, K, G = 4, 40, 36, 2
    ld = 3 << 27
    gu.say("grouped beyond 4 GiB", trans)
    big = torch.empty(3 * ld + 64, dtype=torch.float32, device="cuda")
    r = rng_of(11)
    a = r.uniform(-1, 1, (R, K)).astype(np.float32)
    b = r.uniform(-1, 1, (G, N, K) if trans else (G, K, N)).astype(np.float32)
    for i in range(R):
        big[i * ld:i * ld + K] = torch.from_numpy(a[i])
    B = Buffer(b)
    offsets, rows = np.array([0, 3, 4], np.int32), np.array([0, 2, 3, 1], np.int32)
    off, rw = Buffer(offsets), Buffer(rows)
    for a_div, scatter in ((1, 1), (0, 0)):
        C = Buffer(np.full((R, N), np.nan, np.float32))
        g.sgemm_grouped(G, R, N, K, 1.0, big, ld, a_div, B.ptr, B.ld, N * K, trans, 0.0, C.ptr, N, scatter, off.ptr, rw.ptr)
        torch.cuda.synchronize()
        want, size = ro.grouped(offsets, rows, N, K, 1.0, a, a_div, b, trans, 0.0, np.full((R, N), np.nan), scatter)
        within(C.read(), want, size, 1e-5)
    D = Buffer(np.full((G, K, N), np.nan, np.float32))
    y = r.uniform(-1, 1, (R, N)).astype(np.float32)
    Y = Buffer(y)
    g.sgemm_grouped_tn(G, R, K, N, 1.0, big, ld, 1, Y.ptr, N, 1, 0.0, D.ptr, N, K * N, off.ptr, rw.ptr)
    torch.cuda.synchronize()
    want, size = ro.grouped_tn(offsets, rows, 1.0, a, 1, y, 1, 0.0, np.zeros((G, K, N)))
    within(D.read(), want, size, 1e-5)
    A = Buffer(a)
    g.sgemm_grouped(G, R, N, K, 1.0, A.ptr, K, 1, B.ptr, B.ld, N * K, trans, 0.0, big, ld, True, off.ptr, rw.ptr)
    torch.cuda.synchronize()
    got = np.stack([big[i * ld:i * ld + N].cpu().numpy() for i in range(R)])
    want, size = ro.grouped(offsets, rows, N, K, 1.0, a, 1, b, trans, 0.0, np.full((R, N), np.nan), 1)
    within(got, want, size, 1e-5)


# ---------------------------------------------------------------------------
# weighted sums
# ---------------------------------------------------------------------------
@pytest.mark.parametrize("beta", [0.0, -0.5])
@pytest.mark.parametrize("T,k,N", [(1, 1, 1), (3, 2, 5), (7, 4, 256), (5, 6, 257), (2, 9, 1027), (33, 3, 63), (4, 64, 30)])
def test_combine(T, k, N, beta):
    gu.say("combine", T, k, N, beta)
    r = rng_of(12, T, k, N)
    E = 5
    ids = r.integers(-1, E + 1, (T, k)).astype(np.int32)
    ids[0] = -1
    w = r.uniform(-1, 1, (T, k)).astype(np.float32)
    y, o = (r.uniform(-1, 1, s).astype(np.float32) for s in ((T * k, N), (T, N)))
    there = (ids >= 0) & (ids < E)
    y[~there.reshape(-1)] = np.nan  # not read
    I, W, Y = Buffer(ids.reshape(-1)), Buffer(w.reshape(-1)), Buffer(y, N + 1, 1)
    ref_y = np.nan_to_num(y).reshape(T, k, N).astype(np.float64)
    for weights in (W, None):
        O = Buffer(o if beta else np.full_like(o, np.nan), N + 2, 2)
        g.sgemm_combine(T, k, N, E, I.ptr, None if weights is None else W.ptr, Y.ptr, Y.ld, beta, O.ptr, O.ld)
        torch.cuda.synchronize()
        f = np.where(there, w if weights is not None else 1.0, 0.0)[:, :, None].astype(np.float64)
        want = (f * ref_y).sum(1) + beta * o
        within(O.read(), want, (np.abs(f) * np.abs(ref_y)).sum(1) + abs(beta) * np.abs(o), (k + 2) * U24)
    D = r.uniform(-1, 1, (T, N)).astype(np.float32)
    dout, dY = Buffer(D, N + 3, 1), Buffer(np.full((T * k, N), np.nan, np.float32), N + 1, 3)
    dw = Buffer(np.full(T * k, np.nan, np.float32))
    g.sgemm_combine_grad(T, k, N, E, I.ptr, W.ptr, dout.ptr, dout.ld, Y.ptr, Y.ld, dY.ptr, dY.ld, dw.ptr)
    torch.cuda.synchronize()
    want = np.where(there, w, 0)[:, :, None] * D[:, None, :]  # one float32 product: exact
    assert np.array_equal(dY.read().reshape(T, k, N), want)
    dots = (ref_y * D[:, None, :]).sum(2) * there
    within(dw.read().reshape(T, k), dots, (np.abs(ref_y) * np.abs(D[:, None, :])).sum(2), 1e-5)
    before = dw.read()
    g.sgemm_combine_grad(T, k, N, E, I.ptr, None, dout.ptr, dout.ld, None, Y.ld, dY.ptr, dY.ld, None)
    torch.cuda.synchronize()
    assert np.array_equal(dY.read().reshape(T, k, N), there[:, :, None] * D[:, None, :])
    g.sgemm_combine_grad(T, k, N, E, None, None, dout.ptr, dout.ld, Buffer(np.nan_to_num(y)).ptr, N, None, N, dw.ptr)
    torch.cuda.synchronize()
    assert np.array_equal(dw.read()[there.reshape(-1)], before[there.reshape(-1)])


# ---------------------------------------------------------------------------
# adapters
# ---------------------------------------------------------------------------
ADAPTERS = [
    # M, N, K, G, rank
    (1, 1, 1, 1, 1), (1, 64, 32, 3, 4), (1, 257, 130, 2, 16), (3, 33, 65, 5, 7), (16, 100, 96, 16, 8),
    (17, 63, 64, 2, 3), (29, 255, 200, 32, 64), (40, 130, 70, 4, 33), (64, 96, 128, 1, 16), (70, 65, 33, 6, 256),
    (150, 140, 132, 7, 16), (300, 68, 257, 3, 24), (8, 2060, 40, 4, 5), (5, 40, 2100, 3, 12), (260, 300, 64, 200, 8),
    (64, 33, 700, 64, 40), (65, 200, 4100, 1, 20), (200, 190, 4100, 2, 9), (640, 100, 90, 1, 96), (33, 16500, 48, 9, 50),
]


def adapter_inputs(M, N, K, G, rank, full):
    r = rng_of(13, M, N, K, G, rank)
    f = lambda *s: r.uniform(-1, 1, s).astype(np.float32)  # noqa: E731
    ids = r.integers(0, G, M).astype(np.int32)
    if M > 4:
        ids[1], ids[M // 2] = -1, G
    ranks = None if full else r.integers(0, rank + 1, G).astype(np.int32)
    if ranks is not None and G > 2:
        ranks[0], ranks[1] = rank + 9, -3
    scales = None if full else f(G)
    U, V = f(G, K, rank), f(G, rank, N)
    u, v = U.copy(), V.copy()
    if ranks is not None:  # what lies beyond a rank is not used
        for i in range(G):
            n = min(max(int(ranks[i]), 0), rank)
            U[i, :, n:], V[i, n:] = np.nan, np.nan
            u[i, :, n:], v[i, n:] = 0, 0
    return f, ids, ranks, scales, (U, u), (V, v)


@pytest.mark.parametrize("full", [True, False], ids=["full", "ranks"])
@pytest.mark.parametrize("case", ADAPTERS, ids=lambda c: "x".join(map(str, c)))
def test_adapters(case, full):
    M, N, K, G, rank = case
    gu.say("adapters", case, full)
    f, ids, ranks, scales, (U, u), (V, v) = adapter_inputs(M, N, K, G, rank, full)
    a, b, c0 = f(M, K), f(K, N), f(M, N)
    need = g.sgemm_adapters_workspace_size(M, N, K, G, rank)
    ws = torch.full((need + 256,), 0xFF, dtype=torch.uint8, device="cuda")
    for alpha, beta, pad, mis in ((1.0, 0.0, 0, 0), (-1.5, 0.5, 1, 1), (0.5, 1.0, 4, 0)):
        A, B = Buffer(a, K + pad, mis), Buffer(b, N + pad, mis)
        C = Buffer(c0 if beta else np.full_like(c0, np.nan), N + pad, mis)
        UB, VB = Buffer(U, rank + pad, mis), Buffer(V, N + 2 * pad, mis)
        I = Buffer(ids)
        R = None if ranks is None else Buffer(ranks)
        S = None if scales is None else Buffer(scales)
        g.sgemm_adapters(M, N, K, alpha, A.ptr, A.ld, B.ptr, B.ld, beta, C.ptr, C.ld, G, rank, I.ptr,
                         R and R.ptr, S and S.ptr, UB.ptr, UB.ld, UB.stride, VB.ptr, VB.ld, VB.stride, ws, need)
        torch.cuda.synchronize()
        want, size = ro.adapters(a, b, ids, ranks, scales, u, v, alpha, beta, c0)
        within(C.read(), want, size, 1e-5, "C")
        assert (ws[need:] == 0xFF).all()


@pytest.mark.parametrize("full", [True, False], ids=["full", "ranks"])
@pytest.mark.parametrize("case", ADAPTERS, ids=lambda c: "x".join(map(str, c)))
def test_adapters_grad(case, full):
    M, N, K, G, rank = case
    gu.say("adapters_grad", case, full)
    f, ids, ranks, scales, (U, u), (V, v) = adapter_inputs(M, N, K, G, rank, full)
    a, b, dc, du0, dv0 = f(M, K), f(K, N), f(M, N), f(G, K, rank), f(G, rank, N)
    need = g.sgemm_adapters_grad_workspace_size(M, N, K, G, rank)
    ws = torch.full((need + 256,), 0xFF, dtype=torch.uint8, device="cuda")
    for alpha, beta, pad, mis, wanted in ((1.0, 0.0, 0, 0, "both"), (-1.5, 0.5, 1, 1, "both"),
                                          (1.0, 0.0, 0, 0, "rows"), (1.0, 0.0, 0, 0, "adapters")):
        A, B, D = Buffer(a, K + pad, mis), Buffer(b, N + pad, mis), Buffer(dc, N + 3 * pad, mis)
        UB, VB = Buffer(U, rank + pad, mis), Buffer(V, N + 2 * pad, mis)
        fresh = lambda x: x if beta else np.full_like(x, np.nan)  # noqa: E731
        dA = Buffer(np.full((M, K), np.nan, np.float32), K + pad, mis)
        dU, dV = Buffer(fresh(du0), rank + pad, mis), Buffer(fresh(dv0), N + pad, mis)
        I = Buffer(ids)
        R = None if ranks is None else Buffer(ranks)
        S = None if scales is None else Buffer(scales)
        on = wanted != "rows"
        g.sgemm_adapters_grad(M, N, K, alpha, A.ptr, A.ld, B.ptr, B.ld, D.ptr, D.ld, G, rank, I.ptr, R and R.ptr,
                              S and S.ptr, UB.ptr, UB.ld, UB.stride, VB.ptr, VB.ld, VB.stride, beta,
                              dA.ptr if wanted != "adapters" else None, dA.ld, dU.ptr if on else None, dU.ld,
                              dU.stride, dV.ptr if on else None, dV.ld, dV.stride, ws, need)
        torch.cuda.synchronize()
        (oa, sa), (ou, su), (ov, sv) = ro.adapters_grad(a, b, dc, ids, ranks, scales, u, v, alpha, beta, du0, dv0)
        if wanted != "adapters":
            within(dA.read(), oa, sa, 1e-5, "dA")
        if on:
            within(dU.read(), ou, su, 1e-5, "dU")
            within(dV.read(), ov, sv, 1e-5, "dV")
        assert (ws[need:] == 0xFF).all()


@pytest.mark.parametrize("M,N,K,G,rank", [(8200, 2052, 100, 5, 24), (2048, 8200, 516, 3, 130)])
def test_adapters_of_many_rows(M, N, K, G, rank):
    """The tiles that only large products take, against float64 on the GPU."""
    gu.say("adapters of many rows", M, N, K, G, rank)
    f, ids, ranks, scales, (U, u), (V, v) = adapter_inputs(M, N, K, G, rank, False)
    cu = lambda x: torch.from_numpy(x).cuda()  # noqa: E731
    a, b, i, r, s, U, V = map(cu, (f(M, K), f(K, N), ids, ranks, scales, U, V))
    dc = cu(f(M, N))
    c, da, du, dv = (torch.full(x, NAN, device="cuda") for x in ((M, N), (M, K), (G, K, rank), (G, rank, N)))
    ws = torch.empty(max(g.sgemm_adapters_workspace_size(M, N, K, G, rank),
                         g.sgemm_adapters_grad_workspace_size(M, N, K, G, rank)), dtype=torch.uint8, device="cuda")
    g.sgemm_adapters(M, N, K, 1.25, a, K, b, N, 0.0, c, N, G, rank, i, r, s, U, rank, K * rank, V, N, rank * N, ws)
    g.sgemm_adapters_grad(M, N, K, 1.25, a, K, b, N, dc, N, G, rank, i, r, s, U, rank, K * rank, V, N, rank * N, 0.0,
                          da, K, du, rank, K * rank, dv, N, rank * N, ws)
    torch.cuda.synchronize()
    a, b, dc, u, v, s = (x.double() for x in (a, b, dc, cu(u), cu(v), s))
    want, size = a @ b, a.abs() @ b.abs()
    wa, sa = dc @ b.t(), dc.abs() @ b.t().abs()
    for e in range(G):
        m = torch.nonzero(i == e).reshape(-1)
        h, ha = a[m] @ u[e] * s[e], a[m].abs() @ u[e].abs() * s[e].abs()
        d, da_ = dc[m] @ v[e].t() * s[e], dc[m].abs() @ v[e].t().abs() * s[e].abs()
        want[m] += h @ v[e]
        size[m] += 2 * ha @ v[e].abs()
        wa[m] += d @ u[e].t()
        sa[m] += 2 * da_ @ u[e].t().abs()
        within(du[e].cpu().numpy(), (1.25 * a[m].t() @ d).cpu().numpy(), (2.5 * a[m].t().abs() @ da_).cpu().numpy(), 1e-5, "dU")
        within(dv[e].cpu().numpy(), (1.25 * h.t() @ dc[m]).cpu().numpy(), (2.5 * ha.t() @ dc[m].abs()).cpu().numpy(), 1e-5, "dV")
    within(c.cpu().numpy(), 1.25 * want.cpu().numpy(), 1.25 * size.cpu().numpy(), 1e-5, "C")
    within(da.cpu().numpy(), 1.25 * wa.cpu().numpy(), 1.25 * sa.cpu().numpy(), 1e-5, "dA")


@pytest.mark.parametrize("trans", [False, True], ids=["nn", "nt"])
@pytest.mark.parametrize("R,G,N,K", [(40000, 3, 260, 130), (9000, 70, 515, 70), (20000, 7, 1027, 40)])
def test_grouped_of_many_rows(R, G, N, K, trans):
    """The tiles that only many rows take, and the gradients by B, against float64 on the GPU."""
    gu.say("grouped of many rows", R, G, N, K, trans)
    gen = torch.Generator(device="cuda").manual_seed(R + trans)
    ids = torch.randint(-1, G, (R,), generator=gen, device="cuda", dtype=torch.int32)
    f = lambda *s: torch.rand(*s, generator=gen, device="cuda") * 2 - 1  # noqa: E731
    a, b = f(R, K), f(G, N, K) if trans else f(G, K, N)
    c, db = torch.full((R, N), NAN, device="cuda"), torch.full((G, K, N), NAN, device="cuda")
    off, rows = torch.empty(G + 1, dtype=torch.int32, device="cuda"), torch.empty(R, dtype=torch.int32, device="cuda")
    ws = torch.empty(g.sgemm_group_rows_workspace_size(R, G), dtype=torch.uint8, device="cuda")
    g.sgemm_group_rows(R, G, ids, off, rows, ws)
    g.sgemm_grouped(G, R, N, K, 1.0, a, K, 1, b, b.shape[2], N * K, trans, 0.0, c, N, True, off, rows)
    y = f(R, N)
    g.sgemm_grouped_tn(G, R, K, N, 1.0, a, K, 1, y, N, 1, 0.0, db, N, K * N, off, rows)
    torch.cuda.synchronize()
    for e in range(G):
        m = torch.nonzero(ids == e).reshape(-1)
        x, w, z = a[m].double(), (b[e].t() if trans else b[e]).double(), y[m].double()
        within(c[m].cpu().numpy(), (x @ w).cpu().numpy(), (x.abs() @ w.abs()).cpu().numpy(), 1e-5, "C")
        within(db[e].cpu().numpy(), (x.t() @ z).cpu().numpy(), (x.t().abs() @ z.abs()).cpu().numpy(), 1e-5, "dB")
    assert torch.isnan(c[ids < 0]).all()


def test_adapters_without_a_product():
    c = rng_of(14).uniform(-1, 1, (5, 6)).astype(np.float32)
    need = max(g.sgemm_adapters_workspace_size(5, 6, k, 2, 4) for k in (0, 3))
    ws = torch.empty(need, dtype=torch.uint8, device="cuda")
    for K, alpha in ((0, 1.0), (3, 0.0)):
        C = Buffer(c, 7)
        g.sgemm_adapters(5, 6, K, alpha, 0, 3, 0, 6, 0.5, C.ptr, 7, 2, 4, 0, None, None, 0, 4, 12, 0, 6, 24, ws)
        torch.cuda.synchronize()
        assert np.array_equal(C.read(), c * np.float32(0.5))
    # no rows, and alpha 0: the adapters' gradients keep beta times what they held, dA is 0
    du, dv = (rng_of(15).uniform(-1, 1, s).astype(np.float32) for s in ((2, 3, 4), (2, 4, 6)))
    ws = torch.empty(g.sgemm_adapters_grad_workspace_size(5, 6, 3, 2, 4), dtype=torch.uint8, device="cuda")
    for M, alpha in ((0, 1.0), (5, 0.0)):
        dU, dV, dA = Buffer(du), Buffer(dv), Buffer(np.full((M, 3), np.nan, np.float32))
        g.sgemm_adapters_grad(M, 6, 3, alpha, 0, 3, 0, 6, 0, 6, 2, 4, 0, None, None, 0, 4, 12, 0, 6, 24, 0.5,
                              dA.ptr, 3, dU.ptr, 4, 12, dV.ptr, 6, 24, ws)
        torch.cuda.synchronize()
        assert np.array_equal(dU.read(), du * np.float32(0.5)) and np.array_equal(dV.read(), dv * np.float32(0.5))
        assert (dA.read() == 0).all()


# ---------------------------------------------------------------------------
# as they are used
# ---------------------------------------------------------------------------
class Layer:
    """A layer of experts over the library's calls, forward and back: logits = X Wr, the router,
    H = silu-free product with W1, product with W2, weighted sum."""

    def __init__(self, T, D, F, E, k, seed=0):
        r = rng_of(16, T, D, F, E, k, seed)
        f = lambda *s: torch.from_numpy(r.uniform(-1, 1, s).astype(np.float32)).cuda()  # noqa: E731
        self.T, self.D, self.F, self.E, self.k = T, D, F, E, k
        self.x, self.wr, self.w1, self.w2 = f(T, D), f(D, E), f(E, D, F), f(E, F, D)
        self.dout = f(T, D)
        e = lambda *s: torch.full(s, NAN, device="cuda")  # noqa: E731
        i = lambda *s: torch.full(s, -1, dtype=torch.int32, device="cuda")  # noqa: E731
        R = T * k
        self.logits, self.weights, self.ids = e(T, E), e(T, k), i(T, k)
        self.offsets, self.rows = i(E + 1), i(R)
        self.h, self.y, self.out = e(R, F), e(R, D), e(T, D)
        self.dy, self.dh, self.dxs, self.dx = e(R, D), e(R, F), e(R, D), e(T, D)
        self.dw, self.dl, self.dw1, self.dw2 = e(T, k), e(T, E), e(E, D, F), e(E, F, D)
        self.space = torch.empty(max(256, g.sgemm_group_rows_workspace_size(R, E)), dtype=torch.uint8, device="cuda")

    def run(self, stream=None):
        T, D, F, E, k = self.T, self.D, self.F, self.E, self.k
        R = T * k
        o = dict(stream=stream)
        g.sgemm(T, E, D, 1.0, self.x, D, self.wr, E, 0.0, self.logits, E, **o)
        g.sgemm_route(T, E, k, 0, self.logits, E, None, 1, 1, 1, True, 1.0, self.ids, self.weights, **o)
        g.sgemm_group_rows(R, E, self.ids, self.offsets, self.rows, self.space, **o)
        g.sgemm_grouped(E, R, F, D, 1.0, self.x, D, k, self.w1, F, D * F, False, 0.0, self.h, F, False, self.offsets,
                        self.rows, **o)
        g.sgemm_grouped(E, R, D, F, 1.0, self.h, F, 0, self.w2, D, D * F, False, 0.0, self.y, D, True, self.offsets,
                        self.rows, **o)
        g.sgemm_combine(T, k, D, E, self.ids, self.weights, self.y, D, 0.0, self.out, D, **o)
        # and back
        g.sgemm_combine_grad(T, k, D, E, self.ids, self.weights, self.dout, D, self.y, D, self.dy, D, self.dw, **o)
        g.sgemm_grouped_tn(E, R, F, D, 1.0, self.h, F, 0, self.dy, D, 1, 0.0, self.dw2, D, D * F, self.offsets,
                           self.rows, **o)
        g.sgemm_grouped(E, R, F, D, 1.0, self.dy, D, 1, self.w2, D, D * F, True, 0.0, self.dh, F, False,
                        self.offsets, self.rows, **o)
        g.sgemm_grouped_tn(E, R, D, F, 1.0, self.x, D, k, self.dh, F, 0, 0.0, self.dw1, F, D * F, self.offsets,
                           self.rows, **o)
        g.sgemm_grouped(E, R, D, F, 1.0, self.dh, F, 0, self.w1, F, D * F, True, 0.0, self.dxs, D, True,
                        self.offsets, self.rows, **o)
        g.sgemm_combine(T, k, D, E, self.ids, None, self.dxs, D, 0.0, self.dx, D, **o)
        g.sgemm_route_grad(T, E, k, 0, self.logits, E, True, 1.0, self.ids, self.dw, self.dl, E, **o)

    def outputs(self):
        return {n: getattr(self, n) for n in ("ids", "offsets", "rows", "weights", "out", "dx", "dw", "dl", "dw1", "dw2")}

    def wipe(self):
        for n, v in self.outputs().items():
            v.fill_(-1 if v.dtype == torch.int32 else NAN)

    def reference(self):
        """The same layer in float64 with autograd, for the experts the router chose."""
        x, w1, w2 = (v.double().cpu().requires_grad_(True) for v in (self.x, self.w1, self.w2))
        logits = self.logits.double().cpu().requires_grad_(True)
        ids = self.ids.cpu().long()
        w = torch.softmax(logits.gather(1, ids), 1)
        out = sum(w[:, j:j + 1] * torch.einsum("td,tdf,tfe->te", x, w1[ids[:, j]], w2[ids[:, j]])
                  for j in range(self.k))
        out.backward(self.dout.double().cpu())
        return dict(weights=w.detach(), out=out.detach(), dx=x.grad, dw1=w1.grad, dw2=w2.grad, dl=logits.grad)


LAYERS = [(1, 40, 24, 4, 2), (5, 33, 31, 6, 3), (70, 64, 96, 8, 2), (300, 48, 36, 5, 2)]


@pytest.mark.parametrize("shape", LAYERS, ids=lambda s: "x".join(map(str, s)))
def test_layer_forward_and_back(shape):
    gu.say("layer", shape)
    layer = Layer(*shape)
    layer.run()
    torch.cuda.synchronize()
    want_ids, want_w = ro.route(layer.logits.cpu().numpy(), layer.k, renorm=True)
    assert np.array_equal(layer.ids.cpu().numpy(), want_ids)
    ref = layer.reference()
    for name, want in ref.items():
        got = getattr(layer, name).double().cpu()
        # three products one after the other and a sum: 4 * 1e-5 of the terms, whose size is at
        # most that of the largest element times the number of cancelling terms; in the 2-norm
        # random errors of 2^-24 per operation leave less than 1e-5
        assert (got - want).norm() <= 1e-5 * want.norm() + 1e-30, name


@pytest.mark.parametrize("shape", LAYERS[1:3], ids=lambda s: "x".join(map(str, s)))
def test_layer_captured_and_replayed(shape):
    """Replays between eager runs of the same and of another layer, each compared bit for bit."""
    gu.say("layer captured", shape)
    layer, other = Layer(*shape), Layer(*LAYERS[2], seed=3)
    layer.run()
    torch.cuda.synchronize()
    want = {n: v.clone() for n, v in layer.outputs().items()}
    stream = torch.cuda.Stream()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=stream):
        layer.run()
    for replay in range(4):
        layer.wipe()
        other.run()
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        for n, v in layer.outputs().items():
            assert torch.equal(v, want[n]), (replay, n)
        if replay == 1:
            layer.wipe()
            layer.run()
            torch.cuda.synchronize()
            for n, v in layer.outputs().items():
                assert torch.equal(v, want[n]), n


def test_layers_on_two_streams_at_once():
    gu.say("two streams")
    layers = [Layer(*LAYERS[2], seed=i) for i in range(2)]
    wants = []
    for layer in layers:
        layer.run()
        torch.cuda.synchronize()
        wants.append({n: v.clone() for n, v in layer.outputs().items()})
        layer.wipe()
    streams = [torch.cuda.Stream() for _ in layers]
    torch.cuda.synchronize()
    for _ in range(5):
        for layer, stream in zip(layers, streams):
            layer.run(stream)
    torch.cuda.synchronize()
    for layer, want in zip(layers, wants):
        for n, v in layer.outputs().items():
            assert torch.equal(v, want[n]), n


def test_adapters_captured_and_replayed():
    M, N, K, G, rank = 40, 130, 70, 4, 33
    f, ids, ranks, scales, (U, _), (V, _) = adapter_inputs(M, N, K, G, rank, False)
    cu = lambda x: torch.from_numpy(x).cuda()  # noqa: E731
    a, b, dc, i, r, s, u, v = map(cu, (f(M, K), f(K, N), f(M, N), ids, ranks, scales, U, V))
    c, da, du, dv = (torch.empty(x, device="cuda") for x in ((M, N), (M, K), (G, K, rank), (G, rank, N)))
    ws = torch.empty(max(g.sgemm_adapters_workspace_size(M, N, K, G, rank),
                         g.sgemm_adapters_grad_workspace_size(M, N, K, G, rank)), dtype=torch.uint8, device="cuda")

    def both():
        g.sgemm_adapters(M, N, K, 1.0, a, K, b, N, 0.0, c, N, G, rank, i, r, s, u, rank, K * rank, v, N, rank * N, ws)
        g.sgemm_adapters_grad(M, N, K, 1.0, a, K, b, N, dc, N, G, rank, i, r, s, u, rank, K * rank, v, N, rank * N,
                              0.0, da, K, du, rank, K * rank, dv, N, rank * N, ws)
    both()
    torch.cuda.synchronize()
    want = [x.clone() for x in (c, da, du, dv)]
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        both()
    for _ in range(4):
        for x in (c, da, du, dv):
            x.fill_(NAN)
        ws.fill_(0xFF)
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(x, y) for x, y in zip((c, da, du, dv), want))
        both()
        torch.cuda.synchronize()
        assert all(torch.equal(x, y) for x, y in zip((c, da, du, dv), want))


def test_tensor_checks():
    x = torch.zeros(4, 8, device="cuda")
    ids = torch.zeros(4, 2, dtype=torch.int32, device="cuda")
    w = torch.zeros(4, 2, device="cuda")
    call = lambda **k: g.sgemm_route(*{**dict(T=4, E=8, k=2, scoring=0, logits=x, ldl=8, bias=None, groups=1,  # noqa: E731
                                              top_groups=1, group_best=1, renorm=True, scale=1.0, ids=ids, weights=w), **k}.values())
    call()
    for bad, kind in ((dict(logits=x.double()), TypeError), (dict(ids=ids.long()), TypeError), (dict(logits=x.cpu()), TypeError),
                      (dict(T=5), ValueError), (dict(ldl=9), ValueError), (dict(ids=ids.t().contiguous().t()), ValueError),
                      (dict(logits=torch.zeros(8, 4, device="cuda").t()), ValueError)):
        with pytest.raises(kind):
            call(**bad)
    wide = torch.zeros(4, 20, device="cuda")
    call(logits=wide[:, 3:11], ldl=20)
    torch.cuda.synchronize()
