"""The norm, 8-bit rows and their product, the gated projections and their gradients against
their 64-bit plain forms (block_oracle), through the public binding.

Tolerances.  What is computed in 64 bits and rounded once is off by at most 2^-24 of the value
(ONCE: 1% more, for what 64 bits lose).  Whole numbers and scales of 8-bit rows are equal to
the definition's on the float32 row.  Sums of float32 products follow the library's rule, 1e-5
of the sum of the terms' magnitudes.  The activation's product takes at most ten roundings of
2^-24 of its magnitude (block_oracle.act gives it): the exponential 2, the sum, the quotient,
the other side's product, two products, and 3 for the argument.  A slope takes at most 16 of
its terms', which 1e-5 of the sum of products covers with what the sum itself loses.
dweight is a 64-bit sum of shares that are rounded once each, and rounded: 2 2^-24 of its terms
(rows too long for registers add a rounding per row to a share)."""
import numpy as np
import pytest
import torch

import fp32_gemm_03_amd as g
from tests import block_oracle as bo
from tests import gpu_util as gu
from tests.test_rows_gpu import NAN, U24, Buffer, rng_of, within

pytestmark = pytest.mark.gpu
ONCE = 1.01 * U24
SUM = 1e-5
ACT = 10 * U24


@pytest.fixture(autouse=True)
def _gpu_available():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")


class Bytes:
    """rows x cols int8 with a leading dimension and an offset in a band of `fill`."""

    def __init__(self, data, ld=None, offset=0, fill=85):
        data = np.asarray(data, np.int8)
        rows, cols = data.shape
        ld = cols if ld is None else ld
        self.ld, self.fill = ld, fill
        self.index = 64 + offset + np.arange(rows)[:, None] * ld + np.arange(cols)[None, :]
        host = np.full((int(self.index.max()) + 1 if data.size else 64) + 64, fill, np.int8)
        host[self.index.reshape(-1)] = data.reshape(-1)
        self.owner = torch.from_numpy(host).cuda()
        self.ptr = self.owner.data_ptr() + 64 + offset

    def read(self):
        host = self.owner.cpu().numpy()
        outside = np.ones(len(host), bool)
        outside[self.index.reshape(-1)] = False
        assert (host[outside] == self.fill).all(), "written outside"
        return host[self.index]


def floats(*shape, fill=7.0, ld=None):
    return Buffer(np.full(shape, fill, np.float32), ld)


# ---------------------------------------------------------------------------
# norm
# ---------------------------------------------------------------------------
def stream(T, N, seed, special=True):
    r = rng_of(11, T, N, seed)
    x = (r.standard_normal((T, N)) * np.exp(r.standard_normal(N))).astype(np.float32)
    if special:
        for t in range(0, T, 9):
            x[t] = 0.0
        for t in range(2, T, 9):
            x[t] *= np.float32(1e-30)  # squares vanish in 32 bits
        for t in range(3, T, 9):
            x[t] *= np.float32(1e30)   # and overflow
        for t in range(4, T, 18):
            x[t, N // 2] = np.nan
        for t in range(5, T, 18):
            x[t, N - 1] = -np.inf
        for t in range(6, T, 9):
            x[t] = np.round(x[t] * 2) / 2  # halves of the largest
        for t in range(7, T, 9):
            x[t] = np.float32(1e-42)       # below the normal range
    return x


NORMS = [(1, 1), (1, 4096), (3, 63), (19, 64), (4, 255), (7, 256), (6, 257), (11, 512), (5, 513), (19, 1000), (5, 1023),
         (9, 1025), (4, 2048), (3, 2049), (19, 4095), (2, 4097), (3, 8191), (2, 8193), (2, 16384), (3, 16385), (19, 40003),
         (700, 129)]


@pytest.mark.parametrize("residual", [False, True])
@pytest.mark.parametrize("T,N", NORMS)
def test_norm(T, N, residual):
    gu.say("norm", T, N, residual)
    eps = 1e-5
    x = stream(T, N, 1)
    r = stream(T, N, 2, special=False) if residual else None
    if residual and T > 4:
        r[0] = 0.0
    w = (1 + 0.3 * rng_of(12, N).standard_normal(N)).astype(np.float32) if N % 2 else None
    want_h, want = bo.norm(x, r, w, eps)
    X, R = Buffer(x, N + 1), Buffer(r, N + 3) if residual else None
    W = Buffer(w) if w is not None else None
    S, Y = floats(T, N, ld=N + 2), floats(T, N, ld=N + 5)
    Q, scales = Bytes(np.full((T, N), 3), N + 1), floats(T)
    for outputs in ((True, True, True), (True, False, True), (False, True, False), (False, False, True)):
        s, y, q = outputs
        g.sgemm_norm(T, N, X.ptr, X.ld, R.ptr if residual else None, R.ld if residual else N, W.ptr if W else None, eps,
                     S.ptr if s else None, S.ld, Y.ptr if y else None, Y.ld, Q.ptr if q else None, Q.ld,
                     scales.ptr if q else None)
        torch.cuda.synchronize()
        if s:
            assert np.array_equal(S.read().view(np.uint32) & 0x7fffffff,
                                  np.where(np.isnan(want_h), np.float32(NAN), want_h).view(np.uint32) & 0x7fffffff) \
                or np.array_equal(S.read(), want_h, equal_nan=True)
        if y:
            got = Y.read()
            within(got, want, np.abs(want), ONCE, "y")
        if q:
            got = Y.read()  # of the first call: y and the 8-bit rows are of the same rounded numbers
            want_q, want_s = bo.quantize(got)
            assert np.array_equal(Q.read(), want_q)
            assert np.array_equal(scales.read(), want_s, equal_nan=True)


@pytest.mark.parametrize("N", [100, 4096, 20000])
def test_norm_in_place(N):
    """sum in x's or residual's place, y in x's, residual's or sum's."""
    gu.say("norm in place", N)
    T, eps = 5, 2.0 ** -10
    x, r = stream(T, N, 3, special=False), stream(T, N, 4, special=False)
    h, y = bo.norm(x, r, None, eps)
    q, s = None, None
    for sum_at, y_at in (("x", None), ("r", "x"), ("r", "r"), (None, "x"), ("x", "r"), ("x", "x"), (None, "r")):
        b = {"x": Buffer(x, N + 1), "r": Buffer(r, N + 1)}
        Q, scales = Bytes(np.zeros((T, N)), N), floats(T)
        g.sgemm_norm(T, N, b["x"].ptr, N + 1, b["r"].ptr, N + 1, None, eps, b[sum_at].ptr if sum_at else None, N + 1,
                     b[y_at].ptr if y_at else None, N + 1, Q.ptr, Q.ld, scales.ptr)
        torch.cuda.synchronize()
        if y_at:
            within(b[y_at].read(), y, np.abs(y), ONCE, f"y in {y_at}")
        if sum_at and sum_at != y_at:
            assert np.array_equal(b[sum_at].read(), h), (sum_at, y_at)
        got = Q.read(), scales.read()
        if q is not None:
            assert np.array_equal(got[0], q) and np.array_equal(got[1], s), (sum_at, y_at)
        q, s = got


def test_norm_of_no_columns():
    scales = floats(3)
    g.sgemm_norm(3, 0, None, 1, None, 1, None, 0.0, None, 1, None, 1, scales.ptr, 1, scales.ptr)
    torch.cuda.synchronize()
    assert np.array_equal(scales.read(), np.zeros(3))


@pytest.mark.parametrize("T,N", NORMS + [(2000, 300), (513, 70)])
def test_norm_grad(T, N):
    gu.say("norm_grad", T, N)
    eps = 2.0 ** -12
    r = rng_of(13, T, N)
    h = stream(T, N, 5, special=False)
    h[T // 3] = 0.0
    dy, ds = (r.standard_normal((T, N)).astype(np.float32) for _ in range(2))
    w = (1 + 0.3 * r.standard_normal(N)).astype(np.float32)
    start = r.standard_normal(N).astype(np.float32)
    H, DY, DS, W = Buffer(h, N + 1), Buffer(dy, N + 2), Buffer(ds, N + 3), Buffer(w)
    need = g.sgemm_norm_grad_workspace_size(T, N)
    space = torch.full((need,), 0xFF, dtype=torch.uint8, device="cuda")  # NaN
    rows = 1 + (-(-T // 512) if N > 8192 else 0)
    for weighted, streamed, beta in ((True, True, 0.0), (False, False, 0.5), (True, False, 1.0)):
        want, size, dw, dw_size = bo.norm_grad(h, w if weighted else None, eps, dy, ds if streamed else None)
        first = None
        for parts in ("both", "dh", "dweight", "both"):
            DH, DW = floats(T, N, ld=N + 4), Buffer(np.full(N, NAN, np.float32) if beta == 0 else start)
            g.sgemm_norm_grad(T, N, H.ptr, H.ld, W.ptr if weighted else None, eps, DY.ptr, DY.ld,
                              DS.ptr if streamed else None, DS.ld, DH.ptr if parts != "dweight" else None, DH.ld, beta,
                              DW.ptr if parts != "dh" else None, space if parts != "dh" else None)
            torch.cuda.synchronize()
            if parts != "dweight":
                # one rounding, and 2^-45 of the terms for what cancels in 64 bits
                within(DH.read(), want, np.abs(want) + 2.0 ** -21 * size, ONCE, "dh")
            if parts != "dh":
                within(DW.read(), dw + beta * start, dw_size + np.abs(beta * start), (1 + rows) * U24, "dweight")
            if parts == "both":
                got = DH.read().tobytes() + DW.read().tobytes()
                assert first is None or got == first, "not the same run to run"
                first = got


def test_norm_grad_in_place_and_without_rows():
    T, N = 6, 1000
    r = rng_of(14)
    h, dy, ds, w = (r.standard_normal(s).astype(np.float32) for s in ((T, N), (T, N), (T, N), N))
    want, size, _, _ = bo.norm_grad(h, w, 0.0, dy, ds)
    H, W = Buffer(h), Buffer(w)
    for place in ("dy", "ds", "h"):
        b = {"dy": Buffer(dy), "ds": Buffer(ds), "h": Buffer(h)}
        g.sgemm_norm_grad(T, N, b["h"].ptr, N, W.ptr, 0.0, b["dy"].ptr, N, b["ds"].ptr, N, b[place].ptr, N, 0.0, None)
        torch.cuda.synchronize()
        within(b[place].read(), want, np.abs(want) + 2.0 ** -21 * size, ONCE, place)
    start = r.standard_normal(N).astype(np.float32)
    for beta in (0.0, 0.5):
        DW = Buffer(start)
        g.sgemm_norm_grad(0, N, None, N, W.ptr, 0.0, None, N, None, N, None, N, beta, DW.ptr)
        torch.cuda.synchronize()
        assert np.array_equal(DW.read(), np.float32(beta) * start)


# ---------------------------------------------------------------------------
# rows to 8 bits
# ---------------------------------------------------------------------------
@pytest.mark.parametrize("T,N", NORMS)
def test_quantize(T, N):
    gu.say("quantize", T, N)
    x = stream(T, N, 6)
    X = Buffer(x, N + 1)
    for offset, ld in ((0, N), (1, N + 3)):
        Q, scales = Bytes(np.full((T, N), 3), ld, offset), floats(T)
        g.sgemm_quantize(T, N, X.ptr, X.ld, 0, None, N, Q.ptr, Q.ld, scales.ptr)
        torch.cuda.synchronize()
        want_q, want_s = bo.quantize(x)
        assert np.array_equal(Q.read(), want_q)
        assert np.array_equal(scales.read(), want_s, equal_nan=True)


@pytest.mark.parametrize("kind", [0, 1, 2])
@pytest.mark.parametrize("T,N", [(1, 1), (19, 64), (3, 255), (5, 1023), (9, 2048), (19, 4095), (2, 8193), (2, 17001)])
def test_quantize_gated(T, N, kind):
    """act(gate) x is rounded once from 64 bits; the whole numbers are those of a row that is off by at
    most that rounding, so next to a border they may be the neighbour."""
    gu.say("quantize gated", T, N, kind)
    r = rng_of(15, T, N, kind)
    x = stream(T, N, 7, special=False)
    gate = (3 * r.standard_normal((T, N))).astype(np.float32)
    if T > 8:
        gate[1, N // 3], gate[2] = -np.inf, -np.inf
        gate[3, N // 3], x[4, 0], gate[5, 1] = np.inf, np.inf, np.nan
        gate[6] = -1e30
        gate[7] = np.linspace(-60, 60, N).astype(np.float32)
    with np.errstate(all="ignore"):
        a = bo.act(kind, gate)[0]
        v = a * x.astype(np.float64)
    X, G = Buffer(x, N + 1), Buffer(gate, N + 2)
    Q, scales = Bytes(np.full((T, N), 3), N), floats(T)
    g.sgemm_quantize(T, N, X.ptr, X.ld, kind, G.ptr, G.ld, Q.ptr, Q.ld, scales.ptr)
    torch.cuda.synchronize()
    q, s = Q.read(), scales.read()
    good = np.isfinite(v.astype(np.float32)).all(1)
    assert np.array_equal(np.isnan(s), ~good)
    assert (q[~good] == 0).all()
    v, q, s = v[good], q[good], s[good].astype(np.float64)
    most = np.abs(v).max(1, initial=0)
    # the maximum is rounded to 32 bits, the scale again
    assert (np.abs(s - most / 127) <= 2.02 * U24 * most / 127 + 1e-45).all()
    steps = np.divide(127.0 * v, most[:, None], out=np.zeros_like(v), where=most[:, None] > 1e-37)
    off = np.abs(q - steps)
    live = most > 1e-37
    assert (off[live] <= 0.5 + 127 * 3 * U24).all()


def test_quantize_halves():
    """Half of the row's largest number is 63.5 steps: to the even one, in every kernel."""
    for N in (4, 300, 4096, 20000):
        x = np.zeros((2, N), np.float32)
        x[:, 0], x[:, 1], x[:, 2], x[:, N - 1] = 3.3, 1.65, -1.65, -3.3
        x[1] *= np.float32(2.0 ** -40)
        X, Q, scales = Buffer(x), Bytes(np.zeros((2, N)), N), floats(2)
        g.sgemm_quantize(2, N, X.ptr, N, 0, None, N, Q.ptr, N, scales.ptr)
        torch.cuda.synchronize()
        want, want_s = bo.quantize(x)
        assert np.array_equal(Q.read(), want) and np.array_equal(scales.read(), want_s)
        assert want[0, 0] == 127 and abs(int(want[0, 1])) in (63, 64)


# ---------------------------------------------------------------------------
# 8-bit products
# ---------------------------------------------------------------------------
I8S = [(1, 1, 1), (1, 64, 128), (1, 500, 1000), (3, 17, 5), (16, 33, 127), (17, 31, 129), (29, 100, 640), (33, 20, 255),
       (64, 130, 300), (65, 64, 64), (100, 90, 130), (130, 260, 257), (200, 1500, 96), (1000, 70, 1025), (600, 3000, 384),
       (2049, 1793, 145), (4100, 4100, 70), (2, 300, 20011), (70, 40, 131071),
       (2050, 2051, 33), (1030, 4093, 40)]


@pytest.mark.parametrize("M,N,K", I8S)
def test_i8(M, N, K):
    gu.say("i8", M, N, K)
    r = rng_of(16, M, N, K)
    A, B = (r.integers(-128, 128, s).astype(np.int8) for s in ((M, K), (N, K)))
    if K > 100000:
        A[:], B[:] = -128, -128  # the largest sum
        B[0] = 127
    sa, sb = (np.exp(r.standard_normal(n)).astype(np.float32) / 127 for n in (M, N))
    C0 = r.standard_normal((M, N)).astype(np.float32)
    word = lambda n: -(-n // 4) * 4  # noqa: E731
    SA, SB = Buffer(sa), Buffer(sb)
    layouts = [(word(K), 0), (word(K) + 4, 4)]
    if M * N * K < 1e8:
        layouts += [(K, 0), (K + 1, 3), (word(K), 1)]
    for ld, offset in layouts:
        a, b = Bytes(A, ld, offset), Bytes(B, ld + 8 if ld % 4 == 0 else ld, offset)
        for alpha, beta, scaled in ((1.0, 0.0, True), (-0.75, 0.5, True), (2.0, 1.0, False)):
            want, size = bo.i8(A, sa if scaled else None, B, sb if scaled else None, alpha, beta, C0)
            C = Buffer(C0 if beta else np.full((M, N), NAN, np.float32), N + 3)
            g.sgemm_i8(M, N, K, alpha, a.ptr, a.ld, SA.ptr if scaled else None, b.ptr, b.ld,
                       SB.ptr if scaled else None, beta, C.ptr, C.ld)
            torch.cuda.synchronize()
            within(C.read(), want, np.abs(want) + 2.0 ** -26 * size, ONCE, f"ld {ld} offset {offset} beta {beta}")


def test_i8_scales_and_special_cases():
    M, N, K = 5, 40, 64
    r = rng_of(17)
    A, B = (r.integers(-128, 128, s).astype(np.int8) for s in ((M, K), (N, K)))
    sa, sb = np.ones(M, np.float32), np.ones(N, np.float32)
    sa[1], sb[3] = np.nan, 0.0
    C0 = r.standard_normal((M, N)).astype(np.float32)
    a, b, SA, SB = Bytes(A), Bytes(B), Buffer(sa), Buffer(sb)
    C = Buffer(C0)
    g.sgemm_i8(M, N, K, 1.0, a.ptr, K, SA.ptr, b.ptr, K, SB.ptr, 0.0, C.ptr, N)
    torch.cuda.synchronize()
    got = C.read()
    assert np.isnan(got[1]).all() and (got[[0, 2, 3, 4], 3] == 0).all() and np.isfinite(got[[0, 2, 3, 4]]).all()
    for alpha, k in ((0.0, K), (1.0, 0)):  # the operands and the scales are not read
        for beta in (0.0, -0.5):
            for rows, cols in ((M, N), (100, 90), (300, 200)):
                start = np.full((rows, cols), NAN, np.float32) if beta == 0 else rng_of(18).standard_normal((rows, cols)).astype(np.float32)
                C = Buffer(start, cols + 1)
                nan = Buffer(np.full(512, NAN, np.float32))
                g.sgemm_i8(rows, cols, k, alpha, None, K, nan.ptr, None, K, nan.ptr, beta, C.ptr, cols + 1)
                torch.cuda.synchronize()
                assert np.array_equal(C.read(), np.zeros((rows, cols)) if beta == 0 else np.float32(beta) * start)


# ---------------------------------------------------------------------------
# gated projections
# ---------------------------------------------------------------------------
GATED = [(1, 1, 1), (1, 100, 333), (5, 17, 3), (16, 64, 128), (17, 33, 65), (29, 300, 515), (33, 20, 31), (64, 130, 100),
         (65, 64, 32), (70, 129, 66), (200, 100, 45), (130, 1000, 129), (600, 700, 64), (1030, 1030, 40), (2050, 2050, 67), (100, 2100, 50), (20, 4700, 40),
         (30, 9300, 30), (4100, 33, 4100),
         (1900, 70, 1000), (300, 515, 200), (600, 130, 203), (130, 700, 1030), (1100, 40, 515), (261, 2049, 130),
         (320, 2999, 67), (455, 2276, 131), (456, 2304, 32), (257, 4000, 5)]


def operands(T, N, K, seed):
    r = rng_of(19, T, N, K, seed)
    scale = 1.5 / np.sqrt(K)
    return [(r.standard_normal(s) * f).astype(np.float32) for s, f in (((T, K), 1), ((K, N), scale), ((K, N), scale))]


def check_forward(kind, x, G, U, y, gate, up):
    want_g, size_g, want_u, size_u = bo.gated(kind, x, G, U)
    within(gate, want_g, size_g, SUM, "gate")
    within(up, want_u, size_u, SUM, "up")
    a, size = bo.act(kind, gate)
    u = up.astype(np.float64)
    within(y, a * u, size * np.abs(u) + 1e-30, ACT, "y")


@pytest.mark.parametrize("T,N,K", GATED)
def test_gated(T, N, K):
    for kind in (0, 1, 2):
        gu.say("gated", T, N, K, kind)
        x, G, U = operands(T, N, K, kind)
        for pad in (0, 1, 4):
            X, GB, UB = Buffer(x, K + pad), Buffer(G, N + pad), Buffer(U, N + 2 * pad)
            Y, gate, up = (floats(T, N, ld=N + pad) for _ in range(3))
            g.sgemm_gated(T, N, K, kind, X.ptr, X.ld, GB.ptr, GB.ld, UB.ptr, UB.ld, Y.ptr, Y.ld, gate.ptr, gate.ld, up.ptr,
                          up.ld)
            torch.cuda.synchronize()
            y = Y.read()
            check_forward(kind, x, G, U, y, gate.read(), up.read())
            Y = floats(T, N, ld=N + pad)  # without what the gradient needs: the same
            g.sgemm_gated(T, N, K, kind, X.ptr, X.ld, GB.ptr, GB.ld, UB.ptr, UB.ld, Y.ptr, Y.ld, None, N, None, N)
            torch.cuda.synchronize()
            assert np.array_equal(Y.read(), y)


@pytest.mark.parametrize("T", [3, 70, 1030])
def test_gated_nan_and_infinity_stay_in_their_rows_and_columns(T):
    N, K = 1030, 37
    x, G, U = operands(T, N, K, 9)
    x[1, 3], G[5, 7], U[6, 9] = np.nan, np.inf, np.nan
    X, GB, UB, Y = Buffer(x, K + 1), Buffer(G, N + 1), Buffer(U, N + 1), floats(T, N)
    g.sgemm_gated(T, N, K, 0, X.ptr, X.ld, GB.ptr, GB.ld, UB.ptr, UB.ld, Y.ptr, Y.ld, None, N, None, N)
    torch.cuda.synchronize()
    y = Y.read()
    assert np.isnan(y[1]).all() and np.isnan(y[:, 9]).all()
    rest = np.ones((T, N), bool)
    rest[1], rest[:, 7], rest[:, 9] = False, False, False
    assert np.isfinite(y[rest]).all()
    # a gate of -infinity is closed, one of infinity passes infinity on
    column = y[[t for t in range(T) if t != 1], 7]
    assert (np.isinf(column) | (column == 0)).all()


def test_gated_without_a_sum():
    for kind in (0, 1, 2):
        Y, gate, up = floats(70, 9), floats(70, 9), floats(70, 9)
        g.sgemm_gated(70, 9, 0, kind, None, 1, None, 9, None, 9, Y.ptr, 9, gate.ptr, 9, up.ptr, 9)
        torch.cuda.synchronize()
        assert not Y.read().any() and not gate.read().any() and not up.read().any()


def backward(kind, x, G, U, gate, up, dy, beta, dG0, dU0, pad, parts="both"):
    T, K = x.shape
    N = G.shape[1]
    X, GB, UB, GA, UP, DY = (Buffer(v, v.shape[1] + pad) for v in (x, G, U, gate, up, dy))
    DX = floats(T, K, ld=K + pad)
    DG, DU = (Buffer(v, N + pad) for v in (dG0, dU0))
    need = g.sgemm_gated_grad_workspace_size(T, N, K)
    space = torch.full((need + 1024,), 0xFF, dtype=torch.uint8, device="cuda")  # NaN
    g.sgemm_gated_grad(T, N, K, kind, X.ptr, X.ld, GB.ptr, GB.ld, UB.ptr, UB.ld, GA.ptr, GA.ld, UP.ptr, UP.ld, DY.ptr,
                       DY.ld, DX.ptr if parts != "weights" else None, DX.ld, beta,
                       DG.ptr if parts != "rows" else None, DG.ld, DU.ptr if parts != "rows" else None, DU.ld, space)
    torch.cuda.synchronize()
    assert bool((space[need:] == 0xFF).all()), "beyond the workspace"
    return DX.read(), DG.read(), DU.read()


@pytest.mark.parametrize("T,N,K", GATED)
def test_gated_grad(T, N, K):
    for kind in (0, 1, 2):
        gu.say("gated_grad", T, N, K, kind)
        r = rng_of(20, T, N, K, kind)
        x, G, U = operands(T, N, K, kind)
        gate, up, dy = (r.standard_normal((T, N)).astype(np.float32) * s for s in (np.float32(2), np.float32(1), np.float32(1)))
        grads, sizes = bo.gated_grad(kind, x, G, U, gate, up, dy)
        first = None
        for pad, beta, parts in ((0, 0.0, "both"), (1, 0.5, "both"), (4, 1.0, "both"), (1, 0.0, "rows"), (1, 0.0, "weights")):
            dG0, dU0 = (np.full((K, N), NAN, np.float32) if beta == 0 else r.standard_normal((K, N)).astype(np.float32)
                        for _ in range(2))
            got = backward(kind, x, G, U, gate, up, dy, beta, dG0, dU0, pad, parts)
            old = [0.0 if beta == 0 else beta * v.astype(np.float64) for v in (dG0, dU0)]
            if parts != "weights":
                within(got[0], grads[0], sizes[0], SUM, "dx")
            if parts != "rows":
                within(got[1], grads[1] + old[0], sizes[1] + np.abs(old[0]), SUM, "dG")
                within(got[2], grads[2] + old[1], sizes[2] + np.abs(old[1]), SUM, "dU")
            if beta == 0.0 and parts == "both":
                again = backward(kind, x, G, U, gate, up, dy, beta, dG0, dU0, pad, parts)
                assert all(np.array_equal(a, b) for a, b in zip(got, again)), "not the same run to run"


def test_gated_grad_of_no_rows():
    K, N = 9, 7
    start = [rng_of(21, i).standard_normal((K, N)).astype(np.float32) for i in range(2)]
    empty = np.zeros((0, N), np.float32)
    got = backward(0, np.zeros((0, K), np.float32), start[0], start[1], empty, empty, empty, 0.5, start[0], start[1], 0)
    assert np.array_equal(got[1], 0.5 * start[0]) and np.array_equal(got[2], 0.5 * start[1])
    DX = floats(4, K)
    g.sgemm_gated_grad(4, 0, K, 0, None, K, None, 1, None, 1, None, 1, None, 1, None, 1, DX.ptr, K, 0.0, None, 1, None, 1,
                       None)
    torch.cuda.synchronize()
    assert not DX.read().any()
