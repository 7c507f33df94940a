"""The block's operators at sizes and in forms that their parametrised tests do not reach, and
which kernels all those sizes launch: every one that the library holds.

Tolerances are those of test_block_gpu; dweight is a 64-bit sum of shares that are rounded once
each, and rounded: 2 2^-24 of its terms (1% more for what 64 bits lose), for rows of any length."""
import ctypes

import numpy as np
import pytest
import torch

import fp32_gemm_03_amd as g
from fp32_gemm_03_amd import build
from tests import block_oracle as bo
from tests import gpu_util as gu
from tests import test_block_gpu as tb
from tests.test_block_gpu import ONCE, SUM, Bytes, backward, check_forward, floats, operands, stream
from tests.test_rows_gpu import NAN, U24, Buffer, rng_of, within

pytestmark = pytest.mark.gpu


@pytest.fixture(autouse=True)
def _gpu_available():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")


# ---------------------------------------------------------------------------
# the norm's outputs, each combination by itself
# ---------------------------------------------------------------------------
@pytest.mark.parametrize("residual", [False, True])
@pytest.mark.parametrize("T,N", tb.NORMS)
def test_norm_writes_what_is_asked_for(T, N, residual):
    """Buffers of their own for every combination of outputs: what is asked for is written, the bits
    the same in all of them, and what is not is left as it was."""
    gu.say("norm's outputs", T, N, residual)
    eps = 1e-5
    x = stream(T, N, 1)
    r = stream(T, N, 2, special=False) if residual else None
    w = (1 + 0.3 * rng_of(12, N).standard_normal(N)).astype(np.float32) if N % 2 else None
    want_h, want = bo.norm(x, r, w, eps)
    X, R = Buffer(x, N + 1), Buffer(r, N + 3) if residual else None
    W = Buffer(w) if w is not None else None
    first = None
    for s, y, q in ((True, True, True), (True, True, False), (True, False, True), (False, True, True),
                    (True, False, False), (False, True, False), (False, False, True)):
        S, Y, scales = floats(T, N, ld=N + 2), floats(T, N, ld=N + 5), floats(T)
        Q = Bytes(np.full((T, N), -128), N + 1)  # (no row to 8 bits has a -128)
        g.sgemm_norm(T, N, X.ptr, X.ld, R.ptr if residual else None, R.ld if residual else N, W.ptr if W else None, eps,
                     S.ptr if s else None, S.ld, Y.ptr if y else None, Y.ld, Q.ptr if q else None, Q.ld,
                     scales.ptr if q else None)
        torch.cuda.synchronize()
        got = S.read(), Y.read(), Q.read(), scales.read()
        if first is None:
            first = got
            # equal numbers and zeros of the same sign
            assert np.array_equal(got[0], want_h, equal_nan=True)
            assert np.array_equal(np.signbit(got[0]) & ~np.isnan(got[0]), np.signbit(want_h) & ~np.isnan(want_h))
            within(got[1], want, np.abs(want), ONCE, "y")
            want_q, want_s = bo.quantize(got[1])
            assert np.array_equal(got[2], want_q) and np.array_equal(got[3], want_s, equal_nan=True)
        for name, v, all_, asked, left in zip(("sum", "y", "q", "scales"), got, first, (s, y, q, q), (7.0, 7.0, -128, 7.0)):
            if asked:
                assert np.array_equal(v.view(np.uint8), all_.view(np.uint8)), (name, s, y, q)
            else:
                assert (v == left).all(), (name, "written", s, y, q)


# ---------------------------------------------------------------------------
# dweight of more rows than it has shares
# ---------------------------------------------------------------------------
@pytest.mark.parametrize("N", [300, 8192, 8195, 20003])
def test_shares_of_dweight_are_summed_in_64_bits(N):
    """Rows of 2^24, of 1 and of -2^24 in one share: in 32 bits the 1 is lost to the first."""
    gu.say("dweight of far terms", N)
    dy = torch.empty(1536, N, device="cuda")
    for at, v in enumerate((2.0 ** 24, 1.0, -2.0 ** 24)):
        dy[512 * at:512 * (at + 1)] = v
    h, dw = torch.ones_like(dy), torch.empty(N, device="cuda")
    space = torch.empty(g.sgemm_norm_grad_workspace_size(1536, N), dtype=torch.uint8, device="cuda")
    g.sgemm_norm_grad(1536, N, h, N, None, 0.0, dy, N, None, N, None, N, 0.0, dw, space)
    assert bool((dw == 512.0).all())


@pytest.mark.parametrize("T,N", [(512, 8194), (513, 8194), (2100, 8195)])
def test_norm_grad_of_many_long_rows(T, N):
    """Rows too long for registers, one to a share, two, and more than a turn takes."""
    gu.say("norm_grad of long rows", T, N)
    eps = 2.0 ** -12
    r = rng_of(60, T, N)
    h = stream(T, N, 8, special=False)
    h[T // 3] = 0.0
    dy, ds = (r.standard_normal((T, N)).astype(np.float32) for _ in range(2))
    w, start = (r.standard_normal(N).astype(np.float32) for _ in range(2))
    H, DS, W = Buffer(h, N + 1), Buffer(ds, N + 3), Buffer(w)
    need = g.sgemm_norm_grad_workspace_size(T, N)
    for streamed, beta in ((True, 0.0), (False, 0.5)):
        want, size, dw, dw_size = bo.norm_grad(h, w if streamed else None, eps, dy, ds if streamed else None)
        first = None
        for parts in ("both", "in place", "dh", "dweight"):
            space = torch.full((need + 1024,), 0xFF, dtype=torch.uint8, device="cuda")  # NaN
            DY, DW = Buffer(dy, N + 2), Buffer(np.full(N, NAN, np.float32) if beta == 0 else start)
            DH = DY if parts == "in place" else floats(T, N, ld=N + 2)
            g.sgemm_norm_grad(T, N, H.ptr, H.ld, W.ptr if streamed else None, eps, DY.ptr, DY.ld,
                              DS.ptr if streamed else None, DS.ld, DH.ptr if parts != "dweight" else None, DH.ld, beta,
                              DW.ptr if parts != "dh" else None, space if parts != "dh" else None, need)
            torch.cuda.synchronize()
            assert bool((space[need:] == 0xFF).all()), "beyond the workspace"
            if parts != "dweight":
                within(DH.read(), want, np.abs(want) + 2.0 ** -21 * size, ONCE, "dh")
            if parts != "dh":
                got = DW.read()
                within(got, dw + beta * start, dw_size + np.abs(beta * start), 2.02 * U24, "dweight")
                assert first is None or np.array_equal(got, first)
                first = got


@pytest.mark.parametrize("T,N,weight", [(3700, 9101, False), (400, 90001, True)])
def test_norm_grad_of_rows_larger_than_the_caches(T, N, weight):
    """dh's stores go past the caches: the same numbers, and nothing behind a row is written."""
    gu.say("norm_grad of large rows", T, N)
    gen = torch.Generator(device="cuda").manual_seed(7)
    h, dy, ds = (torch.randn(T, N, generator=gen, device="cuda") for _ in range(3))
    w = torch.randn(N, generator=gen, device="cuda")
    own, dw = torch.full((T, N + 1), 7.0, device="cuda"), torch.empty(N, device="cuda")
    dh = own[:, :N]
    space = torch.empty(g.sgemm_norm_grad_workspace_size(T, N), dtype=torch.uint8, device="cuda")
    g.sgemm_norm_grad(T, N, h, N, w, 2.0 ** -12, dy, N, ds, N, dh, N + 1, 0.0, dw if weight else None, space)
    assert bool((own[:, N] == 7.0).all())
    g64, h64 = dy.double() * w.double(), h.double()
    r = torch.rsqrt(h64.square().mean(1, keepdim=True) + 2.0 ** -12)
    part = h64 * r * r
    want = r * (g64 - part * (g64 * h64).mean(1, keepdim=True)) + ds.double()
    size = r * (g64.abs() + part.abs() * (g64 * h64).abs().mean(1, keepdim=True)) + ds.abs()
    # one rounding, and 2^-45 of the terms for what cancels in 64 bits
    assert bool(((dh.double() - want).abs() <= ONCE * (want.abs() + 2.0 ** -21 * size)).all())
    if weight:
        terms = dy.double() * h64 * r
        assert bool(((dw.double() - terms.sum(0)).abs() <= 2.02 * U24 * terms.abs().sum(0)).all())


def test_norm_grad_of_long_rows_in_a_graph():
    """Captured on a stream of its own and replayed on other inputs, between eager calls."""
    T, N = 770, 8195
    gu.say("norm_grad of long rows in a graph")
    gen = torch.Generator(device="cuda").manual_seed(6)
    h, dy = (torch.randn(T, N, generator=gen, device="cuda") for _ in range(2))
    dh, dw = torch.empty(T, N, device="cuda"), torch.empty(N, device="cuda")
    space, other = (torch.empty(g.sgemm_norm_grad_workspace_size(T, N), dtype=torch.uint8, device="cuda") for _ in range(2))

    def call(dh, dw, space):
        g.sgemm_norm_grad(T, N, h, N, None, 1e-5, dy, N, None, N, dh, N, 0.0, dw, space)
    side, graph = torch.cuda.Stream(), torch.cuda.CUDAGraph()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        call(dh, dw, space)
        side.synchronize()
        with torch.cuda.graph(graph, stream=side):
            call(dh, dw, space)
    torch.cuda.synchronize()
    want_dh, want_dw = torch.empty_like(dh), torch.empty_like(dw)
    for turn in range(3):
        h.mul_(-0.75).add_(0.01 * turn)
        graph.replay()
        torch.cuda.synchronize()
        call(want_dh, want_dw, other)
        torch.cuda.synchronize()
        assert torch.equal(dh, want_dh) and torch.equal(dw, want_dw), turn
        space.fill_(0xFF)
        dw.zero_()


# ---------------------------------------------------------------------------
# large tiles: remainders in every direction, strides, beta
# ---------------------------------------------------------------------------
LARGE_I8 = [(2313, 3337, 70), (2313, 3341, 129), (2700, 3205, 400)]


@pytest.mark.parametrize("M,N,K", LARGE_I8)
def test_i8_of_large_products(M, N, K):
    """256 x 256 tiles; C's rows on half lines, where its stores go past the caches, and not."""
    gu.say("large i8", M, N, K)
    r = rng_of(61, M, N, K)
    A, B = (r.integers(-128, 128, s).astype(np.int8) for s in ((M, K), (N, K)))
    sa, sb = (np.exp(r.standard_normal(n)).astype(np.float32) / 127 for n in (M, N))
    C0 = r.standard_normal((M, N)).astype(np.float32)
    SA, SB = Buffer(sa), Buffer(sb)
    word = -(-K // 4) * 4
    a, b = Bytes(A, word + 4, 4), Bytes(B, word, 0)
    for alpha, beta, scaled in ((1.0, 0.0, True), (-0.75, 0.5, True), (2.0, 1.0, False)):
        want, size = bo.i8(A, sa if scaled else None, B, sb if scaled else None, alpha, beta, C0)
        for ldc, offset in ((-(-N // 16) * 16, 0), (N + 3, 0), (-(-N // 16) * 16, 5)):
            C = Buffer(C0 if beta else np.full((M, N), NAN, np.float32), ldc, offset)
            g.sgemm_i8(M, N, K, alpha, a.ptr, a.ld, SA.ptr if scaled else None, b.ptr, b.ld,
                       SB.ptr if scaled else None, beta, C.ptr, ldc)
            torch.cuda.synchronize()
            within(C.read(), want, np.abs(want) + 2.0 ** -26 * size, ONCE, f"ldc {ldc} offset {offset} beta {beta}")
    nan = Buffer(np.full(max(M, N), NAN, np.float32))
    for alpha, k in ((0.0, K), (1.0, 0)):  # the operands and the scales are not read
        C = Buffer(C0, N + 3)
        g.sgemm_i8(M, N, k, alpha, None, word, nan.ptr, None, word, nan.ptr, -0.5, C.ptr, C.ld)
        torch.cuda.synchronize()
        assert np.array_equal(C.read(), np.float32(-0.5) * C0)


LARGE_GATED = [(2251, 651, 67), (2251, 651, 5), (1801, 3351, 67), (1801, 3351, 32)]


@pytest.mark.parametrize("T,N,K", LARGE_GATED)
def test_gated_of_many_rows(T, N, K):
    """128 x 64 and 256 x 128 tiles of y."""
    for kind, pad in ((0, 1), (1, 0), (2, 4)):
        gu.say("gated of many rows", T, N, K, kind)
        x, G, U = operands(T, N, K, kind)
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
    x[1, K - 1], G[K - 2, 7], U[0, 9] = np.nan, np.inf, np.nan  # stay in their row and columns
    X, GB, UB, Y = Buffer(x, K + 1), Buffer(G, N + 1), Buffer(U, N + 1), floats(T, N)
    g.sgemm_gated(T, N, K, kind, X.ptr, X.ld, GB.ptr, GB.ld, UB.ptr, UB.ld, Y.ptr, Y.ld, None, N, None, N)
    torch.cuda.synchronize()
    y = Y.read()
    rest = np.ones((T, N), bool)
    rest[1], rest[:, 7], rest[:, 9] = False, False, False
    assert np.isnan(y[1]).all() and np.isnan(y[:, 9]).all() and np.isfinite(y[rest]).all()


LARGE_WEIGHTS = [(70, 2701, 2201), (33, 2701, 2201)]


@pytest.mark.parametrize("T,N,K", LARGE_WEIGHTS)
def test_gated_grad_of_large_weights(T, N, K):
    """dG and dU in 256 x 256 tiles."""
    r = rng_of(62, T, N, K)
    x, G, U = operands(T, N, K, 5)
    gate, up, dy = (r.standard_normal((T, N)).astype(np.float32) for _ in range(3))
    start = [r.standard_normal((K, N)).astype(np.float32) for _ in range(2)]
    nan = np.full((K, N), NAN, np.float32)
    for kind, pad, beta, parts in ((0, 0, 0.0, "both"), (1, 1, 0.5, "weights"), (2, 4, 1.0, "both")):
        gu.say("gated_grad of large weights", T, N, K, kind)
        grads, sizes = bo.gated_grad(kind, x, G, U, gate, up, dy)
        got = backward(kind, x, G, U, gate, up, dy, beta, *((nan, nan) if beta == 0 else start), pad, parts)
        if parts == "both":
            within(got[0], grads[0], sizes[0], SUM, "dx")
        for name, have, want, size, old in zip(("dG", "dU"), got[1:], grads[1:], sizes[1:], start):
            within(have, want + beta * old.astype(np.float64), size + beta * np.abs(old), SUM, name)


# few rows and a long K: 32 x 32 tiles of dx; dx alone of some hundred rows on 32 x 64 tiles
MORE_GATED = [(30, 33, 4200), (338, 100, 2571)]


@pytest.mark.parametrize("T,N,K", MORE_GATED)
def test_gated_grad_of_more_sizes(T, N, K):
    tb.test_gated_grad(T, N, K)


MORE_ROWS = [(5, 300), (3, 511), (3, 5000), (2, 8191)]


@pytest.mark.parametrize("kind", [0, 1, 2])
@pytest.mark.parametrize("T,N", MORE_ROWS)
def test_quantize_gated_of_more_columns(T, N, kind):
    tb.test_quantize_gated(T, N, kind)


# ---------------------------------------------------------------------------
# what is launched
# ---------------------------------------------------------------------------
class Dim3(ctypes.Structure):
    _fields_ = [(name, ctypes.c_uint) for name in "xyz"]


class KernelNode(ctypes.Structure):  # hipKernelNodeParams
    _fields_ = [("block", Dim3), ("extra", ctypes.c_void_p), ("func", ctypes.c_void_p), ("grid", Dim3),
                ("params", ctypes.c_void_p), ("shared", ctypes.c_uint)]


def recorded(call, stream):
    """The names of the kernels that a call launches on a stream: they are recorded into a graph, and
    the graph is dropped."""
    lib, vp = g.load_library(), ctypes.c_void_p  # (its look-ups find the HIP library it is linked to)

    def hip(name, *args):
        assert getattr(lib, name)(*args) == 0, name
    hip("hipStreamBeginCapture", vp(stream), 1)  # this thread's calls only
    status, graph, n = ctypes.c_int(0), vp(), ctypes.c_size_t(0)
    try:
        hip("hipStreamIsCapturing", vp(stream), ctypes.byref(status))
        assert status.value == 1
        call()
    finally:
        hip("hipStreamEndCapture", vp(stream), ctypes.byref(graph))
    hip("hipGraphGetNodes", graph, None, ctypes.byref(n))
    nodes, names = (vp * n.value)(), []
    hip("hipGraphGetNodes", graph, nodes, ctypes.byref(n))
    name_of = lib.hipKernelNameRefByPtr
    name_of.restype = ctypes.c_char_p
    for node in nodes:
        of = KernelNode()
        hip("hipGraphKernelNodeGetParams", vp(node), ctypes.byref(of))
        names.append(name_of(vp(of.func), vp(stream)).decode())
    hip("hipGraphDestroy", graph)
    return names


def sizes_of(test, names):
    return [s for m in test.pytestmark if m.name == "parametrize" and m.args[0] == names for s in m.args[1]]


def test_every_kernel_is_launched_by_a_tested_size():
    """A choice that is priced anew can take a kernel's only sizes away from it: then this names the
    kernel.  One buffer stands for all operands, as large as the largest (nothing runs on it)."""
    gu.say("recorded")
    room = torch.empty(1 << 28, dtype=torch.uint8, device="cuda")
    p, side = room.data_ptr(), torch.cuda.Stream()
    s = side.cuda_stream
    seen = set()

    def add(fn, *args):
        seen.update(recorded(lambda: fn(*args, stream=s), s))

    for T, N in tb.NORMS:
        add(g.sgemm_norm, T, N, p, N, None, N, None, 1.0, None, N, p, N, p, N, p)
        add(g.sgemm_quantize, T, N, p, N, 0, None, N, p, N, p)
    for T, N in sizes_of(tb.test_norm_grad, "T,N") + sizes_of(test_norm_grad_of_many_long_rows, "T,N"):
        add(g.sgemm_norm_grad, T, N, p, N, None, 1.0, p, N, None, N, p, N, 0.0, p, p, 1 << 28)
    for T, N in sizes_of(tb.test_quantize_gated, "T,N") + MORE_ROWS:
        for kind in range(3):
            add(g.sgemm_quantize, T, N, p, N, kind, p, N, p, N, p)
    for M, N, K in tb.I8S + LARGE_I8:
        for ld in (-(-K // 4) * 4, K + 1):
            add(g.sgemm_i8, M, N, K, 1.0, p, ld, None, p, ld, None, 0.0, p, N + 3)
    far = 2_100_000  # the strides of test_gated_with_strides_beyond_the_fast_kernels
    for T, N, K, ldx in [(*size, size[2]) for size in tb.GATED + LARGE_GATED + LARGE_WEIGHTS + MORE_GATED] + [(5, 9, 6, far)]:
        add(g.sgemm_gated, T, N, K, 0, p, ldx, p, N, p, N, p, N, p, N, p, N)
        for kind, dx, dw in ((0, p, p), (1, p, None), (2, None, p)):
            add(g.sgemm_gated_grad, T, N, K, kind, p, ldx, p, N, p, N, p, N, p, N, p, N, dx, K, 0.0, dw, N, dw, N, p, 1 << 28)
    held = set(build.kernel_resources(source=2)) | {k for k in build.kernel_resources(source=1) if "thin_twice" in k}
    assert len(held) > 80
    missing = sorted(held - seen)
    assert not missing, build.demangle(missing)
