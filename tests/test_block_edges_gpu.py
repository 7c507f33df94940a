"""Corners of a feed-forward block's operators that their parametrised tests do not reach: strides
that 32-bit offsets do not reach, rows billions of elements apart, streams, graphs, what the binding
refuses, and runs of the operators together, in FP32 with gradients and in 8 bits.

Tolerances are those of test_block_gpu; of a run of products one after the other, 1e-5 of the
result's size for each (the errors of one enter the next as a perturbation of its input)."""
import numpy as np
import pytest
import torch

import fp32_gemm_03_amd as g
from tests import block_oracle as bo
from tests import gpu_util as gu
from tests.test_block_gpu import ONCE, SUM, Bytes, check_forward, floats, operands, stream
from tests.test_rows_gpu import NAN, Buffer, rng_of, within

pytestmark = pytest.mark.gpu


@pytest.fixture(autouse=True)
def _gpu_available():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")


def spread(data, ld, kind):
    """The rows of a host matrix ld elements apart, on the GPU (the rest is left as it comes)."""
    data = torch.from_numpy(np.ascontiguousarray(data)).to(kind)
    owner = torch.empty((data.shape[0] - 1) * ld + data.shape[1], dtype=kind, device="cuda")
    view = owner.as_strided(data.shape, (ld, 1))
    view.copy_(data)
    return owner, view


# ---------------------------------------------------------------------------
# strides
# ---------------------------------------------------------------------------
@pytest.mark.parametrize("wide", ["A", "B", "C"])
def test_i8_with_strides_beyond_the_fast_kernels(wide):
    M, N, K = 5, 7, 70
    gu.say("i8 wide", wide)
    r = rng_of(30)
    A, B = (r.integers(-128, 128, s).astype(np.int8) for s in ((M, K), (N, K)))
    lda, ldb = (9_000_000 if wide == n else 72 for n in "AB")
    ldc = 2_200_000 if wide == "C" else N
    a, _ = spread(A, lda, torch.int8)
    b, _ = spread(B, ldb, torch.int8)
    c, C = spread(np.zeros((M, N), np.float32), ldc, torch.float32)
    g.sgemm_i8(M, N, K, 1.0, a, lda, None, b, ldb, None, 0.0, c, ldc)
    assert np.array_equal(C.cpu().numpy(), A.astype(np.float64) @ B.astype(np.float64).T)


@pytest.mark.parametrize("wide", ["x", "G", "U"])
def test_gated_with_strides_beyond_the_fast_kernels(wide):
    T, N, K = 5, 9, 6
    gu.say("gated wide", wide)
    x, G, U = operands(T, N, K, 1)
    ldx, ldg, ldu = (2_100_000 if wide == n else d for n, d in (("x", K), ("G", N), ("U", N)))
    (xo, _), (go, _), (uo, _) = (spread(v, ld, torch.float32) for v, ld in ((x, ldx), (G, ldg), (U, ldu)))
    y, gate, up = (torch.empty(T, N, device="cuda") for _ in range(3))
    g.sgemm_gated(T, N, K, 2, xo, ldx, go, ldg, uo, ldu, y, N, gate, N, up, N)
    check_forward(2, x, G, U, *(v.cpu().numpy() for v in (y, gate, up)))
    dy = rng_of(31).standard_normal((T, N)).astype(np.float32)
    dx, dG, dU = torch.empty(T, K, device="cuda"), *(torch.full((K, N), 2.0, device="cuda") for _ in range(2))
    space = torch.empty(g.sgemm_gated_grad_workspace_size(T, N, K), dtype=torch.uint8, device="cuda")
    g.sgemm_gated_grad(T, N, K, 2, xo, ldx, go, ldg, uo, ldu, gate, N, up, N, torch.from_numpy(dy).cuda(), N, dx, K, 0.5,
                       dG, N, dU, N, space)
    grads, sizes = bo.gated_grad(2, x, G, U, gate.cpu().numpy(), up.cpu().numpy(), dy)
    for got, want, size, old in zip((dx, dG, dU), grads, sizes, (0.0, 1.0, 1.0)):
        within(got.cpu().numpy(), want + old, size + old, SUM, "gradient")


@pytest.mark.parametrize("N", [200, 20000])
def test_rows_billions_of_elements_apart(N):
    """The second row of a matrix whose leading dimension is the largest int."""
    gu.say("far rows", N)
    ld = 2 ** 31 - 1
    x = stream(2, N, 40, special=False)
    far, view = spread(x, ld, torch.float32)
    h, y = bo.norm(x, None, None, 0.5)
    out, q, s = torch.empty(2, N, device="cuda"), torch.empty(2, N, dtype=torch.int8, device="cuda"), torch.empty(2, device="cuda")
    g.sgemm_norm(2, N, far, ld, None, ld, None, 0.5, None, ld, out, N, q, N, s)
    within(out.cpu().numpy(), y, np.abs(y), ONCE, "y")
    g.sgemm_quantize(2, N, far, ld, 0, None, N, q, N, s)
    want_q, want_s = bo.quantize(x)
    assert np.array_equal(q.cpu().numpy(), want_q) and np.array_equal(s.cpu().numpy(), want_s)
    dh = torch.empty(2, N, device="cuda")
    g.sgemm_norm_grad(2, N, far, ld, None, 0.5, out, N, None, N, dh, N, 0.0, None)
    want, size, _, _ = bo.norm_grad(x, None, 0.5, out.cpu().numpy(), None)
    within(dh.cpu().numpy(), want, np.abs(want) + 2.0 ** -21 * size, ONCE, "dh")
    g.sgemm_norm(2, N, out, N, None, N, None, 0.5, far, ld, None, N, None, N, None)  # sum written far apart
    assert torch.equal(view, out)


def test_many_rows():
    """More rows than a grid of 16 bits, and shares of dweight of more rows than one."""
    T, N = 70001, 20
    x = stream(T, N, 41, special=False)
    h, y = bo.norm(x, None, None, 0.5)
    X, Y = Buffer(x), floats(T, N)
    g.sgemm_norm(T, N, X.ptr, N, None, N, None, 0.5, None, N, Y.ptr, N, None, N, None)
    torch.cuda.synchronize()
    within(Y.read(), y, np.abs(y), ONCE, "y")
    want, size, dw, dw_size = bo.norm_grad(x, None, 0.5, x, None)
    DW = Buffer(np.full(N, NAN, np.float32))
    space = torch.empty(g.sgemm_norm_grad_workspace_size(T, N), dtype=torch.uint8, device="cuda")
    g.sgemm_norm_grad(T, N, X.ptr, N, None, 0.5, X.ptr, N, None, N, None, N, 0.0, DW.ptr, space)
    torch.cuda.synchronize()
    within(DW.read(), dw, dw_size, 2 * 2.0 ** -24, "dweight")


def test_the_same_projection_twice():
    """G and U one matrix: y = act(x G) (x G), and both its gradients."""
    T, N, K = 37, 70, 50
    x, G, _ = operands(T, N, K, 3)
    X, GB = Buffer(x), Buffer(G)
    Y, gate, up = floats(T, N), floats(T, N), floats(T, N)
    g.sgemm_gated(T, N, K, 0, X.ptr, K, GB.ptr, N, GB.ptr, N, Y.ptr, N, gate.ptr, N, up.ptr, N)
    torch.cuda.synchronize()
    check_forward(0, x, G, G, Y.read(), gate.read(), up.read())
    assert np.array_equal(gate.read(), up.read())


# ---------------------------------------------------------------------------
# streams and graphs
# ---------------------------------------------------------------------------
def everything(T, N, K, seed):
    """One call of each operator on buffers of its own: the calls, and what they write."""
    gen = torch.Generator(device="cuda").manual_seed(seed)
    rnd = lambda *s: torch.randn(*s, generator=gen, device="cuda")  # noqa: E731
    x, r, w, dy, ds = rnd(T, K), rnd(T, K), rnd(K), rnd(T, K), rnd(T, K)
    G, U, dz = rnd(K, N) / K ** 0.5, rnd(K, N) / K ** 0.5, rnd(T, N)
    out = {n: torch.zeros(*s, device="cuda") for n, s in dict(
        sum=(T, K), y=(T, K), dh=(T, K), dw=(K,), z=(T, N), gate=(T, N), up=(T, N), dx=(T, K), dG=(K, N), dU=(K, N),
        C=(T, N), s=(T,), s2=(T,), sb=(N,)).items()}
    out |= {n: torch.zeros(*s, dtype=torch.int8, device="cuda") for n, s in dict(q=(T, K), q2=(T, N), qb=(N, K)).items()}
    B = rnd(N, K)
    space = torch.empty(max(g.sgemm_norm_grad_workspace_size(T, K), g.sgemm_gated_grad_workspace_size(T, N, K)),
                        dtype=torch.uint8, device="cuda")
    o = out

    def calls(stream=None):
        g.sgemm_norm(T, K, x, K, r, K, w, 1e-5, o["sum"], K, o["y"], K, o["q"], K, o["s"], stream=stream)
        g.sgemm_quantize(N, K, B, K, 0, None, K, o["qb"], K, o["sb"], stream=stream)
        g.sgemm_i8(T, N, K, 1.0, o["q"], K, o["s"], o["qb"], K, o["sb"], 0.0, o["C"], N, stream=stream)
        g.sgemm_gated(T, N, K, 0, o["y"], K, G, N, U, N, o["z"], N, o["gate"], N, o["up"], N, stream=stream)
        g.sgemm_quantize(T, N, o["up"], N, 0, o["gate"], N, o["q2"], N, o["s2"], stream=stream)
        g.sgemm_gated_grad(T, N, K, 0, o["y"], K, G, N, U, N, o["gate"], N, o["up"], N, dz, N, o["dx"], K, 0.0, o["dG"], N,
                           o["dU"], N, space, stream=stream)
        g.sgemm_norm_grad(T, K, o["sum"], K, w, 1e-5, o["dx"], K, ds, K, o["dh"], K, 0.0, o["dw"], space, stream=stream)
    return calls, out, (x, r, dz)


@pytest.mark.parametrize("T,N,K", [(1, 64, 256), (40, 520, 132), (300, 260, 516)])
def test_streams(T, N, K):
    """The same bits on torch's current stream, on a stream given, and on its raw handle."""
    calls, out, _ = everything(T, N, K, 1)
    calls()
    torch.cuda.synchronize()
    want = {n: v.clone() for n, v in out.items()}
    side = torch.cuda.Stream()
    for given in (side, side.cuda_stream, None):
        for v in out.values():
            v.zero_()
        torch.cuda.synchronize()
        if given is None:
            with torch.cuda.stream(side):
                calls()
        else:
            calls(given)
        side.synchronize()
        assert all(torch.equal(out[n], want[n]) for n in out), given


def test_two_streams_at_once():
    """Every operator on two streams, a workspace each: the bits that each has alone."""
    sets = [everything(300, 260, 516, 3), everything(130, 516, 260, 4)]
    want = []
    for calls, out, _ in sets:
        calls()
        torch.cuda.synchronize()
        want.append({n: v.clone() for n, v in out.items()})
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    for _, out, _ in sets:
        for v in out.values():
            v.zero_()
    torch.cuda.synchronize()
    for _ in range(5):
        for (calls, _, _), stream in zip(sets, streams):
            calls(stream)
    torch.cuda.synchronize()
    for (_, out, _), w in zip(sets, want):
        assert all(torch.equal(out[n], w[n]) for n in out)


@pytest.mark.parametrize("T,N,K", [(1, 64, 256), (40, 520, 132), (300, 260, 516)])
def test_graphs(T, N, K):
    """Captured once, replayed on new inputs between eager calls of another set that shares nothing."""
    calls, out, inputs = everything(T, N, K, 2)
    other, _, _ = everything(T, N, K, 3)
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        calls()
        side.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=side):
            calls()
    torch.cuda.synchronize()
    for turn in range(4):
        for v in inputs:
            v.mul_(-0.75).add_(0.01 * turn)
        for v in out.values():
            v.zero_()
        graph.replay()
        other()
        torch.cuda.synchronize()
        got = {n: v.clone() for n, v in out.items()}
        calls()
        torch.cuda.synchronize()
        assert all(torch.equal(out[n], got[n]) for n in out), turn


# ---------------------------------------------------------------------------
# what the binding refuses
# ---------------------------------------------------------------------------
def test_tensors_that_do_not_fit_are_refused():
    T, N, K = 4, 8, 12
    f = lambda *s: torch.zeros(*s, device="cuda")  # noqa: E731
    b = lambda *s: torch.zeros(*s, dtype=torch.int8, device="cuda")  # noqa: E731
    norm = [T, N, f(T, N), N, f(T, N), N, f(N), 1e-5, f(T, N), N, f(T, N), N, b(T, N), N, f(T)]
    i8 = [T, N, K, 1.0, b(T, K), K, f(T), b(N, K), K, f(N), 0.0, f(T, N), N]
    gated = [T, N, K, 0, f(T, K), K, f(K, N), N, f(K, N), N, f(T, N), N, f(T, N), N, f(T, N), N]
    for fn, args in ((g.sgemm_norm, norm), (g.sgemm_i8, i8), (g.sgemm_gated, gated)):
        fn(*args)
        for at, v in enumerate(args):
            if not isinstance(v, torch.Tensor):
                continue
            short = v.reshape(-1)[:-1]
            other = v.to(torch.float64) if v.dtype is torch.float32 else v.to(torch.uint8)
            for bad, error in ((short, ValueError), (other, TypeError), (v.cpu(), TypeError)):
                with pytest.raises(error):
                    fn(*args[:at], bad, *args[at + 1:])
            if v.dim() == 2:
                with pytest.raises(ValueError):
                    fn(*args[:at], torch.zeros(v.shape[1], v.shape[0], dtype=v.dtype, device="cuda").t(), *args[at + 1:])
    with pytest.raises(ValueError):
        g.sgemm_norm_grad(T, N, f(T, N), N, None, 0.0, f(T, N), N, None, N, None, N, 0.0, f(N), f(64), -1)
    torch.cuda.synchronize()


# ---------------------------------------------------------------------------
# runs of the operators together
# ---------------------------------------------------------------------------
@pytest.mark.parametrize("T,K,F,kind", [(1, 96, 160, 0), (33, 130, 97, 1), (300, 128, 260, 2)])
def test_a_block_in_fp32_and_back(T, K, F, kind):
    """norm, gated projections, the projection down and the residual's addition; and the gradients
    of every input and weight, against the formulas' in 64 bits on the CPU."""
    gu.say("block", T, K, F, kind)
    gen = torch.Generator().manual_seed(5)
    rnd = lambda *s: torch.randn(*s, generator=gen, dtype=torch.float64)  # noqa: E731
    host = dict(x=rnd(T, K), res=rnd(T, K), w=1 + 0.2 * rnd(K), G=rnd(K, F) / K ** 0.5, U=rnd(K, F) / K ** 0.5,
                D=rnd(F, K) / F ** 0.5, dout=rnd(T, K))
    host = {n: v.float().double() for n, v in host.items()}
    d = {n: v.float().cuda() for n, v in host.items()}
    e = lambda *s: torch.empty(*s, device="cuda")  # noqa: E731
    h, y, z, gate, up, out = e(T, K), e(T, K), e(T, F), e(T, F), e(T, F), e(T, K)
    eps = 2.0 ** -17
    g.sgemm_norm(T, K, d["x"], K, d["res"], K, d["w"], eps, h, K, y, K, None, K, None)
    g.sgemm_gated(T, F, K, kind, y, K, d["G"], F, d["U"], F, z, F, gate, F, up, F)
    out.copy_(h)
    g.sgemm(T, K, F, 1.0, z, F, d["D"], K, 1.0, out, K)
    dz, dy, dh, dw, dG, dU = e(T, F), e(T, K), e(T, K), e(K), e(K, F), e(K, F)
    dD = e(F, K)
    g.sgemm(T, F, K, 1.0, d["dout"], K, d["D"].t().contiguous(), F, 0.0, dz, F)
    g.sgemm(F, K, T, 1.0, z.t().contiguous(), T, d["dout"], K, 0.0, dD, K)
    space = torch.empty(max(256, g.sgemm_gated_grad_workspace_size(T, F, K), g.sgemm_norm_grad_workspace_size(T, K)),
                        dtype=torch.uint8, device="cuda")
    g.sgemm_gated_grad(T, F, K, kind, y, K, d["G"], F, d["U"], F, gate, F, up, F, dz, F, dy, K, 0.0, dG, F, dU, F, space)
    g.sgemm_norm_grad(T, K, h, K, d["w"], eps, dy, K, d["dout"], K, dh, K, 0.0, dw, space)
    # 64 bits
    leaf = {n: v.clone().requires_grad_(n != "dout") for n, v in host.items()}
    hh = leaf["x"] + leaf["res"]
    yy = hh * torch.rsqrt(hh.square().mean(1, keepdim=True) + eps) * leaf["w"]
    gg = yy @ leaf["G"]
    f = torch.nn.functional
    a = f.silu(gg) if kind == 0 else f.gelu(gg, approximate="tanh" if kind == 2 else "none")
    oo = hh + (a * (yy @ leaf["U"])) @ leaf["D"]
    oo.backward(leaf["dout"])
    for name, got, want in (("out", out, oo.detach()), ("dx", dh, leaf["x"].grad), ("dres", dh, leaf["res"].grad),
                            ("dw", dw, leaf["w"].grad), ("dG", dG, leaf["G"].grad), ("dU", dU, leaf["U"].grad),
                            ("dD", dD, leaf["D"].grad)):
        far = (got.double().cpu() - want).norm() / want.norm()
        assert far < 6 * SUM, (name, float(far))  # at most six products and norms one after the other


@pytest.mark.parametrize("T,K,F,kind", [(1, 96, 160, 0), (33, 130, 97, 2), (300, 128, 260, 1)])
def test_a_block_in_8_bits(T, K, F, kind):
    """norm to 8 bits, one product of gate's and up's channels, the activation to 8 bits, the product
    down onto the residual stream: each step against its definition on what the last one wrote."""
    gu.say("block in 8 bits", T, K, F, kind)
    r = rng_of(50, T, K, F)
    x, res = (r.standard_normal((T, K)).astype(np.float32) for _ in range(2))
    GU, D = r.standard_normal((2 * F, K)).astype(np.float32), r.standard_normal((K, F)).astype(np.float32)
    up4 = lambda n: -(-n // 4) * 4  # noqa: E731
    X, R, W1, W2 = Buffer(x), Buffer(res), Buffer(GU), Buffer(D)
    B, sb, B2, sb2 = Bytes(np.zeros((2 * F, K)), up4(K)), floats(2 * F), Bytes(np.zeros((K, F)), up4(F)), floats(K)
    g.sgemm_quantize(2 * F, K, W1.ptr, K, 0, None, K, B.ptr, B.ld, sb.ptr)
    g.sgemm_quantize(K, F, W2.ptr, F, 0, None, F, B2.ptr, B2.ld, sb2.ptr)
    S, Q, s = floats(T, K), Bytes(np.zeros((T, K)), up4(K)), floats(T)
    H, Q2, s2 = floats(T, 2 * F), Bytes(np.zeros((T, F)), up4(F)), floats(T)
    g.sgemm_norm(T, K, X.ptr, K, R.ptr, K, None, 1e-5, S.ptr, K, None, K, Q.ptr, Q.ld, s.ptr)
    torch.cuda.synchronize()
    total = S.read()
    g.sgemm_i8(T, 2 * F, K, 1.0, Q.ptr, Q.ld, s.ptr, B.ptr, B.ld, sb.ptr, 0.0, H.ptr, 2 * F)
    g.sgemm_quantize(T, F, H.ptr + 4 * F, 2 * F, kind, H.ptr, 2 * F, Q2.ptr, Q2.ld, s2.ptr)
    g.sgemm_i8(T, K, F, 1.0, Q2.ptr, Q2.ld, s2.ptr, B2.ptr, B2.ld, sb2.ptr, 1.0, S.ptr, K)
    torch.cuda.synchronize()
    assert np.array_equal(total, x + res)
    want, _ = bo.i8(Q.read(), s.read(), B.read(), sb.read(), 1.0, 0.0, None)
    h = H.read()
    within(h, want, np.abs(want), ONCE, "H")
    v = bo.act(kind, h[:, :F])[0] * h[:, F:].astype(np.float64)
    q, scale = Q2.read(), s2.read().astype(np.float64)[:, None]
    most = np.abs(v).max(1, keepdims=True)
    assert (np.abs(q - 127 * v / most) <= 0.5 + 127 * 3 * 2.0 ** -24).all() and (np.abs(scale * 127 / most - 1) < 3 * 2.0 ** -24).all()
    want, size = bo.i8(q, s2.read(), B2.read(), sb2.read(), 1.0, 1.0, total)
    within(S.read(), want, np.abs(want) + 2.0 ** -26 * size, ONCE, "out")
