"""The refusals of the calls around products whose B is picked row by row, on the CPU: every
call below stops at an argument check or a documented quick return, before any HIP call.  And the
64-bit plain forms' gradients against differences."""
import ctypes

import numpy as np
import pytest

import fp32_gemm_03_amd as g
from tests import rows_oracle as ro

P = 0x10000  # a fake device address, never dereferenced


def refuse(fn, base, bad, position):
    args = dict(base)
    args.update(bad)
    code = fn(*args.values(), stream=0, check=False)
    assert code == -(100 + position), (bad, code)
    assert g.sgemm_status_string(code) == f"invalid argument {position}"
    with pytest.raises(g.SgemmError):
        fn(*args.values(), stream=0)


ROUTE = dict(T=4, E=8, k=2, scoring=0, logits=P, ldl=8, bias=None, groups=2, top_groups=1, group_best=1, renorm=1,
             scale=1.0, ids=P, weights=P)


@pytest.mark.parametrize("bad,position", [
    (dict(T=-1), 1), (dict(E=0), 2), (dict(E=1025, ldl=1025), 2), (dict(k=0), 3), (dict(k=9), 3),
    (dict(E=128, ldl=128, k=65), 3), (dict(scoring=2), 4), (dict(logits=0), 5), (dict(ldl=7), 6),
    (dict(groups=0), 8), (dict(groups=3), 8), (dict(E=130, ldl=130, groups=65), 8), (dict(top_groups=0), 9),
    (dict(top_groups=3), 9), (dict(group_best=0), 10), (dict(group_best=3), 10), (dict(ids=0), 13), (dict(weights=0), 14),
    (dict(T=-1, E=0), 1)])
def test_route_refuses(bad, position):
    refuse(g.sgemm_route, ROUTE, bad, position)


GRAD = dict(T=4, E=8, k=2, scoring=1, logits=P, ldl=8, renorm=1, scale=1.0, ids=P, dweights=P, dlogits=P, lddl=8)


@pytest.mark.parametrize("bad,position", [
    (dict(T=-1), 1), (dict(E=0), 2), (dict(k=9), 3), (dict(scoring=-1), 4), (dict(logits=0), 5), (dict(ldl=7), 6),
    (dict(ids=0), 9), (dict(dweights=0), 10), (dict(dlogits=0), 11), (dict(lddl=7), 12)])
def test_route_grad_refuses(bad, position):
    refuse(g.sgemm_route_grad, GRAD, bad, position)


GROUP = dict(R=100000, G=8, ids=P, offsets=P, rows=P, workspace=P, workspace_bytes=1 << 20)


@pytest.mark.parametrize("bad,position", [
    (dict(R=-1), 1), (dict(G=0), 2), (dict(G=4097), 2), (dict(ids=0), 3), (dict(offsets=0), 4), (dict(rows=0), 5)])
def test_group_rows_refuses(bad, position):
    refuse(g.sgemm_group_rows, GROUP, bad, position)


def test_group_rows_refuses_a_workspace():
    need = g.sgemm_group_rows_workspace_size(100000, 8)
    assert need > 0 and g.sgemm_group_rows_workspace_size(64, 8) == 0
    assert g.sgemm_group_rows_workspace_size(-1, 8) == 0 and g.sgemm_group_rows_workspace_size(10, 4097) == 0
    for bad in (dict(workspace=0), dict(workspace=P + 128), dict(workspace_bytes=need - 1)):
        assert g.sgemm_group_rows(*{**GROUP, **bad}.values(), stream=0, check=False) == -24


GROUPED = dict(G=3, R=10, N=6, K=5, alpha=1.0, A=P, lda=5, a_div=1, B=P, ldb=6, stride_b=30, trans_b=0, beta=0.0, C=P,
               ldc=6, c_scatter=1, offsets=P, rows=P)


@pytest.mark.parametrize("bad,position", [
    (dict(G=-1), 1), (dict(R=-1), 2), (dict(N=-1), 3), (dict(K=-1), 4), (dict(A=0), 6), (dict(A=P + 2), 6),
    (dict(lda=4), 7), (dict(a_div=-1), 8), (dict(B=0), 9), (dict(B=P + 1), 9), (dict(ldb=5), 10),
    (dict(trans_b=1, ldb=4), 10), (dict(stride_b=-1), 11), (dict(C=0), 14), (dict(C=P + 3), 14), (dict(ldc=5), 15),
    (dict(offsets=0), 17), (dict(rows=0), 18), (dict(rows=0, a_div=0), 18), (dict(rows=0, c_scatter=0), 18)])
def test_grouped_refuses(bad, position):
    refuse(g.sgemm_grouped, GROUPED, bad, position)


def test_grouped_quick_returns():
    for bad in (dict(G=0, offsets=0), dict(R=0, A=0, C=0), dict(N=0, ldb=1, C=0), dict(alpha=0.0, beta=1.0, A=0, B=0),
                dict(K=0, beta=1.0, A=0, B=0)):
        assert g.sgemm_grouped(*{**GROUPED, **bad}.values(), stream=0) == 0


def test_grouped_refuses_a_grid_beyond_one_launch():
    big = dict(R=2 ** 31 - 1, N=2 ** 30, lda=5, ldb=2 ** 30, ldc=2 ** 30)
    assert g.sgemm_grouped(*{**GROUPED, **big}.values(), stream=0, check=False) == -22
    tn = dict(M=2 ** 30, N=2 ** 30, lda=2 ** 30, ldb=2 ** 30, ldc=2 ** 30, stride_c=2 ** 62)
    assert g.sgemm_grouped_tn(*{**TN, **tn}.values(), stream=0, check=False) == -22


TN = dict(G=3, R=10, M=5, N=6, alpha=1.0, A=P, lda=5, a_div=1, B=P, ldb=6, b_div=1, beta=0.0, C=P, ldc=6, stride_c=30,
          offsets=P, rows=P)


@pytest.mark.parametrize("bad,position", [
    (dict(G=-1), 1), (dict(R=-1), 2), (dict(M=-1), 3), (dict(N=-1), 4), (dict(A=0), 6), (dict(lda=4), 7),
    (dict(a_div=-1), 8), (dict(B=0), 9), (dict(ldb=5), 10), (dict(b_div=-2), 11), (dict(C=0), 13), (dict(C=P + 1), 13),
    (dict(ldc=5), 14), (dict(stride_c=29), 15), (dict(offsets=0), 16), (dict(rows=0), 17), (dict(rows=0, a_div=0), 17)])
def test_grouped_tn_refuses(bad, position):
    refuse(g.sgemm_grouped_tn, TN, bad, position)


def test_grouped_tn_quick_returns():
    for bad in (dict(G=0, C=0), dict(M=0, C=0), dict(N=0, C=0), dict(R=0, beta=1.0, A=0, B=0, offsets=0),
                dict(alpha=0.0, beta=1.0, A=0, B=0, offsets=0)):
        assert g.sgemm_grouped_tn(*{**TN, **bad}.values(), stream=0) == 0


COMBINE = dict(T=4, k=2, N=8, E=3, ids=P, weights=P, Y=P, ldy=8, beta=0.0, out=P, ldo=8)


@pytest.mark.parametrize("bad,position", [
    (dict(T=-1), 1), (dict(k=0), 2), (dict(k=65), 2), (dict(N=-1), 3), (dict(E=-1), 4), (dict(Y=0), 7),
    (dict(Y=P + 2), 7), (dict(ldy=7), 8), (dict(out=0), 10), (dict(ldo=7), 11)])
def test_combine_refuses(bad, position):
    refuse(g.sgemm_combine, COMBINE, bad, position)


CGRAD = dict(T=4, k=2, N=8, E=3, ids=P, weights=P, dout=P, ldd=8, Y=P, ldy=8, dY=P, lddy=8, dweights=P)


@pytest.mark.parametrize("bad,position", [
    (dict(T=-1), 1), (dict(k=0), 2), (dict(N=-1), 3), (dict(E=-1), 4), (dict(dout=0), 7), (dict(ldd=7), 8),
    (dict(Y=0), 9), (dict(ldy=7), 10), (dict(dY=P + 1), 11), (dict(lddy=7), 12)])
def test_combine_grad_refuses(bad, position):
    refuse(g.sgemm_combine_grad, CGRAD, bad, position)


def test_quick_returns():
    assert g.sgemm_route(*{**ROUTE, "T": 0, "logits": 0, "ids": 0, "weights": 0}.values(), stream=0) == 0
    assert g.sgemm_route_grad(*{**GRAD, "T": 0, "logits": 0}.values(), stream=0) == 0
    assert g.sgemm_combine(*{**COMBINE, "T": 0, "Y": 0, "out": 0}.values(), stream=0) == 0
    assert g.sgemm_combine(*{**COMBINE, "N": 0, "Y": 0, "out": 0}.values(), stream=0) == 0
    assert g.sgemm_combine_grad(*{**CGRAD, "dY": None, "dweights": None}.values(), stream=0) == 0


ADAPT = dict(M=4, N=6, K=5, alpha=1.0, A=P, lda=5, B=P, ldb=6, beta=0.0, C=P, ldc=6, G=3, rank=2, ids=P, ranks=None,
             scales=None, U=P, ldu=2, stride_u=10, V=P, ldv=6, stride_v=12, workspace=P, workspace_bytes=1 << 30)


@pytest.mark.parametrize("bad,position", [
    (dict(M=-1), 1), (dict(N=-1), 2), (dict(K=-1), 3), (dict(A=0), 5), (dict(lda=4), 6), (dict(B=0), 7),
    (dict(ldb=5), 8), (dict(C=0), 10), (dict(ldc=5), 11), (dict(G=0), 12), (dict(G=4097), 12), (dict(rank=0), 13),
    (dict(rank=257, ldu=257), 13), (dict(ids=0), 14), (dict(U=0), 17), (dict(ldu=1), 18), (dict(stride_u=-1), 19),
    (dict(V=0), 20), (dict(ldv=5), 21), (dict(stride_v=-1), 22)])
def test_adapters_refuses(bad, position):
    refuse(g.sgemm_adapters, ADAPT, bad, position)


AGRAD = dict(M=4, N=6, K=5, alpha=1.0, A=P, lda=5, B=P, ldb=6, dC=P, lddc=6, G=3, rank=2, ids=P, ranks=None, scales=None,
             U=P, ldu=2, stride_u=10, V=P, ldv=6, stride_v=12, beta=0.0, dA=P, ldda=5, dU=P, lddu=2, stride_du=10, dV=P,
             lddv=6, stride_dv=12, workspace=P, workspace_bytes=1 << 30)


@pytest.mark.parametrize("bad,position", [
    (dict(M=-1), 1), (dict(N=-1), 2), (dict(K=-1), 3), (dict(A=0), 5), (dict(lda=4), 6), (dict(B=0), 7), (dict(ldb=5), 8),
    (dict(dC=0), 9), (dict(lddc=5), 10), (dict(G=0), 11), (dict(rank=0), 12), (dict(ids=0), 13), (dict(U=0), 16),
    (dict(ldu=1), 17), (dict(stride_u=-1), 18), (dict(V=0), 19), (dict(ldv=5), 20), (dict(stride_v=-1), 21),
    (dict(dA=P + 1), 23), (dict(ldda=4), 24), (dict(dU=0), 25), (dict(lddu=1), 26), (dict(stride_du=9), 27),
    (dict(dV=0), 28), (dict(lddv=5), 29), (dict(stride_dv=11), 30)])
def test_adapters_grad_refuses(bad, position):
    refuse(g.sgemm_adapters_grad, AGRAD, bad, position)


@pytest.mark.parametrize("M", [0, 1, 29, 64, 65, 512, 513, 2011, 40000])
def test_one_adapters_workspace_for_a_training_step(M):
    for N in (1, 64, 1037, 4096):
        for K in (1, 100, 4096, 20000):
            for G, rank in ((1, 1), (7, 16), (64, 255)):
                assert (g.sgemm_adapters_grad_workspace_size(M, N, K, G, rank)
                        >= g.sgemm_adapters_workspace_size(M, N, K, G, rank) > 0)


def test_adapters_refuse_a_workspace():
    for fn, base, size in ((g.sgemm_adapters, ADAPT, g.sgemm_adapters_workspace_size),
                           (g.sgemm_adapters_grad, AGRAD, g.sgemm_adapters_grad_workspace_size)):
        need = size(4, 6, 5, 3, 2)
        assert need > 0 and size(4, 6, 5, 0, 2) == 0 and size(-1, 6, 5, 3, 2) == 0 and size(4, 6, 5, 3, 257) == 0
        for bad in (dict(workspace=0), dict(workspace=P + 64), dict(workspace_bytes=need - 1)):
            assert fn(*{**base, **bad}.values(), stream=0, check=False) == -24


def test_status_strings_cover_every_position():
    for n in range(1, 33):
        assert g.sgemm_status_string(-100 - n) == f"invalid argument {n}"
    assert g.sgemm_status_string(-100) == "unknown status" and g.sgemm_status_string(-133) == "unknown status"


def test_cpu_tensors_are_refused():
    import torch
    x = torch.zeros(8, 8)
    with pytest.raises(TypeError):
        g.sgemm_combine(4, 2, 8, 3, None, None, x, 8, 0.0, P, 8, stream=0)
    with pytest.raises(TypeError):
        g.sgemm_combine(4, 2, 8, 3, None, None, P, 8, 0.0, x, 8, stream=0)
    with pytest.raises(TypeError):
        g.sgemm_combine(4, 2, 8, 3, torch.zeros(4, 2, dtype=torch.int32), None, P, 8, 0.0, P, 8, stream=0)


def test_int_arguments_are_not_truncated():
    with pytest.raises((ctypes.ArgumentError, TypeError)):
        g.sgemm_combine(4.5, 2, 8, 3, None, None, P, 8, 0.0, P, 8, stream=0)


# ---- the plain forms' gradients against differences -------------------------
@pytest.mark.parametrize("sigmoid", [False, True])
@pytest.mark.parametrize("renorm", [False, True])
def test_route_gradient_is_the_weights_slope(sigmoid, renorm):
    r = np.random.default_rng(5)
    x = r.standard_normal((4, 9)) * 1.3
    ids, _ = ro.route(x, 3, sigmoid=sigmoid, renorm=renorm)
    c = r.standard_normal((4, 3))

    def loss(v):
        out = 0.0
        for t in range(len(v)):
            s = ro.scores(v[t], sigmoid)[ids[t]]
            out += float((c[t] * (s / s.sum() if renorm else s)).sum())
        return out * 1.7
    got, _ = ro.route_grad(x, ids, c, sigmoid=sigmoid, renorm=renorm, scale=1.7)
    h = 1e-6
    for t in range(4):
        for e in range(9):
            up, down = x.copy(), x.copy()
            up[t, e] += h
            down[t, e] -= h
            # central differences: h^2 of curvature and 1e-16 / h of rounding
            assert abs((loss(up) - loss(down)) / (2 * h) - got[t, e]) < 1e-8


def test_adapter_and_product_gradients_are_slopes():
    r = np.random.default_rng(6)
    M, N, K, G, n = 5, 4, 3, 3, 2
    A, B, U, V = (r.standard_normal(s) for s in ((M, K), (K, N), (G, K, n), (G, n, N)))
    ids, ranks, scales = np.array([0, 2, -1, 2, 0]), np.array([2, 2, 1]), r.standard_normal(G)
    D = r.standard_normal((M, N))
    zero = np.zeros((M, N))

    def loss(a, u, v):
        return float((ro.adapters(a, B, ids, ranks, scales, u, v, 1.3, 0.0, zero)[0] * D).sum())
    grads = ro.adapters_grad(A, B, D, ids, ranks, scales, U, V, 1.3, 0.0, np.zeros_like(U), np.zeros_like(V))
    h = 1e-5
    for which, x in enumerate((A, U, V)):
        for i in np.ndindex(x.shape):
            args = [A, U, V]
            up, down = x.copy(), x.copy()
            up[i] += h
            down[i] -= h
            args[which] = up
            high = loss(*args)
            args[which] = down
            # the loss is linear in each operand: the difference is exact but for rounding
            assert abs((high - loss(*args)) / (2 * h) - grads[which][0][i]) < 1e-8
    # the products' gradient, through the same sums
    offsets, rows = ro.group_rows(ids, G)
    W = r.standard_normal((G, K, N))

    def product(w):
        return float((np.nan_to_num(ro.grouped(offsets, rows, N, K, 1.0, A, 1, w, False, 0.0, zero, 1)[0]) * D).sum())
    got = ro.grouped_tn(offsets, rows, 1.0, A, 1, D, 1, 0.0, np.zeros_like(W))[0]
    for i in np.ndindex(W.shape):
        up, down = W.copy(), W.copy()
        up[i] += h
        down[i] -= h
        assert abs((product(up) - product(down)) / (2 * h) - got[i]) < 1e-8


@pytest.mark.parametrize("fn,base", [
    (g.sgemm_route, ROUTE), (g.sgemm_route_grad, GRAD), (g.sgemm_group_rows, GROUP), (g.sgemm_grouped, GROUPED),
    (g.sgemm_grouped_tn, TN), (g.sgemm_combine, COMBINE), (g.sgemm_combine_grad, CGRAD), (g.sgemm_adapters, ADAPT),
    (g.sgemm_adapters_grad, AGRAD)], ids=lambda x: getattr(x, "__name__", ""))
def test_every_pointer_is_4_byte_aligned(fn, base):
    pointers = [n for n in base if (base[n] == P or n in ("bias", "ranks", "scales")) and n != "workspace"]
    assert len(pointers) >= 3
    for n in pointers:
        refuse(fn, base, {n: P + 2}, list(base).index(n) + 1)


def test_no_kernel_of_these_uses_scratch():
    """Their kernels too keep their state in registers and LDS (see the library's own such test)."""
    from fp32_gemm_03_amd import build as b
    try:
        res = b.kernel_resources(source=1)
    except (RuntimeError, OSError) as e:
        pytest.skip(f"cannot read the code object: {e}")
    names = dict(zip(res, b.demangle(res)))
    assert any("thin" in n for n in names.values()) and any("route" in n for n in names.values())
    bad = {names[k]: r for k, r in res.items()
           if r.get("private_segment_fixed_size", -1) != 0 or r.get("vgpr_spill_count", -1) != 0}
    assert not bad, bad
    assert all(0 <= r["group_segment_fixed_size"] <= 160 * 1024 for r in res.values())
