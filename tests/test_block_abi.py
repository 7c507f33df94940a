"""The refusals of a feed-forward block's operators, on the CPU: every call below stops at an
argument check or a documented quick return, before any HIP call.  And the 64-bit plain forms'
gradients against differences."""
import numpy as np
import pytest

import fp32_gemm_03_amd as g
from tests import block_oracle as bo
from tests.test_rows_abi import P, refuse

BIG = 2 ** 31 - 1

NORM = dict(T=4, N=8, x=P, ldx=8, residual=P, ldr=8, weight=P, eps=1e-5, sum=P, lds=8, y=P, ldy=8, q=P, ldq=8, scales=P)


@pytest.mark.parametrize("bad,position", [
    (dict(T=-1), 1), (dict(N=-1), 2), (dict(x=0), 3), (dict(x=P + 2), 3), (dict(ldx=7), 4), (dict(residual=P + 1), 5),
    (dict(ldr=7), 6), (dict(residual=None, ldr=7), 6), (dict(weight=P + 2), 7), (dict(eps=-1e-9), 8),
    (dict(eps=float("nan")), 8), (dict(eps=float("inf")), 8), (dict(sum=P + 3), 9), (dict(lds=7), 10),
    (dict(y=P + 2), 11), (dict(ldy=7), 12), (dict(ldq=7), 14), (dict(scales=0), 15), (dict(scales=P + 1), 15),
    (dict(T=-1, N=-1), 1), (dict(N=0, ldx=0), 4)])
def test_norm_refuses(bad, position):
    refuse(g.sgemm_norm, NORM, bad, position)


GRAD = dict(T=4, N=8, h=P, ldh=8, weight=P, eps=1e-5, dy=P, lddy=8, dsum=P, ldds=8, dh=P, lddh=8, beta=0.0, dweight=P,
            workspace=P, workspace_bytes=1 << 20)


@pytest.mark.parametrize("bad,position", [
    (dict(T=-1), 1), (dict(N=-1), 2), (dict(h=0), 3), (dict(h=P + 1), 3), (dict(ldh=7), 4), (dict(weight=P + 2), 5),
    (dict(eps=-1.0), 6), (dict(dy=0), 7), (dict(lddy=7), 8), (dict(dsum=P + 2), 9), (dict(ldds=7), 10),
    (dict(dh=P + 1), 11), (dict(lddh=7), 12), (dict(dweight=P + 2), 14)])
def test_norm_grad_refuses(bad, position):
    refuse(g.sgemm_norm_grad, GRAD, bad, position)


QUANT = dict(T=4, N=8, x=P, ldx=8, activation=0, gate=P, ldg=8, q=P, ldq=8, scales=P)


@pytest.mark.parametrize("bad,position", [
    (dict(T=-1), 1), (dict(N=-1), 2), (dict(x=0), 3), (dict(x=P + 2), 3), (dict(ldx=7), 4), (dict(activation=3), 5),
    (dict(activation=-1, gate=None), 5), (dict(gate=P + 2), 6), (dict(ldg=7), 7), (dict(q=0), 8), (dict(ldq=7), 9),
    (dict(scales=0), 10), (dict(scales=P + 2), 10)])
def test_quantize_refuses(bad, position):
    refuse(g.sgemm_quantize, QUANT, bad, position)


I8 = dict(M=4, N=6, K=8, alpha=1.0, A=P, lda=8, a_scales=P, B=P, ldb=8, b_scales=P, beta=0.0, C=P, ldc=6)


@pytest.mark.parametrize("bad,position", [
    (dict(M=-1), 1), (dict(N=-1), 2), (dict(K=-1), 3), (dict(A=0), 5), (dict(lda=7), 6), (dict(a_scales=P + 2), 7),
    (dict(B=0), 8), (dict(ldb=7), 9), (dict(b_scales=P + 1), 10), (dict(C=0), 12), (dict(C=P + 2), 12),
    (dict(ldc=5), 13), (dict(alpha=0.0, C=0), 12)])
def test_i8_refuses(bad, position):
    refuse(g.sgemm_i8, I8, bad, position)


GATED = dict(T=4, N=6, K=8, activation=0, x=P, ldx=8, G=P, ldg=6, U=P, ldu=6, y=P, ldy=6, gate=P, ldgate=6, up=P, ldup=6)


@pytest.mark.parametrize("bad,position", [
    (dict(T=-1), 1), (dict(N=-1), 2), (dict(K=-1), 3), (dict(activation=3), 4), (dict(x=0), 5), (dict(x=P + 2), 5),
    (dict(ldx=7), 6), (dict(G=0), 7), (dict(ldg=5), 8), (dict(U=0), 9), (dict(U=P + 1), 9), (dict(ldu=5), 10),
    (dict(y=0), 11), (dict(ldy=5), 12), (dict(gate=P + 2), 13), (dict(ldgate=5), 14), (dict(gate=None), 15),
    (dict(up=None), 15), (dict(up=P + 2), 15), (dict(ldup=5), 16)])
def test_gated_refuses(bad, position):
    refuse(g.sgemm_gated, GATED, bad, position)


BACK = dict(T=4, N=6, K=8, activation=0, x=P, ldx=8, G=P, ldg=6, U=P, ldu=6, gate=P, ldgate=6, up=P, ldup=6, dy=P, lddy=6,
            dx=P, lddx=8, beta=0.0, dG=P, lddg=6, dU=P, lddu=6, workspace=P, workspace_bytes=1 << 20)


@pytest.mark.parametrize("bad,position", [
    (dict(T=-1), 1), (dict(N=-1), 2), (dict(K=-1), 3), (dict(activation=-1), 4), (dict(x=0), 5), (dict(ldx=7), 6),
    (dict(G=0), 7), (dict(ldg=5), 8), (dict(U=0), 9), (dict(ldu=5), 10), (dict(gate=0), 11), (dict(ldgate=5), 12),
    (dict(up=0), 13), (dict(ldup=5), 14), (dict(dy=0), 15), (dict(lddy=5), 16), (dict(dx=P + 2), 17), (dict(lddx=7), 18),
    (dict(dG=P + 2), 20), (dict(lddg=5), 21), (dict(dG=None), 22), (dict(dU=None), 22), (dict(lddu=5), 23)])
def test_gated_grad_refuses(bad, position):
    refuse(g.sgemm_gated_grad, BACK, bad, position)


def test_workspaces_are_refused():
    for fn, base, need in ((g.sgemm_norm_grad, GRAD, g.sgemm_norm_grad_workspace_size(4, 8)),
                           (g.sgemm_gated_grad, BACK, g.sgemm_gated_grad_workspace_size(4, 6, 8))):
        assert need > 0
        for bad in (dict(workspace=0), dict(workspace=P + 128), dict(workspace_bytes=need - 1)):
            assert fn(*{**base, **bad}.values(), stream=0, check=False) == -24
    assert g.sgemm_norm_grad_workspace_size(-1, 8) == 0 and g.sgemm_norm_grad_workspace_size(0, 8) == 0
    assert g.sgemm_gated_grad_workspace_size(4, -6, 8) == 0
    for N, K in ((100, 50), (2048, 1024), (1000, 9000), (6, 8)):  # enough for T rows is enough for fewer
        sizes = [g.sgemm_gated_grad_workspace_size(T, N, K) for T in range(300)]
        assert sizes == sorted(sizes)


def test_sizes_beyond_a_launch_are_refused():
    norm = dict(T=BIG, N=1)
    assert g.sgemm_norm(*{**NORM, **norm}.values(), stream=0, check=False) == -22
    assert g.sgemm_norm(*{**NORM, **dict.fromkeys(("N", "ldx", "ldr", "lds", "ldy", "ldq"), BIG)}.values(), stream=0,
                        check=False) == -22
    assert g.sgemm_quantize(*{**QUANT, **norm}.values(), stream=0, check=False) == -22
    assert g.sgemm_norm_grad(*{**GRAD, **norm, "workspace_bytes": 1 << 40}.values(), stream=0, check=False) == -22
    k = g.SGEMM_I8_MAX_K + 1
    assert g.sgemm_i8(*{**I8, "K": k, "lda": k, "ldb": k}.values(), stream=0, check=False) == -22
    wide = dict(M=2 ** 30, N=2 ** 30, ldc=2 ** 30)
    assert g.sgemm_i8(*{**I8, **wide}.values(), stream=0, check=False) == -22
    wide = dict(T=2 ** 30, N=2 ** 30, ldg=2 ** 30, ldu=2 ** 30, ldy=2 ** 30, ldgate=2 ** 30, ldup=2 ** 30)
    assert g.sgemm_gated(*{**GATED, **wide}.values(), stream=0, check=False) == -22
    assert g.sgemm_gated(*{**GATED, "T": BIG}.values(), stream=0, check=False) == -22
    # the last launch of several is too large: refused before the first
    wide = dict.fromkeys(("N", "ldh", "lddy", "ldds", "lddh"), 2 ** 26)
    assert g.sgemm_norm_grad(*{**GRAD, **wide, "workspace_bytes": 1 << 40}.values(), stream=0, check=False) == -22
    wide = dict.fromkeys([name for name in BACK if name in ("N", "K") or name.startswith("ld")], 2 ** 20)
    assert g.sgemm_gated_grad(*{**BACK, **wide, "workspace_bytes": 1 << 40}.values(), stream=0, check=False) == -22


@pytest.mark.parametrize("fn,base,names", [
    (g.sgemm_norm, NORM, ("T", "N", "ldx", "ldr", "lds", "ldy", "ldq")),
    (g.sgemm_norm_grad, GRAD, ("T", "N", "ldh", "lddy", "ldds", "lddh")),
    (g.sgemm_quantize, QUANT, ("T", "N", "ldx", "activation", "ldg", "ldq")),
    (g.sgemm_i8, I8, ("M", "N", "K", "lda", "ldb", "ldc")),
    (g.sgemm_gated, GATED, ("T", "N", "K", "activation", "ldx", "ldg", "ldu", "ldy", "ldgate", "ldup")),
    (g.sgemm_gated_grad, BACK, ("T", "N", "K", "activation", "ldx", "ldg", "ldu", "ldgate", "ldup", "lddy", "lddx",
                                "lddg", "lddu"))])
def test_integers_beyond_32_bits_are_refused(fn, base, names):
    for name in names:
        for off in (1 << 32, -(1 << 32)):
            with pytest.raises(ValueError):
                fn(*{**base, name: base[name] + off}.values(), stream=0)


def test_quick_returns():
    assert g.sgemm_norm(*{**NORM, "T": 0, "x": 0, "scales": 0}.values(), stream=0) == 0
    assert g.sgemm_norm(*{**NORM, "N": 0, "x": 0, "q": 0}.values(), stream=0) == 0
    assert g.sgemm_norm(*{**NORM, "sum": None, "y": None, "q": None}.values(), stream=0) == 0
    assert g.sgemm_norm_grad(*{**GRAD, "N": 0, "h": 0, "dy": 0}.values(), stream=0) == 0
    assert g.sgemm_norm_grad(*{**GRAD, "dh": None, "dweight": None, "workspace": None}.values(), stream=0) == 0
    assert g.sgemm_quantize(*{**QUANT, "T": 0, "x": 0, "q": 0, "scales": 0}.values(), stream=0) == 0
    for bad in (dict(M=0, C=0), dict(N=0, C=0), dict(K=0, A=0, B=0, beta=1.0), dict(alpha=0.0, A=0, B=0, beta=1.0)):
        assert g.sgemm_i8(*{**I8, **bad}.values(), stream=0) == 0
    for bad in (dict(T=0, x=0, y=0), dict(N=0, G=0, U=0, y=0)):
        assert g.sgemm_gated(*{**GATED, **bad}.values(), stream=0) == 0
    for bad in (dict(K=0, x=0, G=0), dict(dx=None, dG=None, dU=None, workspace=None, gate=0),
                dict(T=0, x=0, dy=0, beta=1.0, workspace=None), dict(N=0, dx=None, workspace=None)):
        assert g.sgemm_gated_grad(*{**BACK, **bad}.values(), stream=0) == 0


def test_tensors_are_refused():
    """What the binding sees of a tensor before its address goes on (here: not on a GPU)."""
    import torch
    host = torch.zeros(64)
    with pytest.raises(TypeError):
        g.sgemm_norm(*{**NORM, "x": host}.values(), stream=0)
    with pytest.raises(TypeError):
        g.sgemm_quantize(*{**QUANT, "q": host}.values(), stream=0)
    with pytest.raises(TypeError):
        g.sgemm_i8(*{**I8, "A": host.to(torch.int8)}.values(), stream=0)


# ---------------------------------------------------------------------------
# the plain forms' gradients against differences
# ---------------------------------------------------------------------------
def _difference(f, v, at, step):
    out = []
    for sign in (1.0, -1.0):
        w = v.copy()
        w[at] += sign * step
        out.append(f(w))
    return (out[0] - out[1]) / (2 * step)


@pytest.mark.parametrize("kind", [0, 1, 2])
def test_slopes_against_differences(kind):
    x = np.linspace(-9.0, 9.0, 181)
    h = 1e-5
    near = (bo.act(kind, x + h)[0] - bo.act(kind, x - h)[0]) / (2 * h)
    # the third derivative is below 3: h^2 / 2, and 2^-52 9 / h of rounding
    assert np.abs(bo.slope(kind, x)[0] - near).max() < 1e-9
    assert np.array_equal(bo.slope(kind, np.array([-np.inf, np.inf]))[0], [0.0, 1.0])


def test_norm_grad_against_differences():
    r = np.random.default_rng(3)
    x, w, dy, ds = (r.standard_normal(s) for s in ((3, 7), 7, (3, 7), (3, 7)))
    eps = 2.0 ** -6

    def loss(x, w):
        n = x / np.sqrt((x * x).mean(1, keepdims=True) + eps) * w
        return (n * dy).sum() + (x * ds).sum()
    dh, _, dw, _ = bo.norm_grad(x, w, eps, dy, ds)
    for at in np.ndindex(3, 7):
        assert abs(_difference(lambda v: loss(v, w), x, at, 1e-5) - dh[at]) < 1e-8
    for at in np.ndindex(7):
        assert abs(_difference(lambda v: loss(x, v), w, at, 1e-5) - dw[at]) < 1e-8


@pytest.mark.parametrize("kind", [0, 1, 2])
def test_gated_grad_against_differences(kind):
    r = np.random.default_rng(4)
    x, G, U, dy = (r.standard_normal(s) for s in ((3, 4), (4, 5), (4, 5), (3, 5)))

    def loss(x, G, U):
        return (bo.act(kind, x @ G)[0] * (x @ U) * dy).sum()
    grads, _ = bo.gated_grad(kind, x, G, U, x @ G, x @ U, dy)
    for i, v in enumerate((x, G, U)):
        for at in np.ndindex(*v.shape):
            near = _difference(lambda w: loss(*[w if j == i else o for j, o in enumerate((x, G, U))]), v, at, 1e-5)
            assert abs(near - grads[i][at]) < 1e-7


def test_block_kernels_use_no_scratch():
    """Their kernels too keep their state in registers and LDS (see the library's own such test)."""
    from fp32_gemm_03_amd import build as b
    try:
        resources = b.kernel_resources(source=2)
    except (RuntimeError, OSError) as e:
        pytest.skip(f"cannot read the code object: {e}")
    assert len(resources) > 40
    for name, r in resources.items():
        assert r["private_segment_fixed_size"] == 0 and r["vgpr_spill_count"] == 0, name
        assert 0 <= r["group_segment_fixed_size"] <= 160 * 1024, name
