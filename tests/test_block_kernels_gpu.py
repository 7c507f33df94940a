"""The block's operators at sizes and in forms that their parametrised tests do not reach.

Tolerances are those of test_block_gpu; dweight is a 64-bit sum of shares that are rounded once
each, and rounded: 2 2^-24 of its terms (1% more for what 64 bits lose), for rows of any length."""
import numpy as np
import pytest
import torch

import fp32_gemm_03_amd as g
from tests import block_oracle as bo
from tests import gpu_util as gu
from tests.test_block_gpu import ONCE, floats, stream
from tests.test_rows_gpu import NAN, U24, Buffer, rng_of, within

pytestmark = pytest.mark.gpu


@pytest.fixture(autouse=True)
def _gpu_available():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")


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
