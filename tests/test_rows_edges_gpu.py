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
from tests.test_rows_gpu import U24, Buffer, call_route, within

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
