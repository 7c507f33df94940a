"""Corners of the calls around products whose B is picked row by row that show without a GPU:
sizes that are refused before any HIP call, and calls from several threads."""
import pytest

import fp32_gemm_03_amd as g
from tests.test_rows_abi import ADAPT, AGRAD, CGRAD, COMBINE, GROUPED, TN

INT_MAX = 2 ** 31 - 1
TOO_LARGE = -22


@pytest.mark.parametrize("fn,base,sizes", [
    (g.sgemm_grouped, GROUPED, dict(G=INT_MAX)), (g.sgemm_grouped, GROUPED, dict(G=INT_MAX - 63)),
    (g.sgemm_grouped, GROUPED, dict(K=INT_MAX, lda=INT_MAX)), (g.sgemm_grouped, GROUPED, dict(R=2 ** 29)),
    (g.sgemm_grouped, GROUPED, dict(K=INT_MAX - 31, lda=INT_MAX, ldb=INT_MAX, trans_b=1)),
    (g.sgemm_grouped_tn, TN, dict(R=INT_MAX)), (g.sgemm_grouped_tn, TN, dict(R=INT_MAX - 31, a_div=0, b_div=0)),
    (g.sgemm_grouped_tn, TN, dict(R=INT_MAX - 15, a_div=1 << 20, b_div=1 << 20)),
    (g.sgemm_combine_grad, CGRAD, dict(N=INT_MAX, ldd=INT_MAX, ldy=INT_MAX, lddy=INT_MAX)),
    (g.sgemm_combine_grad, CGRAD, dict(N=INT_MAX - 1023, ldd=INT_MAX, ldy=INT_MAX, lddy=INT_MAX)),
    (g.sgemm_adapters, ADAPT, dict(M=2 ** 29, workspace_bytes=1 << 50)),
    (g.sgemm_adapters, ADAPT, dict(K=INT_MAX, lda=INT_MAX, workspace_bytes=1 << 50)),
    (g.sgemm_adapters_grad, AGRAD, dict(M=2 ** 29, workspace_bytes=1 << 50)),
    (g.sgemm_adapters_grad, AGRAD, dict(K=INT_MAX, lda=INT_MAX, ldda=INT_MAX, stride_du=1 << 40, workspace_bytes=1 << 50)),
    (g.sgemm_adapters_grad, AGRAD, dict(N=INT_MAX, ldb=INT_MAX, lddc=INT_MAX, ldv=INT_MAX, lddv=INT_MAX,
                                        stride_dv=1 << 40, workspace_bytes=1 << 50)),
], ids=lambda v: getattr(v, "__name__", None) or (",".join(v) if len(v) < 9 else "_"))
def test_sizes_next_to_2_31_are_refused(fn, base, sizes):
    """A kernel's loop that steps past INT_MAX would not end: such a size is turned away."""
    assert fn(*{**base, **sizes}.values(), stream=0, check=False) == TOO_LARGE
    with pytest.raises(g.SgemmError):
        fn(*{**base, **sizes}.values(), stream=0)


def test_first_calls_of_two_threads(monkeypatch):
    """A call that begins while another thread's first one is looking up what it asks torch for
    looks it up itself: it does not run with half of it."""
    import threading

    import torch
    seen, errors = [], []

    def other():
        try:
            seen.append(g._begin(7))
        except Exception as e:  # noqa: BLE001
            errors.append(e)

    real = torch._C

    class Slow:
        """torch, where each of the first look-ups lets another thread's call through."""

        def __init__(self):
            self.asked = set()

        def __getattr__(self, name):
            if name.startswith("_cuda") and name not in self.asked:
                self.asked.add(name)
                t = threading.Thread(target=other)
                t.start()
                t.join(60)
            return getattr(real, name)

    device = torch.cuda.current_device if torch.cuda.is_available() else lambda: 0
    slow = Slow()
    monkeypatch.setattr(torch, "_C", slow)
    monkeypatch.setattr(torch.cuda, "is_initialized", lambda: True)
    monkeypatch.setattr(real, "_cuda_getDevice", device, raising=False)
    for name in ("_torch", "_F32", "_I32", "_raw_stream", "_get_device"):
        monkeypatch.setattr(g, name, None)
    monkeypatch.setattr(g, "_on_gpu", False)
    mine = g._begin(7)
    monkeypatch.undo()
    assert not errors and len(seen) == len(slow.asked) >= 2 and set(seen) == {mine}


@pytest.mark.parametrize("workspace", ["address", "tensor", "none"])
def test_a_negative_workspace_size_is_refused(monkeypatch, workspace):
    """In C it would be the largest size there is."""
    class Space:  # as much of a GPU tensor as the binding looks at
        is_cuda, device, nbytes = True, "cuda:0", 512

        def data_ptr(self):
            return 0x10000

        def is_contiguous(self):
            return True

        def get_device(self):
            return -1  # the current device, where none is in use

        def numel(self):
            return 512

        def element_size(self):
            return 1
    x = {"address": 0x10000, "tensor": Space(), "none": None}[workspace]
    with pytest.raises(ValueError):
        g._space(x, -1, -1)
    with pytest.raises(ValueError):
        g.sgemm_group_rows(100000, 8, 0x10000, 0x10000, 0x10000, x, -256, stream=0)
    assert g._space(x, 256, -1) == (None if x is None else 0x10000, 256)


@pytest.mark.parametrize("fn,base,name", [
    (g.sgemm_grouped, GROUPED, "a_div"), (g.sgemm_grouped_tn, TN, "a_div"), (g.sgemm_grouped_tn, TN, "b_div"),
    (g.sgemm_combine, COMBINE, "E"), (g.sgemm_combine_grad, CGRAD, "E")],
    ids=lambda v: getattr(v, "__name__", None) or (v if isinstance(v, str) else "_"))
@pytest.mark.parametrize("value", [2 ** 31, 2 ** 32, 2 ** 32 + 1, -2 ** 32, -2 ** 31 - 1])
def test_integers_beyond_32_bits_are_refused(fn, base, name, value):
    """Their low 32 bits would be another division of the slots (2^32: none, so that rows of A beyond
    the one asked for are read), or another number of experts."""
    with pytest.raises(ValueError):
        fn(*{**base, name: value}.values(), stream=0, check=False)
