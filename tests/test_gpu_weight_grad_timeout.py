"""A weight gradient whose waits run out: no value of a tile that was not finished
passes for a result, the error word says so, and the context stays usable.  The
kernel's producers are told to stop early; every wait is bounded to 0.2 s."""
import time

import pytest
import torch

from test_gpu_checkpoint import check_wgrad, flp, make  # noqa: F401 (flp: fixture)

pytestmark = pytest.mark.gpu
LIMIT_NS = 200_000_000


def run(flp, odd, stall):  # noqa: F811
    ws = torch.empty(flp.SELFTEST_WEIGHT_GRAD_BYTES, dtype=torch.uint8, device="cuda")
    t0 = time.perf_counter()
    st = flp.selftest_weight_grad_timeout(odd, stall, LIMIT_NS, workspace=ws)
    assert time.perf_counter() - t0 < 5.0
    o, K = flp.SELFTEST_WEIGHT_GRAD_OUTPUT_OFFSET, 521 if odd else 520
    return st, ws[o:o + 136 * K * 4].view(torch.float32).view(136, K)


@pytest.mark.parametrize("odd", [False, True])
def test_a_stalled_contraction_leaves_nan(flp, odd):  # noqa: F811
    st, dw = run(flp, odd, -1)
    assert st == flp.FLP_OK and not dw.any()
    assert run(flp, odd, 6)[0] == flp.FLP_OK        # both tiles need six blocks
    for stall in (0, 1, 2, 3, 5):                   # before any data, between runs, between tiles, in the second one
        st, dw = run(flp, odd, stall)
        assert st == flp.FLP_ERR_TIMEOUT, stall
        if odd or stall < 3:
            assert torch.isnan(dw).all(), stall
        else:                                       # the first tile, 512 columns, was finished
            assert not dw[:, :512].any() and torch.isnan(dw[:, 512:]).all(), stall
    dy, kept = make(flp, 777, 264, 1000)            # the real call still works
    check_wgrad(flp, dy, kept, flp.checkpoint_weight_grad(dy, kept))


def test_arguments(flp):  # noqa: F811
    small = torch.empty(1024, dtype=torch.uint8, device="cuda")
    assert flp.selftest_weight_grad_timeout(False, 0, LIMIT_NS, workspace=small) == flp.FLP_ERR_WORKSPACE
    for limit in (0, -1, 61 * 10**9):
        assert flp.selftest_weight_grad_timeout(False, 0, limit) == flp.FLP_ERR_INVALID_ARG
