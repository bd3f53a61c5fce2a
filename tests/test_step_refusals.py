"""Refusals of the training-step entry points that test_step_abi.py does not reach:
pointers that are not aligned to their elements (an access through one would fault),
and the arguments of the entry points beside them.  On the CPU: returned before a
device is touched."""
import ctypes

import pytest


@pytest.fixture(scope="module")
def flp():
    from entropy_loss_gb300 import build, flp as _flp
    build.build()
    _flp.load()
    return _flp


@pytest.fixture(scope="module")
def b():
    buf = ctypes.create_string_buffer(8192 + 16)
    yield (ctypes.addressof(buf) + 15) // 16 * 16


@pytest.mark.parametrize("which", ["mean", "rstd"])
def test_layer_norm_statistics(flp, b, which):
    a = dict(mean=b, rstd=b)
    a[which] = b + 2
    assert flp.load().flp_layer_norm(b, 64, 1, b, b, 1, 4, 64, 1e-5, b, 64, a["mean"], a["rstd"], None, None,
                                     None) == flp.FLP_ERR_INVALID_ARG


@pytest.mark.parametrize("which", ["mean", "rstd", "dweight", "dbias"])
def test_layer_norm_backward_outputs(flp, b, which):
    a = dict(mean=b, rstd=b, dweight=b, dbias=b)
    a[which] = b + 1
    assert flp.load().flp_layer_norm_backward(b, 64, b, 64, None, None, 1, b, 1, a["mean"], a["rstd"], 4, 64, b, 64,
                                              a["dweight"], a["dbias"], b, 4096, None) == flp.FLP_ERR_INVALID_ARG


@pytest.mark.parametrize("over", [dict(loss=2), dict(counts=4), dict(experts=4)])
def test_balance_loss_outputs_and_experts(flp, b, over):
    a = {k: b + over.get(k, 0) for k in ("loss", "counts", "experts")}
    assert flp.load().flp_balance_loss(b, 8, 0, None, a["experts"], 4, 8, 2, 1.0, a["loss"], b, a["counts"], b, 4096,
                                       None) == flp.FLP_ERR_INVALID_ARG


def test_balance_loss_gradient_type(flp, b):
    call = lambda dt, gt, grad=b: flp.load().flp_balance_loss_ex(b, 8, dt, None, None, 4, 8, 2, 1.0, b, grad, gt, b, b, 4096,
                                                                 None)
    for dt, gt, grad in ((0, 1, b), (1, 2, b), (0, -1, b), (1, 0, b + 2), (0, 0, b + 2)):
        assert call(dt, gt, grad) == flp.FLP_ERR_INVALID_ARG


def test_weight_gradient_selftest(flp, b):
    f = flp.load().flp_selftest_weight_grad_timeout
    assert f(None, 1 << 30, 0, 1, 1000, None) == flp.FLP_ERR_WORKSPACE
    assert f(b, 8192, 0, 1, 1000, None) == flp.FLP_ERR_WORKSPACE
    assert f(b + 4, 1 << 30, 0, 1, 1000, None) == flp.FLP_ERR_WORKSPACE
    for limit in (0, -5, 61 * 10**9):
        assert f(b, 1 << 30, 0, 1, limit, None) == flp.FLP_ERR_INVALID_ARG


def test_weight_gradient_sizes_beyond_the_tiling(flp, b):
    """2^23 tiles of 256 x 512 (4 TB of dW): refused like every other argument, before a device is touched."""
    need = ctypes.c_size_t(0)
    N, K = 256 << 12, 512 << 11
    assert flp.load().flp_checkpoint_weight_grad(b, N, b, b, 8, N, K, b, 0, 0, b, 4096, None) == flp.FLP_ERR_UNSUPPORTED
    assert flp.load().flp_checkpoint_weight_grad_workspace(b, N, 8, N, K, 0, ctypes.byref(need)) == flp.FLP_ERR_UNSUPPORTED
