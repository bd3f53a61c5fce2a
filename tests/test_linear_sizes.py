"""Sizes that the linear layer refuses, on the CPU, before a device is touched."""
import ctypes

import pytest


@pytest.fixture(scope="module")
def flp():
    from entropy_loss_gb300 import build, flp as _flp
    build.build()
    _flp.load()
    return _flp


# Contractions above 131072 keep partial tiles of 256 x 256 outputs for each run: 2^22 at most.
@pytest.mark.parametrize("M,N,K", [(256, 256 * 513, 2 ** 30), (256, 2 ** 30, 256 * 513), (256 * 2, 256 * 2 ** 20, 131073 * 2)])
def test_deep_contractions_of_too_many_outputs(flp, M, N, K):
    b = (ctypes.addressof(ctypes.create_string_buffer(64)) + 15) // 16 * 16
    lib = flp.load()
    need = ctypes.c_size_t(0)
    ld = 2 ** 30
    assert lib.flp_linear_workspace(b, ld, b, ld, M, N, K, ctypes.byref(need)) == flp.FLP_ERR_UNSUPPORTED
    assert lib.flp_linear(b, ld, b, ld, None, 1, 0, None, 0, M, N, K, b, ld, None, 0, b, 64, None) == flp.FLP_ERR_UNSUPPORTED
    assert lib.flp_linear_backward(b, ld, b, ld, b, ld, None, 0, 0, M, N, K, b, ld, b, 0, None, b, 64, None) == flp.FLP_ERR_UNSUPPORTED


def test_terms_of_the_backward_pass(flp):
    buf = ctypes.create_string_buffer(64)
    b = (ctypes.addressof(buf) + 15) // 16 * 16
    need = ctypes.c_size_t(0)

    def call(terms, M=4):
        return flp.load().flp_linear_backward_ex(b, 32, b, 64, b, 64, b, 32, 2, terms, M, 32, 64, b, 64, b, 0, None, b, 16, None)

    def query(terms, M=4):
        return flp.load().flp_linear_backward_workspace_ex(b, 32, b, 64, b, 64, 2, terms, 1, 1, 1, M, 32, 64, 0, ctypes.byref(need))

    for f in (call, query):
        for terms in (-1, 3):
            assert f(terms) == flp.FLP_ERR_INVALID_ARG
        assert f(2, 2 ** 29 + 1) == flp.FLP_ERR_UNSUPPORTED
