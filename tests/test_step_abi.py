"""The training-step entry points on the CPU: argument errors are returned before
a device is touched."""
import ctypes

import pytest


@pytest.fixture(scope="module")
def lib():
    from entropy_loss_gb300 import build, flp
    build.build()
    return flp.load()


@pytest.fixture(scope="module")
def buf():
    b = ctypes.create_string_buffer(8192 + 16)
    return b, (ctypes.addressof(b) + 15) // 16 * 16


def test_layer_norm(lib, buf):
    from entropy_loss_gb300 import flp
    b = buf[1]

    def call(**o):
        a = dict(X=b, ldx=64, dt=1, w=b, bias=b, pt=1, M=4, H=64, eps=1e-5, Y=b, ldy=64, q=None, s=None)
        a.update(o)
        return lib.flp_layer_norm(a["X"], a["ldx"], a["dt"], a["w"], a["bias"], a["pt"], a["M"], a["H"], a["eps"], a["Y"],
                                  a["ldy"], b, b, a["q"], a["s"], None)

    bad, no = flp.FLP_ERR_INVALID_ARG, flp.FLP_ERR_UNSUPPORTED
    for o in (dict(M=-1), dict(H=0), dict(dt=2), dict(pt=7), dict(X=None), dict(Y=None), dict(ldx=63), dict(ldy=0),
              dict(X=b + 1), dict(w=b + 1), dict(eps=-1.0), dict(eps=float("inf")), dict(q=b), dict(s=b),
              dict(q=b + 8, s=b)):
        assert call(**o) == bad, o
    assert call(H=16385, ldx=20000, ldy=20000) == no
    assert call(M=2**31) == no
    assert call(M=0, X=None, Y=None) == flp.FLP_OK


def test_layer_norm_backward(lib, buf):
    from entropy_loss_gb300 import flp
    b = buf[1]

    def call(**o):
        a = dict(dY=b, lddy=64, X=b, ldx=64, q=None, s=None, dt=1, w=b, pt=1, mean=b, rstd=b, M=4, H=64, dX=b, lddx=64)
        a.update(o)
        return lib.flp_layer_norm_backward(a["dY"], a["lddy"], a["X"], a["ldx"], a["q"], a["s"], a["dt"], a["w"], a["pt"],
                                           a["mean"], a["rstd"], a["M"], a["H"], a["dX"], a["lddx"], b, b, b, 4096, None)

    for o in (dict(M=-1), dict(H=0), dict(dt=5), dict(X=None), dict(q=b, s=b), dict(X=None, q=b), dict(mean=None),
              dict(rstd=None), dict(dY=None), dict(dX=None), dict(lddy=1), dict(lddx=1), dict(ldx=1), dict(dY=b + 1)):
        assert call(**o) == flp.FLP_ERR_INVALID_ARG, o
    assert call(H=20000, lddy=20000, ldx=20000, lddx=20000) == flp.FLP_ERR_UNSUPPORTED


def test_checkpoints(lib, buf):
    from entropy_loss_gb300 import flp
    b = buf[1]
    pack = lambda X=b, ld=64, dt=1, M=2, H=64, q=b, s=b: lib.flp_checkpoint_pack(X, ld, dt, M, H, q, s, None)
    unpack = lambda X=b, ld=64, dt=1, M=2, H=64, q=b, s=b: lib.flp_checkpoint_unpack(q, s, M, H, X, ld, dt, None)
    for f in (pack, unpack):
        for o in (dict(M=-1), dict(H=0), dict(dt=3), dict(X=None), dict(q=None), dict(s=None), dict(q=b + 4), dict(ld=63),
                  dict(X=b + 1)):
            assert f(**o) == flp.FLP_ERR_INVALID_ARG, o
        assert f(M=0, X=None) == flp.FLP_OK


def test_weight_gradient(lib, buf):
    from entropy_loss_gb300 import flp
    b = buf[1]

    def call(**o):
        a = dict(dY=b, ld=16, q=b, s=b, M=8, N=16, K=32, dW=b, dt=0, acc=0)
        a.update(o)
        return lib.flp_checkpoint_weight_grad(a["dY"], a["ld"], a["q"], a["s"], a["M"], a["N"], a["K"], a["dW"], a["dt"],
                                              a["acc"], b, 4096, None)

    for o in (dict(M=-1), dict(N=0), dict(K=0), dict(dt=4), dict(ld=15), dict(dY=b + 1), dict(dY=None), dict(dW=None),
              dict(dW=b + 4), dict(q=None), dict(s=None)):
        assert call(**o) == flp.FLP_ERR_INVALID_ARG, o
    assert call(acc=1, dt=1) == flp.FLP_ERR_UNSUPPORTED
    assert call(M=2**31) == flp.FLP_ERR_UNSUPPORTED
    assert lib.flp_checkpoint_weight_grad_workspace(b, 16, 8, 16, 32, 0, None) == flp.FLP_ERR_INVALID_ARG


def test_balance_loss(lib, buf):
    from entropy_loss_gb300 import flp
    b = buf[1]

    def call(**o):
        a = dict(z=b, ld=8, dt=0, T=4, E=8, k=2, coef=1.0, loss=b, grad=b, counts=b)
        a.update(o)
        return lib.flp_balance_loss(a["z"], a["ld"], a["dt"], None, None, a["T"], a["E"], a["k"], a["coef"], a["loss"],
                                    a["grad"], a["counts"], b, 4096, None)

    for o in (dict(T=-1), dict(E=0), dict(k=0), dict(k=9), dict(dt=2), dict(loss=None), dict(counts=None), dict(z=None),
              dict(ld=7), dict(z=b + 2), dict(grad=b + 2), dict(coef=float("nan"))):
        assert call(**o) == flp.FLP_ERR_INVALID_ARG, o
    assert call(E=1025, ld=2000) == flp.FLP_ERR_UNSUPPORTED
    assert call(T=2**31) == flp.FLP_ERR_UNSUPPORTED


def test_binding_refuses_before_loading_anything_on_a_device():
    import torch
    from entropy_loss_gb300 import flp
    x = torch.zeros(4, 64)
    for f in (lambda: flp.layer_norm(x), lambda: flp.checkpoint_pack(x), lambda: flp.balance_loss(x, 2),
              lambda: flp.layer_norm_backward(x, x, None, x[:, 0], x[:, 0]),
              lambda: flp.checkpoint_unpack(flp.Checkpoint8(x.to(torch.int8), x[:, :2].to(torch.uint8), 64, x.dtype))):
        with pytest.raises(ValueError):
            f()
