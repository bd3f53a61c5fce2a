"""Refusals of the expert, linear and given-logits entry points, on the CPU: argument
errors are returned before a device is touched."""
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


def test_expert_sort(flp, b):
    def call(**o):
        a = dict(e=b, T=4, k=2, E=8, rows=b, slots=b, counts=b, offsets=b, ws=b, n=8192)
        a.update(o)
        return flp.load().flp_expert_sort(a["e"], a["T"], a["k"], a["E"], a["rows"], a["slots"], a["counts"], a["offsets"],
                                          a["ws"], a["n"], None)

    for o in (dict(T=-1), dict(k=0), dict(E=0), dict(e=None), dict(rows=None), dict(slots=None), dict(counts=None),
              dict(offsets=None), dict(e=b + 4), dict(rows=b + 2), dict(slots=b + 1), dict(counts=b + 4), dict(offsets=b + 4)):
        assert call(**o) == flp.FLP_ERR_INVALID_ARG, o
    for o in (dict(E=1025), dict(T=2 ** 31), dict(T=2 ** 30, k=2), dict(T=2 ** 40, k=2 ** 40),
              dict(T=1, k=2 ** 31 - 1), dict(T=1, k=2 ** 30 + 1)):
        assert call(**o) == flp.FLP_ERR_UNSUPPORTED, o
    for o in (dict(T=5000, ws=None), dict(T=5000, n=4096), dict(T=5000, ws=b + 4)):
        assert call(**o) == flp.FLP_ERR_WORKSPACE, o
    need = ctypes.c_size_t(7)
    query = flp.load().flp_expert_sort_workspace
    assert query(100, 2, 8, ctypes.byref(need)) == flp.FLP_OK and need.value == 0
    assert query(5000, 2, 8, ctypes.byref(need)) == flp.FLP_OK and need.value > 0
    assert query(5000, 2, 8, None) == flp.FLP_ERR_INVALID_ARG
    assert query(5000, 2, 1025, ctypes.byref(need)) == flp.FLP_ERR_UNSUPPORTED


def test_expert_rows(flp, b):
    lib = flp.load()

    def gather(**o):
        a = dict(x=b, ldx=64, dt=1, T=4, H=64, k=2, rows=b, total=b, xs=b, ldxs=64, w=None, wt=0)
        a.update(o)
        return lib.flp_expert_gather(a["x"], a["ldx"], a["dt"], a["T"], a["H"], a["k"], a["rows"], a["total"], a["xs"], a["ldxs"],
                                     None)

    def combine(**o):
        a = dict(x=b, ldx=64, dt=1, T=4, H=64, k=2, rows=b, total=b, xs=b, ldxs=64, w=b, wt=0)
        a.update(o)
        return lib.flp_expert_combine(a["xs"], a["ldxs"], a["dt"], a["w"], a["wt"], a["T"], a["H"], a["k"], a["rows"], a["total"],
                                      a["x"], a["ldx"], None)

    def backward(**o):
        a = dict(x=b, ldx=64, dt=1, T=4, H=64, k=2, rows=b, total=b, xs=b, ldxs=64, w=b, wt=0, dys=b, lddys=64, dw=b)
        a.update(o)
        return lib.flp_expert_combine_backward(a["x"], a["ldx"], a["xs"], a["ldxs"], a["dt"], a["w"], a["wt"], a["T"], a["H"],
                                               a["k"], a["rows"], a["total"], a["dys"], a["lddys"], a["dw"], None)

    for f in (gather, combine, backward):
        for o in (dict(T=-1), dict(H=0), dict(k=0), dict(dt=2), dict(x=None), dict(xs=None), dict(rows=None), dict(total=None),
                  dict(rows=b + 2), dict(total=b + 4), dict(ldx=63), dict(ldxs=63), dict(x=b + 1), dict(xs=b + 1)):
            assert f(**o) == flp.FLP_ERR_INVALID_ARG, (f, o)
        for o in (dict(T=2 ** 30, k=2), dict(T=1, k=2 ** 31 - 1), dict(T=1, k=2 ** 30 + 1)):
            assert f(**o) == flp.FLP_ERR_UNSUPPORTED, (f, o)
        assert f(T=0, x=None, xs=None, rows=None, total=None) == flp.FLP_OK
    for f in (combine, backward):
        for o in (dict(wt=2), dict(w=b + 2), dict(w=b + 1, wt=1)):
            assert f(**o) == flp.FLP_ERR_INVALID_ARG, (f, o)
    for o in (dict(dys=None), dict(lddys=1), dict(dys=b + 1), dict(dw=b + 2)):
        assert backward(**o) == flp.FLP_ERR_INVALID_ARG, o


def test_token_logprob(flp, b):
    def call(**o):
        a = dict(x=b, ld=64, dt=1, y=b, M=4, V=64, s=1.0, lp=b, lse=b, e=b, k=2, tv=b, ti=b)
        a.update(o)
        return flp.load().flp_token_logprob(a["x"], a["ld"], a["dt"], a["y"], a["M"], a["V"], -100, a["s"], a["lp"], a["lse"], a["e"],
                                            a["k"], a["tv"], a["ti"], None)

    for o in (dict(M=-1), dict(V=0), dict(dt=2), dict(x=None), dict(y=None), dict(y=b + 4), dict(ld=63), dict(x=b + 1), dict(s=0.0),
              dict(s=-1.0), dict(s=float("nan")), dict(s=float("inf")), dict(s=3e38), dict(lp=None), dict(lse=None), dict(k=-1),
              dict(k=65), dict(V=1, k=2), dict(tv=None), dict(ti=None), dict(lp=b + 2), dict(lse=b + 2), dict(e=b + 1),
              dict(tv=b + 2), dict(ti=b + 4)):
        assert call(**o) == flp.FLP_ERR_INVALID_ARG, o
    for o in (dict(k=33), dict(M=2 ** 31), dict(V=2 ** 31, ld=2 ** 31)):
        assert call(**o) == flp.FLP_ERR_UNSUPPORTED, o
    assert call(M=0, x=None, y=None, lp=None, lse=None, tv=None, ti=None) == flp.FLP_OK


def test_token_logprob_backward(flp, b):
    def call(**o):
        a = dict(x=b, ld=64, dt=1, y=b, M=4, V=64, s=1.0, lse=b, e=b, gl=b, ge=b, dx=b, lddx=64)
        a.update(o)
        return flp.load().flp_token_logprob_backward(a["x"], a["ld"], a["dt"], a["y"], a["M"], a["V"], -100, a["s"], a["lse"], a["e"],
                                                     a["gl"], a["ge"], a["dx"], a["lddx"], None)

    for o in (dict(M=-1), dict(V=0), dict(dt=5), dict(x=None), dict(y=None), dict(ld=1), dict(s=0.0), dict(lse=None), dict(e=None),
              dict(lse=b + 1), dict(e=b + 2), dict(gl=b + 2), dict(ge=b + 2), dict(dx=None), dict(lddx=63), dict(dx=b + 1)):
        assert call(**o) == flp.FLP_ERR_INVALID_ARG, o
    assert call(M=0, x=None, y=None, lse=None, dx=None) == flp.FLP_OK


def test_linear(flp, b):
    def call(**o):
        a = dict(x=b, ldx=64, w=b, ldw=64, bias=b, bt=1, act=2, r=b, ldr=32, M=4, N=32, K=64, y=b, ldy=32, pre=b, ldp=32)
        a.update(o)
        return flp.load().flp_linear(a["x"], a["ldx"], a["w"], a["ldw"], a["bias"], a["bt"], a["act"], a["r"], a["ldr"], a["M"], a["N"],
                                     a["K"], a["y"], a["ldy"], a["pre"], a["ldp"], b, 8192, None)

    for o in (dict(M=-1), dict(N=0), dict(K=0), dict(x=None), dict(w=None), dict(y=None), dict(ldx=63), dict(ldw=63), dict(ldy=31),
              dict(ldr=31), dict(ldp=31), dict(x=b + 1), dict(w=b + 1), dict(y=b + 1), dict(r=b + 1), dict(pre=b + 1), dict(act=5),
              dict(act=-1), dict(bt=2), dict(bias=b + 2, bt=0), dict(bias=b + 1)):
        assert call(**o) == flp.FLP_ERR_INVALID_ARG, o
    for o in (dict(M=2 ** 31), dict(K=2 ** 31, ldx=2 ** 31, ldw=2 ** 31), dict(N=2 ** 31), dict(M=2 ** 28, N=2 ** 24),
              dict(K=2 ** 31 - 2000, ldx=2 ** 31, ldw=2 ** 31)):
        assert call(**o) == flp.FLP_ERR_UNSUPPORTED, o
    assert call(M=0, x=None, y=None) == flp.FLP_OK
    assert flp.load().flp_linear_workspace(b, 64, b, 64, 4, 32, 64, None) == flp.FLP_ERR_INVALID_ARG


def test_linear_backward(flp, b):
    def call(**o):
        a = dict(dy=b, lddy=32, x=b, ldx=64, w=b, ldw=64, pre=b, ldp=32, act=2, M=4, N=32, K=64, dx=b, lddx=64, dw=b, dwt=0, db=b)
        a.update(o)
        return flp.load().flp_linear_backward(a["dy"], a["lddy"], a["x"], a["ldx"], a["w"], a["ldw"], a["pre"], a["ldp"], a["act"],
                                              a["M"], a["N"], a["K"], a["dx"], a["lddx"], a["dw"], a["dwt"], a["db"], b, 8192, None)

    for o in (dict(M=-1), dict(N=0), dict(K=0), dict(dy=None), dict(x=None), dict(w=None), dict(pre=None), dict(lddy=31), dict(ldx=63),
              dict(ldw=63), dict(ldp=31), dict(lddx=63), dict(dy=b + 1), dict(x=b + 1), dict(w=b + 1), dict(pre=b + 1), dict(dx=b + 1),
              dict(dw=b + 4), dict(db=b + 2), dict(act=9), dict(dwt=3)):
        assert call(**o) == flp.FLP_ERR_INVALID_ARG, o
    assert call(M=2 ** 31) == flp.FLP_ERR_UNSUPPORTED
    assert call(dx=None, dw=None, db=None, x=None, w=None) == flp.FLP_OK
    assert flp.load().flp_linear_backward_workspace(b, 32, b, 64, b, 64, 2, 1, 1, 1, 4, 32, 64, 0, None) == flp.FLP_ERR_INVALID_ARG


def test_linear_selftest(flp, b):
    f = flp.load().flp_selftest_linear_timeout
    assert f(None, 1 << 30, 0, 1, 1000, None) == flp.FLP_ERR_WORKSPACE
    assert f(b, 8192, 0, 1, 1000, None) == flp.FLP_ERR_WORKSPACE
    assert f(b + 4, 1 << 30, 0, 1, 1000, None) == flp.FLP_ERR_WORKSPACE
    for limit in (0, -5, 61 * 10 ** 9):
        assert f(b, 1 << 30, 0, 1, limit, None) == flp.FLP_ERR_INVALID_ARG
    for form in (-1, 4):
        assert f(b, 1 << 30, form, 1, 1000, None) == flp.FLP_ERR_INVALID_ARG


def test_binding_refuses_before_loading_anything_on_a_device(flp):
    import torch
    x = torch.zeros(4, 64)
    order = flp.ExpertOrder(torch.zeros(4, 1, dtype=torch.int32), torch.zeros(4, dtype=torch.int32), torch.zeros(2, dtype=torch.int64),
                            torch.zeros(3, dtype=torch.int64))
    for f in (lambda: flp.expert_sort(torch.zeros(4, 2, dtype=torch.int64), 2), lambda: flp.expert_sort(torch.zeros(4), 2),
              lambda: flp.expert_gather(x, order), lambda: flp.expert_combine(x, order),
              lambda: flp.expert_combine_backward(x, x, order), lambda: flp.token_logprob(x, x[:, 0].long()),
              lambda: flp.token_logprob_backward(x, x[:, 0].long(), x[:, 0], None, None),
              lambda: flp.linear(x.bfloat16(), x.bfloat16()), lambda: flp.linear(x, x, activation="tanh"),
              lambda: flp.linear_backward(x, x, x)):
        with pytest.raises(ValueError):
            f()
