"""The linear layer and its gradients where values are infinite.

An infinite d = dy act'(v) makes its row of dx and its row of dW infinite, with the signs
of W and x, and its column of dbias; every other element is as it is without it: d is off
by 2^-8 of itself (or less) and the slopes by 2^-17, a bf16 result by half a step, and a
sum by (terms / 16 + 2) 2^-23 of its magnitudes: a step of 16 products loses at most 4.75
last places of the accumulator (a quarter a product, 3/4 of their sum), and partial sums
of centred products stay below a fifth of the magnitudes' sum but for the first few.
v = +-inf gives what the formulas' products give, 0 (gelu: the limit of
v Phi(v)) where the activation has one, and slopes 0 and 1.
"""
import math

import pytest
import torch

from test_gpu_linear import ACTS, act64, flp, matrix  # noqa: F401 (flp: fixture)

pytestmark = pytest.mark.gpu
INF = math.inf


@pytest.mark.parametrize("act", ACTS)
@pytest.mark.parametrize("dw_dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("M,N,K", [(1, 72, 64), (64, 264, 136), (65, 264, 136), (300, 200, 96), (2100, 1032, 4104)])
@pytest.mark.parametrize("value", [INF, -INF])
def test_infinite_upstream_gradient(flp, act, dw_dtype, M, N, K, value):  # noqa: F811
    g = torch.Generator().manual_seed(M + N)
    x, W, dy, pre = (matrix(*shape, 0, 0, g, scale)[1] for shape, scale in (((M, K), 1.0), ((N, K), K ** -0.5), ((M, N), 1.0),
                                                                            ((M, N), 1.5)))
    m, n = M - 1, N // 3
    x[m] = torch.where(x[m] == 0, 1, x[m])
    W[n] = torch.where(W[n] == 0, 1, W[n])
    pre[m, n] = 0.75  # every slope positive
    dy[m, n] = value
    dx, dW, db = flp.linear_backward(dy, x, W, pre if act else None, activation=act, dw_dtype=dw_dtype)
    assert torch.equal(dx[m].float(), value * torch.sign(W[n].float()))
    assert torch.equal(dW[n].float(), value * torch.sign(x[m].float()))
    assert float(db[n]) == value
    slope = act64(pre.double(), act)[1]
    dy[m, n] = 0
    d = dy.double() * slope
    e = 2.0 ** -17 * dy.double().abs() if act else torch.zeros_like(d)
    each = e + 2.0 ** -8 * (d.abs() + e) if act else e
    rows = torch.arange(M, device="cuda") != m
    cols = torch.arange(N, device="cuda") != n
    for got, a, b, off, terms, keep, last in ((dx, d, W.double(), each, 2 * N, rows, 2.0 ** -8),
                                              (dW, d.t(), x.double(), each.t(), 2 * M, cols,
                                               2.0 ** -8 if dw_dtype is torch.bfloat16 else 2.0 ** -24)):
        want = (a @ b)[keep]
        slack = off[keep] @ b.abs() + (terms / 16 + 2) * 2.0 ** -23 * (a[keep].abs() @ b.abs()) * 1.01
        assert bool(((got.double()[keep] - want).abs() <= slack + last * (want.abs() + slack)).all())
    want = d.sum(0)
    assert bool(((db.double() - want).abs() <= e.sum(0) + 2.0 ** -24 * (M / 8 + 64) * d.abs().sum(0))[cols].all())
@pytest.mark.parametrize("act", ACTS)
@pytest.mark.parametrize("M", [1, 3, 200])
def test_infinite_arguments(flp, act, M):  # noqa: F811
    v = torch.tensor([2.0, -2.0, 0.0, -0.0, 1e-30, -1e30, 0.5, -0.5])
    x = torch.zeros(M, 8, dtype=torch.bfloat16, device="cuda")
    x[0, 0] = INF
    W = torch.zeros(8, 8, dtype=torch.bfloat16, device="cuda")
    W[:, 0] = v.to(torch.bfloat16)
    y, pre = flp.linear(x, W, activation=act, keep=True)
    sign = torch.sign(W[:, 0].float())
    kept = torch.where(sign == 0, math.nan, sign * INF)  # 0 inf
    assert torch.equal(torch.nan_to_num(pre[0].float(), 7.0), torch.nan_to_num(kept, 7.0))
    low = {None: -INF, "relu": 0.0, "gelu": 0.0, "gelu_tanh": math.nan, "silu": math.nan}[act]
    want = torch.where(sign == 0, math.nan, torch.where(sign > 0, INF, low))
    assert torch.equal(torch.nan_to_num(y[0].float(), 7.0), torch.nan_to_num(want, 7.0))
    assert bool((y[1:] == 0).all()) and bool((pre[1:] == 0).all())
    if act:
        # slopes 0 and 1 at the ends
        dy = torch.ones(M, 8, dtype=torch.bfloat16, device="cuda")
        _, _, db = flp.linear_backward(dy[:1], x[:1], W, pre[:1], activation=act, want_dx=False, want_dW=False)
        assert torch.equal(db[sign != 0], (sign[sign != 0] > 0).float())
        for far in (11.0, 14.0, 100.0, 1e30) if act == "gelu_tanh" else (100.0, 1e30) if act == "silu" else (14.0, 100.0, 1e30):
            pre[0] = far * sign
            _, _, db = flp.linear_backward(dy[:1], x[:1], W, pre[:1], activation=act, want_dx=False, want_dW=False)
            assert torch.equal(db[sign != 0], (sign[sign != 0] > 0).float()), far
