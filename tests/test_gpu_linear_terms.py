"""The linear layer's backward pass with d as one bf16 number or as the sum of two, as the
caller asks.  Tolerances as in test_gpu_linear.py and test_gpu_linear_far_values.py: d is
off by 2^-8 or 2^-16 of itself and by its slope's 2^-17, the sums by (terms / 16 + 2) 2^-23
of their magnitudes, a bf16 result by half a step on top.
"""
import pytest
import torch

from test_gpu_linear import act64, flp, matrix  # noqa: F401 (flp: fixture)

pytestmark = pytest.mark.gpu


def inputs(M, N, K, pads=(0, 0, 0, 0), offsets=(0, 0, 0, 0)):
    g = torch.Generator().manual_seed(M + N + K)
    return [matrix(*shape, pad, offset, g, scale)[1] for shape, scale, pad, offset in
            zip(((M, K), (N, K), (M, N), (M, N)), (1.0, K ** -0.5, 1.0, 1.5), pads, offsets)]


SHAPES = [(1, 72, 64), (64, 264, 136), (65, 264, 136), (130, 1000, 2047), (300, 2048, 520), (700, 19456, 192), (2050, 1000, 4104),
          (4100, 1000, 4608), (2050, 2048, 4608), (1030, 513, 8199), (2100, 264, 136),
          (40, 300000, 64), (40, 600000, 64),   # runs of a long contraction; more of them than a cluster holds
          (70000, 72, 64)]                      # more than 131072 rows with both numbers


@pytest.mark.parametrize("M,N,K", SHAPES)
@pytest.mark.parametrize("act", ["relu", "gelu", "gelu_tanh", "silu"])
@pytest.mark.parametrize("dw_dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("terms", [1, 2])
def test_terms(flp, M, N, K, act, dw_dtype, terms):  # noqa: F811
    x, W, dy, pre = inputs(M, N, K)
    dx, dW, db = flp.linear_backward(dy, x, W, pre, activation=act, dw_dtype=dw_dtype, d_terms=terms)
    d = dy.double() * act64(pre.double(), act)[1]
    e = 2.0 ** -17 * dy.double().abs()
    each = e + 2.0 ** (-8 * terms) * (d.abs() + e)
    fine = dw_dtype is torch.float32
    for got, a, b, off, n, last in ((dx, d, W.double(), each, terms * N, 2.0 ** -8),
                                    (dW, d.t(), x.double(), each.t(), terms * M, 2.0 ** -24 if fine else 2.0 ** -8)):
        want = a @ b
        slack = off @ b.abs() + (n / 16 + 2) * 2.0 ** -23 * (a.abs() @ b.abs()) * 1.01
        assert bool(((got.double() - want).abs() <= slack + last * (want.abs() + slack)).all())
    # each gradient alone, and what the rule of 0 takes
    for k in range(3):
        alone = flp.linear_backward(dy, x, W, pre, activation=act, dw_dtype=dw_dtype, d_terms=terms, want_dx=k == 0, want_dW=k == 1,
                                    want_dbias=k == 2)
        assert torch.equal(alone[k], (dx, dW, db)[k]) and sum(t is not None for t in alone) == 1
    rule = flp.linear_backward(dy, x, W, pre, activation=act, dw_dtype=dw_dtype)
    if act == "relu" or terms == (2 if M <= 64 else 1):
        assert torch.equal(rule[0], dx)
    if act == "relu" or terms == (2 if M <= 64 or fine else 1):
        assert torch.equal(rule[1], dW)
    assert torch.equal(rule[2], db)


@pytest.mark.parametrize("M,N,K", [(2100, 1033, 4103), (90, 77, 33)])
def test_rows_at_odd_places(flp, M, N, K):  # noqa: F811
    x, W, dy, pre = inputs(M, N, K, (1, 0, 3, 5), (0, 1, 1, 2))
    for dw_dtype in (torch.float32, torch.bfloat16):
        got = flp.linear_backward(dy, x, W, pre, activation="silu", dw_dtype=dw_dtype, d_terms=2)
        want = flp.linear_backward(*(t.contiguous() for t in (dy, x, W, pre)), activation="silu", dw_dtype=dw_dtype, d_terms=2)
        for a, b in zip(got, want):
            assert torch.equal(a, b)


def test_two_terms_in_a_graph_and_through_autograd(flp):  # noqa: F811
    M, N, K = 200, 512, 264
    x, W, dy, pre = inputs(M, N, K)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        flp.linear_backward(dy, x, W, pre, activation="gelu", d_terms=2)
    s.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=s):
        out = flp.linear_backward(dy, x, W, pre, activation="gelu", d_terms=2)
    dy.mul_(-2)
    graph.replay()
    torch.cuda.synchronize()
    for a, b in zip(out, flp.linear_backward(dy, x, W, pre, activation="gelu", d_terms=2)):
        assert torch.equal(a, b)
    for terms in (0, 1, 2):
        leaves = [t.clone().requires_grad_() for t in (x, W)]
        y = flp.fused_linear(*leaves, activation="gelu", d_terms=terms)
        y.backward(dy)
        kept = flp.linear(x, W, activation="gelu", keep=True)[1]
        dx, dW, _ = flp.linear_backward(dy, x, W, kept, activation="gelu", dw_dtype=torch.bfloat16, d_terms=terms)
        assert torch.equal(leaves[0].grad, dx) and torch.equal(leaves[1].grad, dW)
