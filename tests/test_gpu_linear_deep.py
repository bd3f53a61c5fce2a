"""The linear layer's products over very long contractions.

A step of a tensor core takes 16 products into its accumulator: each is cut to a quarter
of the accumulator's last place, toward zero, and their sum to one (products of v beside
2^23: 16 of 0.249 add nothing, 16 of 0.25 add 4, 16 of 0.875 add 12, one of 1.9 adds 1).
Products spread over many quarters lose half of one each, 16 / 8, and their sum 3 / 8 more
(the mean of 0, 1/4, 1/2 and 3/4): 2.375 places a step.  A sum of T steps of positive
products of one distribution holds t / T of itself after t of them, to a hundredth.  With
F = 2^m f, 1 <= f < 2, the mean of the last place over 0 .. F is 2^(m - 23) ((f - 1) / f +
1 / (3 f)) (a fraction 2^-j of [0, 2^m) has places 2^-j as large, and the sum of 4^-j is
1/3), which is (f - 2/3) / f^2 2^-23 F and at most 3/8 2^-23 F (f = 4/3).  So F comes out
too small by at most 1.01 T 2.375 3/8 2^-23 of itself: 8.8e-4 over a run of 131072
products, the longest there is; runs are added in fp32 arithmetic, 2^-24 of the sum each.
524288 products in one run come out some 2.8e-3 too small.

Forward the exact result, rounded, is taken off as the residual, so that what is left is
rounded by 2^-8 of 2^-8 of the result.  Of dx the mean of the signed errors is taken: its
roundings (half a step, 2^-8, at most; scales of rows and columns spread the values over
an octave and a half) have a root mean square below 2^-8 3^-1/2, the mean of 40000 of them
below 1.2e-5; 6e-5 is allowed.
"""
import pytest
import torch

from test_gpu_linear import flp  # noqa: F401 (fixture)

pytestmark = pytest.mark.gpu
RUN = 1.01 * 131072 / 16 * 2.375 * 0.375 * 2.0 ** -23


def positive(rows, cols, seed, by_row=None, by_col=None):
    g = torch.Generator(device="cuda").manual_seed(seed)
    t = torch.rand(rows, cols, generator=g, device="cuda", dtype=torch.bfloat16).add_(0.5)
    return t if by_row is None and by_col is None else t.mul_(by_row[:, None] if by_col is None else by_col)


def some(n, most):
    """Up to `most` of n rows or columns, from the first to the last."""
    return torch.linspace(0, n - 1, min(n, most), device="cuda").long()


@pytest.mark.parametrize("M,N,K", [(2560, 8192, 524288),    # more tiles than CTA pairs, four runs or more each
                                   (2560, 1024, 524288),    # fewer
                                   (300, 513, 1048577),     # rows at odd places; nine runs
                                   (600, 2432, 1040000),    # turned tiles, eight CTAs each
                                   (40, 200, 1100000),      # more than a cluster of them takes
                                   (1, 40, 1100000)])
def test_forward(flp, M, N, K):  # noqa: F811
    x, W = positive(M, K, 1), positive(N, K, 2)
    rows, cols = some(M, 40), some(N, 60)
    want = x[rows].double() @ W[cols].double().t()
    r = torch.zeros(M, N, dtype=torch.bfloat16, device="cuda")
    r[rows[:, None], cols] = -want.to(torch.bfloat16)
    y = flp.linear(x, W, residual=r)
    off = y[rows[:, None], cols].double() - (want + r[rows[:, None], cols].double())
    runs = K // 131072 + 8
    tol = RUN + 2.0 ** -24 * (runs + 2)
    assert float((off.abs() / want).max()) <= tol + 2.0 ** -8 * (2.0 ** -8 + tol)
    assert torch.equal(flp.linear(x, W, residual=r), y)


@pytest.mark.parametrize("M,K,N", [(2560, 8192, 524288),   # more tiles than CTA pairs
                                   (600, 2432, 1040000),   # turned tiles
                                   (40, 1000, 1100000)])   # too deep for a cluster of them
def test_gradient_of_the_input(flp, M, K, N):  # noqa: F811
    g = torch.Generator(device="cuda").manual_seed(3)
    dy = positive(M, N, 1, by_row=1 + torch.rand(M, generator=g, device="cuda", dtype=torch.bfloat16))
    W = positive(N, K, 2, by_col=1 + torch.rand(K, generator=g, device="cuda", dtype=torch.bfloat16))
    x = torch.zeros(M, K, dtype=torch.bfloat16, device="cuda")
    dx, _, _ = flp.linear_backward(dy, x, W, want_dW=False, want_dbias=False)
    rows, cols = some(M, 40), some(K, 1000)
    want = dy[rows].double() @ W[:, cols].double()
    off = ((dx[rows[:, None], cols].double() - want) / want).mean()
    runs = N // 131072 + 8
    assert -(RUN + 2.0 ** -24 * (runs + 2)) - 6e-5 <= float(off) <= 6e-5
