"""The expert, linear and given-logits operators on matrices of more than 2^31 elements,
whose offsets pass 32 bits: rows of both ends and the middle against the same rows in a
small call.  A row's result does not depend on how many rows there are but for the
order of its sums, so the tolerances are twice those of one call (test_gpu_linear.py,
test_gpu_token_logprob.py, test_gpu_experts.py): of bf16 results a step, 2^-7.
"""
import pytest
import torch

from test_gpu_experts import flp  # noqa: F401 (fixture)

pytestmark = pytest.mark.gpu
BF = torch.bfloat16


def normal(rows, cols, seed, scale=1.0):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return torch.empty(rows, cols, dtype=BF, device="cuda").normal_(0, scale, generator=g)


def near(a, b, size=1e-3):
    a, b = a.double(), b.double()
    assert bool(((a - b).abs() <= 2.0 ** -7 * b.abs() + 2.0 ** -16 * size).all())


@pytest.mark.parametrize("extra", [0, 3])
def test_given_logits(flp, extra):  # noqa: F811
    M, V = 16500, 131073
    z = normal(M, V + extra, 1, 2.0)[:, :V]
    y = torch.arange(M, device="cuda") * 7919 % V
    rows = torch.tensor([0, 1, M // 2, M - 2, M - 1], device="cuda")
    lp, lse, ent, val, idx = flp.token_logprob(z, y, top=5)
    few = z[rows].contiguous()
    want = flp.token_logprob(few, y[rows], top=5)
    for a, b in zip((lp, lse, ent, val), want):
        assert bool(((a[rows] - b).abs() <= 1e-5 * (1 + b.abs())).all())
    assert torch.equal(idx[rows], want[4])
    g = torch.full((M,), 0.5, device="cuda")
    dz = flp.token_logprob_backward(z, y, lse, ent, g, g)
    near(dz[rows], flp.token_logprob_backward(few, y[rows], lse[rows], ent[rows], g[:5], g[:5]))
    again = flp.token_logprob_backward(z, y, lse, ent, g, g, out=z)
    assert torch.equal(again[rows], dz[rows])


@pytest.mark.parametrize("H", [5120, 4099])
def test_expert_rows(flp, H):  # noqa: F811
    T, k, E = 67000, 8, 16
    choice = torch.arange(T * k, device="cuda").view(T, k) * 31 % (E + 1)  # some slots without an expert
    order = flp.expert_sort(choice, E)
    x = normal(T, H, 1)
    xs = flp.expert_gather(x, order)
    total = int(order.offsets[-1])
    at = torch.tensor([0, 1, total // 2, total - 1, T * k - 1], device="cuda")
    want = x[order.slots[at].long() // k]
    want[at >= total] = 0
    assert torch.equal(xs[at], want)
    w = torch.rand(T, k, device="cuda")
    y = flp.expert_combine(xs, order, w)
    rows = torch.tensor([0, 1, T // 2, T - 1], device="cuda")
    live = (order.rows.long() < total).double()
    scale = (w.double() * live)[rows].sum(1, keepdim=True)
    near(y[rows], scale * x[rows].double())
    dys, dw = flp.expert_combine_backward(y, xs, order, w)
    slot = order.slots[at].long()
    d = (w.double() * live).reshape(-1)[slot][:, None] * y.double()[slot // k]
    near(dys[at], d)
    want = (y.double()[rows] * x.double()[rows]).sum(1, keepdim=True) * live[rows]
    assert bool(((dw[rows].double() - want).abs() <= 1e-5 * (y.double()[rows] * x.double()[rows]).abs().sum(1, keepdim=True)).all())


@pytest.mark.parametrize("N", [16384, 16387])
def test_linear(flp, N):  # noqa: F811
    M, K = 135000, 64
    x, W = normal(M, K, 1), normal(N, K, 2, 0.125)
    rows = torch.tensor([0, 1, M // 2, M - 2, M - 1], device="cuda")
    r = normal(M, N, 3)
    y, pre = flp.linear(x, W, activation="silu", residual=r, keep=True)
    want, kept = flp.linear(x[rows], W, activation="silu", residual=r[rows], keep=True)
    near(y[rows], want)
    near(pre[rows], kept)
    dx, dW, db = flp.linear_backward(r, x, W, pre, activation="silu", dw_dtype=BF)
    # bf16 d: off by 2^-8 of each of N terms near 0.1 in size, of random sign
    d = r[rows].double() * (torch.sigmoid(pre[rows].double()) * (1 + pre[rows].double() * torch.sigmoid(-pre[rows].double())))
    off = 2.0 ** -8 * (d.abs() @ W.double().abs())
    assert bool(((dx[rows].double() - d @ W.double()).abs() <= off + 2.0 ** -7 * (d @ W.double()).abs()).all())
    cols = torch.tensor([0, N // 2, N - 1], device="cuda")
    p = pre[:, cols].double()
    d = r[:, cols].double() * (torch.sigmoid(p) * (1 + p * torch.sigmoid(-p)))
    want = d.t() @ x.double()
    assert bool(((dW[cols].double() - want).abs() <= 2.0 ** -8 * (d.abs().t() @ x.double().abs()) + 2.0 ** -7 * want.abs()).all())
    assert bool(((db[cols].double() - d.sum(0)).abs() <= 2.0 ** -16 * d.abs().sum(0)).all())
