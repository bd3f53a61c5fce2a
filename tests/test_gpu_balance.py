"""The router balance loss, its gradient and the per-expert counts on the GPU
against the definition in 64 bits.

Tolerances.  The counts are whole numbers: equal.  A probability is off by the
exponential (2 units), its argument (one rounding of a difference below 128:
at most 64 units of 2^-24 of a number whose exponential is that small) and a
sum of up to 32 + 5 terms: below 2^-17 of itself.  The gradient is
coef / N p (a - sum p a), so its error is below 2^-16 coef / N p (|a| + sum p |a|),
and the loss's below 2^-17 coef (1 + sum |a| p).  A bf16 gradient adds 2^-8 of its
value.
"""
import numpy as np
import pytest
import torch

import step_reference as ref

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def flp():
    if not torch.cuda.is_available():
        pytest.skip("needs a CUDA GPU")
    from entropy_loss_gb300 import build, flp as _flp
    build.build()
    _flp.load()
    return _flp


def check(flp, z, k, coef=1.0, mask=None, experts=None):
    loss, grad, counts = flp.balance_loss(z, k, coef=coef, mask=mask, experts=experts)
    Z = z.double().cpu().numpy()
    rl, rg, rc, a, p, n, live = ref.balance(Z, k, coef, None if mask is None else mask.cpu().numpy(),
                                            None if experts is None else experts.cpu().numpy())
    assert np.array_equal(counts.cpu().numpy(), rc)
    assert grad.dtype is z.dtype and grad.shape == z.shape
    G = grad.double().cpu().numpy()
    assert np.array_equal(np.isnan(G), np.isnan(rg))
    got = float(loss)
    if np.isnan(rl):
        assert np.isnan(got)
    else:
        mean_p = p[live].sum(0) / max(n, 1)
        assert abs(got - rl) <= 2.0 ** -17 * abs(coef) * (1 + (np.abs(a) * mean_p).sum())
    ok = ~np.isnan(rg)
    size = abs(coef) / max(n, 1) * p * (np.abs(a) + (p * np.abs(a)).sum(1, keepdims=True))
    tol = 2.0 ** -16 * size + (2.0 ** -8 if z.dtype is torch.bfloat16 else 2.0 ** -22) * np.abs(rg) + 1e-38
    assert np.all(np.abs(G - rg)[ok] <= tol[ok])
    again = flp.balance_loss(z, k, coef=coef, mask=mask, experts=experts)
    assert torch.equal(again[2], counts) and (np.isnan(rl) or torch.equal(again[0], loss))
    assert torch.equal(again[1].nan_to_num(7.0), grad.nan_to_num(7.0))
    # without the gradient: the same loss and counts
    l2, none, c2 = flp.balance_loss(z, k, coef=coef, mask=mask, experts=experts, grad=False)
    assert none is None and torch.equal(c2, counts) and (np.isnan(rl) or torch.equal(l2, loss))


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("T,E,k", [(1, 1, 1), (1, 2, 2), (64, 8, 2), (33, 5, 1), (257, 9, 3), (100, 16, 4), (77, 17, 17), (513, 32, 2),
                                   (300, 60, 4), (130, 64, 6), (999, 100, 8), (50, 128, 8), (61, 160, 6), (700, 256, 8),
                                   (40, 257, 32), (20, 512, 10), (9, 1000, 3), (5, 1024, 1024), (3000, 8, 1)])
def test_loss_gradient_and_counts(flp, T, E, k, dtype):
    g = torch.Generator().manual_seed(T * 31 + E)
    z = (1.5 * torch.randn(T, E, generator=g) + 0.7 * torch.randn(E, generator=g)).to(dtype).cuda()
    check(flp, z, k)
    check(flp, z, k, coef=0.01, mask=(torch.rand(T, generator=g) < 0.7).cuda())


@pytest.mark.parametrize("E,k", [(30, 5), (33, 20), (64, 24), (130, 17), (256, 24), (256, 25), (300, 32), (1000, 20)])
def test_many_chosen_of_odd_rows(flp, E, k):
    """More experts a token than any lane's share, and rows that hold ties, few
    numbers, the type's lowest value, or values that are none."""
    g = torch.Generator().manual_seed(E + k)
    z = torch.randn(600, E, generator=g)
    z[10:20] = torch.randint(0, 3, (10, E), generator=g).float()
    z[20:30, : E // 2] = -float("inf")
    z[30] = -float("inf")
    z[31, 3:] = -float("inf")
    z[32] = torch.finfo(torch.float32).min
    z[33, ::2] = torch.finfo(torch.float32).min
    z[34, 1::2] = 0.0
    z[34, ::2] = -0.0
    z[35] = z[35].sort().values               # the largest are neighbours
    z[36] *= 1e-40                            # subnormal numbers
    check(flp, z.cuda(), k)
    check(flp, z.to(torch.bfloat16).cuda(), k)
    z[40, 0], z[41, E - 1], z[42, 1] = float("nan"), float("inf"), -float("nan")
    check(flp, z.cuda(), k)


def test_many_rows_of_one_warp(flp):
    g = torch.Generator().manual_seed(4)
    for T, E, k in ((90000, 33, 5), (90000, 20, 20), (200000, 8, 2)):
        check(flp, torch.randn(T, E, generator=g).cuda(), k)


def test_ties_go_to_the_lowest_index(flp):
    for E in (3, 8, 40, 200):
        z = torch.zeros(50, E, device="cuda")
        z[10:20] = torch.randint(0, 3, (10, E)).float().cuda()
        z[20:30, ::2] = -0.0
        check(flp, z, min(E, 3))
        check(flp, z.to(torch.bfloat16), min(E, 2))


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_masks_that_leave_nothing(flp, dtype):
    z = torch.randn(40, 24, device="cuda").to(dtype)
    check(flp, z, 4, mask=torch.zeros(40, dtype=torch.bool, device="cuda"))
    z[7] = -float("inf")                      # no expert left
    z[8, 2:] = -float("inf")                  # fewer than top_k left
    z[9, 5] = -float("inf")
    z[10] = torch.finfo(dtype).min            # the type's lowest value is a number
    z[11, 3:] = torch.finfo(dtype).min
    z[12] = torch.finfo(dtype).max
    check(flp, z, 4)
    z[:] = -float("inf")
    check(flp, z, 4)


def test_bad_values_stay_in_their_rows(flp):
    z = torch.randn(40, 24, device="cuda")
    mask = torch.ones(40, dtype=torch.bool, device="cuda")
    z[3, 4], z[5, 6] = float("nan"), float("inf")
    mask[3] = mask[5] = False                 # what masked rows hold is not looked at
    check(flp, z, 4, mask=mask)
    check(flp, z, 4)                          # a NaN loss, and NaN in rows 3 and 5 alone


def test_given_experts(flp):
    g = torch.Generator().manual_seed(1)
    for T, E, k in ((90, 12, 2), (33, 64, 8), (10, 300, 40)):
        z = torch.randn(T, E, generator=g).cuda()
        experts = torch.randint(0, E, (T, k), generator=g)
        experts[::5, 0] = -1                  # dropped slots
        experts[3, 1] = E
        check(flp, z, k, experts=experts.cuda(), mask=(torch.rand(T, generator=g) < 0.8).cuda())
        check(flp, z, k, experts=torch.full((T, k), -1, device="cuda"))


@pytest.mark.parametrize("E,pitch,offset", [(8, 8, 0), (8, 3, 1), (30, 2, 1), (128, 5, 0)])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_pitch_and_alignment(flp, E, pitch, offset, dtype):
    z = ref.rows_of(55, E, dtype, "cuda", pitch, offset, torch.Generator().manual_seed(E))
    check(flp, z, 2)


def test_no_tokens(flp):
    loss, grad, counts = flp.balance_loss(torch.empty(0, 8, device="cuda"), 2)
    assert float(loss) == 0 and grad.shape == (0, 8) and not counts.any()


def test_gradient_against_differences(flp):
    """Central differences of the loss in 64 bits with the counts held, h = 1e-4."""
    g = torch.Generator().manual_seed(9)
    z = torch.randn(12, 10, generator=g).cuda()
    _, grad, counts = flp.balance_loss(z, 3, coef=0.5)
    Z, c = z.double().cpu().numpy(), counts.cpu().numpy()

    def loss(Z):
        e = np.exp(Z - Z.max(1, keepdims=True))
        return 0.5 * 10 * (c / c.sum() * (e / e.sum(1, keepdims=True)).mean(0)).sum()

    for t in range(12):
        for j in range(10):
            d = np.zeros_like(Z)
            d[t, j] = 1e-4
            assert abs((loss(Z + d) - loss(Z - d)) / 2e-4 - float(grad[t, j])) <= 1e-7


def test_even_load_costs_coef(flp):
    E = 16
    z = torch.full((E, E), -30.0, device="cuda")
    z.fill_diagonal_(30.0)
    loss, grad, counts = flp.balance_loss(z, 1, coef=0.25)
    assert abs(float(loss) - 0.25) < 1e-6 and (counts == 1).all() and grad.abs().max() < 1e-7


def test_many_tokens(flp):
    """More rows than the blocks hold at once: against torch in 64 bits."""
    T, E, k = 70001, 64, 6
    z = torch.randn(T, E, device="cuda").to(torch.bfloat16)
    loss, grad, counts = flp.balance_loss(z, k)
    Z = z.double()
    order = torch.sort(Z, dim=1, descending=True, stable=True).indices[:, :k]
    assert torch.equal(counts, torch.bincount(order.reshape(-1), minlength=E))
    p = torch.softmax(Z, 1)
    f = E * counts.double() / (T * k)
    want = p * (f - (p * f).sum(1, keepdim=True)) / T
    assert abs(float(loss) - float((f * p.mean(0)).sum())) <= 2.0 ** -17 * 2
    assert float((grad.double() - want).abs().max()) <= 2.0 ** -8 * float(want.abs().max())


def test_own_stream(flp):
    z = torch.randn(5000, 64, device="cuda")
    a = flp.balance_loss(z, 4)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    b = flp.balance_loss(z, 4, stream=side)
    torch.cuda.current_stream().wait_stream(side)
    assert all(torch.equal(x, y) for x, y in zip(a, b))


def test_refusals(flp):
    z = torch.randn(8, 16, device="cuda")
    for bad in (0, 17, -1):
        with pytest.raises(flp.FlpError) as e:
            flp.balance_loss(z, bad)
        assert e.value.status == flp.FLP_ERR_INVALID_ARG
    with pytest.raises(flp.FlpError) as e:
        flp.balance_loss(torch.zeros(1, 1025, device="cuda"), 1)
    assert e.value.status == flp.FLP_ERR_UNSUPPORTED
    with pytest.raises(flp.FlpError):
        flp.balance_loss(z, 2, coef=float("inf"))
    with pytest.raises(ValueError):
        flp.balance_loss(z.half(), 2)
    with pytest.raises(ValueError):
        flp.balance_loss(z, 2, mask=torch.ones(8, device="cuda"))
    with pytest.raises(ValueError):
        flp.balance_loss(z, 2, mask=torch.ones(7, dtype=torch.bool, device="cuda"))
    with pytest.raises(ValueError):
        flp.balance_loss(z, 2, experts=torch.zeros(8, 3, dtype=torch.int64, device="cuda"))
    with pytest.raises(ValueError):
        flp.balance_loss(z, 2, experts=torch.zeros(8, 2, dtype=torch.int32, device="cuda"))
    with pytest.raises(flp.FlpError) as e:
        flp.balance_loss(torch.randn(5000, 16, device="cuda"), 2,
                         workspace=torch.empty(64, dtype=torch.uint8, device="cuda"))
    assert e.value.status == flp.FLP_ERR_WORKSPACE
