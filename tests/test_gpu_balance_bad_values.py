"""The balance loss when the live rows hold a NaN or +inf: the loss is NaN, and
the gradient in those rows, also where they choose nobody (C = 0)."""
import pytest
import torch

pytestmark = pytest.mark.gpu
BAD = [float("nan"), float("inf")]


@pytest.fixture(scope="module")
def flp():
    if not torch.cuda.is_available():
        pytest.skip("needs a CUDA GPU")
    from entropy_loss_gb300 import build, flp as _flp
    build.build()
    _flp.load()
    return _flp


# one launch of one cluster, and three launches; 8, 16 and 32 lanes a row
SIZES = [(1, 8), (40, 12), (70, 200), (5000, 8), (5000, 100), (3000, 1000)]


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("bad", BAD)
@pytest.mark.parametrize("T,E", SIZES)
def test_every_live_row_is_bad(flp, T, E, bad, dtype):
    z = torch.randn(T, E, device="cuda").to(dtype)
    z[:, E // 2] = bad
    loss, grad, counts = flp.balance_loss(z, 2)
    assert torch.isnan(loss).all() and torch.isnan(grad).all() and not counts.any()
    assert torch.isnan(flp.balance_loss(z, 2, grad=False)[0]).all()
    loss, grad, counts = flp.balance_loss(torch.full_like(z, bad), 2)
    assert torch.isnan(loss).all() and torch.isnan(grad).all() and not counts.any()


@pytest.mark.parametrize("bad", BAD)
@pytest.mark.parametrize("T,E", SIZES)
def test_the_only_live_row_is_bad(flp, T, E, bad):
    z = torch.full((T, E), -float("inf"), device="cuda")   # not live
    z[T // 2, 0] = bad
    loss, grad, counts = flp.balance_loss(z, 2)
    assert torch.isnan(loss).all() and not counts.any()
    assert torch.isnan(grad[T // 2]).all() and not grad[:T // 2].any() and not grad[T // 2 + 1:].any()
    mask = torch.zeros(T, dtype=torch.bool, device="cuda")
    z[:] = bad
    loss, grad, counts = flp.balance_loss(z, 2, mask=mask)   # what masked rows hold is not looked at
    assert float(loss) == 0 and not grad.any() and not counts.any()
    mask[T // 2] = True
    loss, grad, counts = flp.balance_loss(z, 2, mask=mask)
    assert torch.isnan(loss).all() and torch.isnan(grad[T // 2]).all() and not counts.any()
    assert not grad[~mask].any()


@pytest.mark.parametrize("T,E", SIZES)
def test_given_experts_that_are_all_dropped(flp, T, E):
    z = torch.randn(T, E, device="cuda")
    dropped = torch.full((T, 2), -1, device="cuda")
    loss, grad, counts = flp.balance_loss(z, 2, experts=dropped)
    assert float(loss) == 0 and not grad.any() and not counts.any()
    z[T - 1, E - 1] = float("nan")
    loss, grad, counts = flp.balance_loss(z, 2, experts=dropped)
    assert torch.isnan(loss).all() and torch.isnan(grad[T - 1]).all() and not grad[:T - 1].any() and not counts.any()
