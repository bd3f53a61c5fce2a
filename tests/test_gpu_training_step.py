"""The training-step operators together: the differentiable wrappers against
64-bit autograd, and the example's loop.

Tolerance of the gradients.  An 8-bit checkpoint keeps a value to half a step,
at most 2^-7 of its block's largest; over random data that is a relative error
below 2^-6 of the activations in the 2-norm, and it enters the weight gradients
and the norm's backward linearly.  Products and outputs in bf16 add a few times
2^-9.  2 % (relative 2-norm) covers both.
"""
import importlib.util
import os

import pytest
import torch

pytestmark = pytest.mark.gpu
ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.fixture(scope="module")
def flp():
    if not torch.cuda.is_available():
        pytest.skip("needs a CUDA GPU")
    from entropy_loss_gb300 import build, flp as _flp
    build.build()
    _flp.load()
    return _flp


@pytest.fixture(scope="module")
def example(flp):
    spec = importlib.util.spec_from_file_location("training_step", os.path.join(ROOT, "examples", "training_step.py"))
    m = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(m)
    return m


def close(got, want, tol=0.02):
    rel = float((got.double() - want).norm() / want.norm())
    assert rel <= tol, rel


def test_gradients_of_the_whole_step(flp, example):
    rows, inputs, hidden, vocab, experts = 300, 128, 264, 1000, 12
    model = example.Model(inputs, hidden, vocab, experts)
    with torch.no_grad():
        model.norm_w.copy_(1 + 0.2 * torch.randn(hidden, device="cuda"))
        model.norm_b.copy_(0.2 * torch.randn(hidden, device="cuda"))
    x, y = example.batch(rows, inputs, vocab)
    loss, nll, even, counts = model.loss(x, y, top_k=3, balance=0.5)
    loss.backward()

    ref = [p.detach().double().requires_grad_() for p in model.parameters()]
    w_in, w_head, w_router, norm_w, norm_b = ref
    h = x.double() @ w_in.t()
    n = torch.nn.functional.layer_norm(h, (hidden,), norm_w, norm_b, 1e-5)
    tokens = y != -100
    lp = torch.log_softmax(n @ w_head.t(), 1).gather(1, y.clamp(min=0)[:, None])[:, 0]
    p = torch.softmax(n @ w_router.t(), 1)
    f = counts.double() / counts.sum()
    want = -lp[tokens].mean() + 0.5 * experts * (f * p[tokens].mean(0)).sum()
    want.backward()
    assert int(counts.sum()) == 3 * int(tokens.sum())
    assert abs(float(loss.detach()) - float(want.detach())) <= 0.01 * abs(float(want.detach()))
    for got, r in zip(model.parameters(), ref):
        assert got.grad.dtype is got.dtype
        close(got.grad, r.grad)


def test_layer_norm_wrapper(flp):
    for checkpoint, tol in ((False, 0.005), (True, 0.02)):
        x = (torch.randn(70, 300, device="cuda") + 0.5).to(torch.bfloat16).requires_grad_()
        w = torch.randn(300, device="cuda").to(torch.bfloat16).requires_grad_()
        g = torch.randn(300, 70, device="cuda").to(torch.bfloat16).t()  # an upstream gradient that is not contiguous
        flp.fused_layer_norm(x, w, None, checkpoint=checkpoint).backward(g)
        xr, wr = x.detach().double().requires_grad_(), w.detach().double().requires_grad_()
        torch.nn.functional.layer_norm(xr, (300,), wr, None, 1e-5).backward(g.double())
        close(x.grad, xr.grad, tol)
        close(w.grad, wr.grad, tol)


def test_linear_wrapper_keeps_what_is_needed(flp):
    x = torch.randn(64, 96, device="cuda").to(torch.bfloat16)
    w = torch.randn(32, 96, device="cuda").to(torch.bfloat16).requires_grad_()
    flp.checkpoint_linear(x, w).sum().backward()      # no gradient by x
    close(w.grad, torch.ones(64, 32, device="cuda").double().t() @ x.double())
    x.requires_grad_()
    frozen = w.detach()
    flp.checkpoint_linear(x, frozen).sum().backward()  # none by W
    close(x.grad, torch.ones(64, 32, device="cuda").double() @ frozen.double(), 0.005)


def test_balance_wrapper_scales_its_gradient(flp):
    z = torch.randn(50, 8, device="cuda", requires_grad=True)
    loss, counts = flp.fused_balance_loss(z, 2, coef=0.3)
    (3 * loss).backward()
    _, grad, c = flp.balance_loss(z.detach(), 2, coef=0.3)
    assert torch.equal(z.grad, 3 * grad) and torch.equal(counts, c)


def test_example_learns(example):
    history = example.train(steps=12)
    assert all(h == h for h in history)
    assert history[-1] < history[0] - 0.5
