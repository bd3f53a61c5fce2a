"""The differentiable wrappers of the training-step operators: types, scales, and
what they refuse or leave out.

Tolerance of the bf16 balance gradient: each value is rounded to bf16 by half a
unit, and carries the fp32 kernel's error (test_gpu_balance.py): below 2^-7 of
itself.  Rounding to nearest has no direction, so the mean over 4000 values of the
relative error stays below 2^-9 / 8.
"""
import pytest
import torch

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def flp():
    if not torch.cuda.is_available():
        pytest.skip("needs a CUDA GPU")
    from entropy_loss_gb300 import build, flp as _flp
    build.build()
    _flp.load()
    return _flp


@pytest.mark.parametrize("scale", [1.0, 1.00390625 - 2.0 ** -9, 1 / 3, 1000.7])
def test_balance_gradient_in_bf16_is_scaled_without_a_shift(flp, scale):
    g = torch.Generator().manual_seed(2)
    z = torch.randn(500, 8, generator=g).to(torch.bfloat16).cuda().requires_grad_()
    loss, counts = flp.fused_balance_loss(z, 2, coef=0.3)
    (loss * scale).backward()
    assert z.grad.dtype is torch.bfloat16
    p = torch.softmax(z.detach().double(), 1)
    a = 8 * counts.double() / counts.sum() - 1
    want = scale * 0.3 / 500 * p * (a - (p * a).sum(1, keepdim=True))
    off = (z.grad.double() - want) / want.abs().clamp(min=1e-30) * want.sign()
    assert float(off.abs()[want.abs() > 1e-3 * want.abs().max()].max()) <= 2.0 ** -7
    assert abs(float(off[want.abs() > 1e-3 * want.abs().max()].mean())) <= 2.0 ** -12
    # the kernel's fp32 gradient, multiplied in fp32 and rounded once
    _, grad, _ = flp.balance_loss(z.detach(), 2, coef=0.3, grad_dtype=torch.float32)
    assert torch.equal(z.grad, (grad * scale).to(torch.bfloat16))


@pytest.mark.parametrize("T,E", [(1, 1), (40, 7), (40, 8), (100, 64), (700, 100), (700, 101), (3000, 16), (5000, 256), (900, 1000)])
def test_balance_gradient_in_fp32_of_bf16_logits(flp, T, E):
    """In either type the same gradient; the kernel's own bf16 one is its rounding."""
    z = torch.randn(T, E, device="cuda").to(torch.bfloat16)
    loss, full, counts = flp.balance_loss(z, 1, grad_dtype=torch.float32)
    l2, half, c2 = flp.balance_loss(z, 1)
    assert full.dtype is torch.float32 and half.dtype is torch.bfloat16
    assert torch.equal(loss, l2) and torch.equal(counts, c2) and torch.equal(full.to(torch.bfloat16), half)
    # the 32-bit logits of the same values
    assert torch.allclose(flp.balance_loss(z.float(), 1)[1], full, rtol=1e-5, atol=0)
    with pytest.raises(ValueError):
        flp.balance_loss(z.float(), 1, grad_dtype=torch.bfloat16)


# --------------------------------------------------- gradients of gradients

TWICE = "cannot be differentiated again"


def test_balance_gradient_is_not_a_constant_of_the_logits(flp):
    z = torch.randn(50, 8, device="cuda", requires_grad=True)
    w = torch.tensor(2.0, device="cuda", requires_grad=True)
    loss, _ = flp.fused_balance_loss(z, 2)
    dz, = torch.autograd.grad(loss * w, z, create_graph=True)
    with pytest.raises(RuntimeError, match=TWICE):
        torch.autograd.grad(dz.square().sum() + z.sum(), z)
    # the same where the upstream gradient is a constant
    loss, _ = flp.fused_balance_loss(z, 2)
    dz, = torch.autograd.grad(loss, z, create_graph=True)
    with pytest.raises(RuntimeError, match=TWICE):
        torch.autograd.grad(dz.square().sum() + z.sum(), z)
    # the gradient itself is the one without create_graph
    loss, _ = flp.fused_balance_loss(z, 2)
    assert torch.equal(dz.detach(), torch.autograd.grad(loss, z)[0])


@pytest.mark.parametrize("checkpoint", [False, True])
def test_norm_gradient_is_not_a_constant(flp, checkpoint):
    x = torch.randn(20, 64, device="cuda", requires_grad=True)
    w = torch.rand(64, device="cuda", requires_grad=True)
    y = flp.fused_layer_norm(x, w, None, checkpoint=checkpoint)
    dx, dw = torch.autograd.grad(y.square().sum(), (x, w), create_graph=True)
    for d in (dx, dw):
        with pytest.raises(RuntimeError, match=TWICE):
            torch.autograd.grad(d.square().sum() + x.sum() + w.sum(), (x, w), retain_graph=True)
    y = flp.fused_layer_norm(x, w, None, checkpoint=checkpoint)
    once = torch.autograd.grad(y.square().sum(), (x, w))
    assert torch.equal(dx.detach(), once[0]) and torch.equal(dw.detach(), once[1])


def test_linear_gradients_of_gradients(flp):
    """dx = dy W is an ordinary product and can be differentiated, dW cannot."""
    x = torch.randn(32, 64, device="cuda").to(torch.bfloat16).requires_grad_()
    W = torch.randn(16, 64, device="cuda").to(torch.bfloat16).requires_grad_()
    dx, dW = torch.autograd.grad(flp.checkpoint_linear(x, W).float().square().sum(), (x, W), create_graph=True)
    with pytest.raises(RuntimeError, match=TWICE):
        torch.autograd.grad(dW.float().square().sum(), W, retain_graph=True)
    twice, = torch.autograd.grad(dx.float().sum(), x)
    want, = torch.autograd.grad((x.double() @ W.double().t()).square().sum(), x, create_graph=True)
    want, = torch.autograd.grad(want.sum(), x)
    assert float((twice.double() - want.double()).norm() / want.double().norm()) <= 0.02


def test_linear_refuses_what_its_backward_cannot_do(flp):
    x = torch.randn(32, 64, device="cuda")
    W = torch.randn(16, 64, device="cuda", requires_grad=True)
    with pytest.raises(ValueError):
        flp.checkpoint_linear(x, W)
    with pytest.raises(ValueError):
        flp.checkpoint_linear(x.to(torch.bfloat16), W)
    # without a gradient by W nothing is kept
    frozen = W.detach()
    x.requires_grad_()
    flp.checkpoint_linear(x, frozen).sum().backward()
    assert torch.equal(x.grad, torch.ones(32, 16, device="cuda") @ frozen)


def test_the_stream_of_a_device_without_the_short_way(flp):
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        assert flp._stream_of(0) == flp._raw_stream(0) == side.cuda_stream
    assert flp._stream_of(0) == flp._raw_stream(0) == torch.cuda.current_stream().cuda_stream


def test_only_a_backward_pass_is_prepared_for(flp, monkeypatch):
    """Without one no checkpoint is written and no gradient taken, in eval loops
    (no_grad) as well as where no input needs a gradient."""
    seen = []
    norm, pack, balance = flp.layer_norm, flp.checkpoint_pack, flp.balance_loss
    monkeypatch.setattr(flp, "layer_norm", lambda *a, **k: seen.append(k["checkpoint"]) or norm(*a, **k))
    monkeypatch.setattr(flp, "checkpoint_pack", lambda *a, **k: seen.append("pack") or pack(*a, **k))
    monkeypatch.setattr(flp, "balance_loss", lambda *a, **k: seen.append(k["grad"]) or balance(*a, **k))
    x, w = torch.randn(40, 64, device="cuda").to(torch.bfloat16), torch.rand(64, device="cuda")
    W = torch.randn(16, 64, device="cuda").to(torch.bfloat16)

    def forward():
        n = flp.fused_layer_norm(x, w, None, checkpoint=True)
        z = flp.checkpoint_linear(n, W)
        return (n, z, *flp.fused_balance_loss(z, 2))

    plain = forward()
    assert seen == [False, False]
    for t in (x, w, W):
        t.requires_grad_()
    seen.clear()
    with torch.no_grad():
        off = forward()
    assert seen == [False, False] and not any(t.requires_grad for t in off)
    seen.clear()
    on = forward()
    assert seen == [True, "pack", True]
    assert all(torch.equal(a, b) and torch.equal(a, c) for a, b, c in zip(plain, off, on))
    (on[1].float().sum() + on[2]).backward()
    assert all(t.grad is not None for t in (x, w, W))
