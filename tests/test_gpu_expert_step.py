"""The expert, linear and given-logits operators together: the example's step against
64-bit autograd, and its loop.

Tolerance of the gradients.  Every activation and gradient between the operators is
rounded to bf16 (2^-9 of it at most, once an operator): about a dozen such roundings lie
between a parameter and the loss, each entering linearly with a factor near 1 in the
2-norm, and their errors are independent: 12^(1/2) 2^-9 < 0.7 %.  2 % (relative 2-norm).
The choice of experts is taken from the step itself, so that it is the same in both.
"""
import importlib.util
import os

import pytest
import torch

pytestmark = pytest.mark.gpu
ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.fixture(scope="module")
def example():
    if not torch.cuda.is_available():
        pytest.skip("needs a CUDA GPU")
    from entropy_loss_gb300 import build, flp
    build.build()
    flp.load()
    spec = importlib.util.spec_from_file_location("expert_step", os.path.join(ROOT, "examples", "expert_step.py"))
    m = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(m)
    return m


def close(got, want, tol=0.02):
    rel = float((got.double() - want).norm() / want.norm())
    assert rel <= tol, rel


def test_gradients_of_the_whole_step(example):
    rows, inputs, hidden, inner, vocab, experts, top_k = 300, 128, 264, 200, 1001, 5, 2
    model = example.Model(inputs, hidden, inner, vocab, experts)
    with torch.no_grad():
        model.norm_w.copy_(1 + 0.2 * torch.randn(hidden, device="cuda"))
        model.b_in.copy_(0.2 * torch.randn(hidden, device="cuda"))
    x, y = example.batch(rows, inputs, vocab)
    loss, nll, even, counts, choice = model.loss(x, y, top_k=top_k, balance=0.5)
    loss.backward()

    ref = [p.detach().double().requires_grad_() for p in model.parameters()]
    w_in, b_in, w_router, w_head, norm_w, norm_b = ref[:6]
    up, down = ref[6:6 + experts], ref[6 + experts:]
    h = torch.nn.functional.gelu(x.double() @ w_in.t() + b_in)
    n = torch.nn.functional.layer_norm(h, (hidden,), norm_w, norm_b, 1e-5)
    scores = n @ w_router.t()
    tokens = y != -100
    # an expert's weight goes by the logits of the chosen, padding's by any of them: it counts nowhere
    weights = torch.softmax(scores.gather(1, choice.clamp(min=0)), 1)
    mixed = torch.zeros_like(h)
    for e in range(experts):
        out = torch.nn.functional.silu(n @ up[e].t()) @ down[e].t()
        mixed = mixed + (weights * (choice == e)).sum(1, keepdim=True) * out
    lp = torch.log_softmax((h + mixed) @ w_head.t(), 1).gather(1, y.clamp(min=0)[:, None])[:, 0]
    p = torch.softmax(scores, 1)
    f = counts.double() / counts.sum()
    want = -lp[tokens].mean() + 0.5 * experts * (f * p[tokens].mean(0)).sum()
    want.backward()
    assert int(counts.sum()) == top_k * int(tokens.sum())
    assert torch.equal(counts, torch.bincount(choice[choice >= 0], minlength=experts))
    assert abs(float(loss.detach()) - float(want.detach())) <= 0.01 * abs(float(want.detach()))
    for got, r in zip(model.parameters(), ref):
        assert got.grad.dtype is got.dtype
        close(got.grad, r.grad)


def test_example_runs(example):
    history = example.train(steps=3)
    assert len(history) == 3 and all(v == v for v in history)
