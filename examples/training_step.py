"""A training step with the library's operators, end to end on synthetic data.

A small model of one projection, a final layer norm, a mixture-of-experts router
and the fused head:

    h      = x W_in^T                      checkpoint_linear: x is kept in 8 bits
    n      = layer_norm(h)                 fused_layer_norm: h is kept in 8 bits
    lp     = log softmax(n W_head^T)[y]    fused_linear_logprob: logits never stored
    loss   = -mean(lp) + balance(n W_router^T)

trained with plain gradient steps on a fixed batch, some of whose tokens are
padding.  Prints the loss of every step.

    python examples/training_step.py [--steps 20]
"""
import argparse
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
from entropy_loss_gb300 import build, flp  # noqa: E402


class Model:
    def __init__(self, inputs, hidden, vocab, experts, device="cuda", seed=0):
        g = torch.Generator().manual_seed(seed)

        def weight(rows, cols):
            w = torch.randn(rows, cols, generator=g) / cols ** 0.5
            return w.to(device, torch.bfloat16).requires_grad_()

        self.w_in, self.w_head, self.w_router = weight(hidden, inputs), weight(vocab, hidden), weight(experts, hidden)
        self.norm_w = torch.ones(hidden, device=device, requires_grad=True)
        self.norm_b = torch.zeros(hidden, device=device, requires_grad=True)

    def parameters(self):
        return [self.w_in, self.w_head, self.w_router, self.norm_w, self.norm_b]

    def loss(self, x, y, top_k=2, balance=0.01):
        """(loss, token loss, balance loss, tokens per expert)"""
        h = flp.checkpoint_linear(x, self.w_in)
        n = flp.fused_layer_norm(h, self.norm_w, self.norm_b, checkpoint=True)
        logprob, _ = flp.fused_linear_logprob(n, self.w_head, y, compute_entropy=False)
        tokens = y != -100
        nll = -logprob.sum() / tokens.sum()
        even, counts = flp.fused_balance_loss(n @ self.w_router.t(), top_k, mask=tokens, coef=balance)
        return nll + even, nll, even, counts


def batch(rows, inputs, vocab, device="cuda", seed=1):
    g = torch.Generator().manual_seed(seed)
    x = torch.randn(rows, inputs, generator=g).to(device, torch.bfloat16)
    y = torch.randint(0, vocab, (rows,), generator=g)
    y[torch.rand(rows, generator=g) < 0.1] = -100  # padding
    return x, y.to(device)


def train(steps=20, rows=512, inputs=256, hidden=512, vocab=4096, experts=16, rate=0.5):
    model = Model(inputs, hidden, vocab, experts)
    x, y = batch(rows, inputs, vocab)
    history = []
    for step in range(steps):
        loss, nll, even, counts = model.loss(x, y)
        loss.backward()
        with torch.no_grad():
            for p in model.parameters():
                p -= rate * p.grad
                p.grad = None
        history.append(float(loss.detach()))
        print(f"step {step:3d}  loss {history[-1]:.4f}  token loss {float(nll.detach()):.4f}  balance {float(even.detach()):.5f}  "
              f"tokens per expert {int(counts.min())}..{int(counts.max())}")
    return history


if __name__ == "__main__":
    ap = argparse.ArgumentParser(description=__doc__.splitlines()[0])
    ap.add_argument("--steps", type=int, default=20)
    build.build()
    train(ap.parse_args().steps)
