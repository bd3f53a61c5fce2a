"""A training step with a mixture of experts, end to end on synthetic data.

    h       = gelu(x W_in^T + b_in)              fused_linear
    n       = layer_norm(h)                      fused_layer_norm
    choice  = the top_k experts of n W_router^T, weights their softmax
    m       = h + sum_j weights_j expert_j(n)    expert_sort, fused_expert_gather, a fused_linear
                                                 pair an expert, fused_expert_combine
    lp      = log softmax(m W_head^T)[y]         fused_linear, fused_token_logprob
    loss    = -mean(lp) + balance(n W_router^T)  fused_balance_loss

trained with plain gradient steps on a fixed batch, some of whose tokens are padding.
Prints the loss of every step and, at the end, the most likely tokens of one position.

    python examples/expert_step.py [--steps 20]
"""
import argparse
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
from entropy_loss_gb300 import build, flp  # noqa: E402


class Model:
    def __init__(self, inputs, hidden, inner, vocab, experts, device="cuda", seed=0):
        g = torch.Generator().manual_seed(seed)

        def weight(rows, cols):
            w = torch.randn(rows, cols, generator=g) / cols ** 0.5
            return w.to(device, torch.bfloat16).requires_grad_()

        self.w_in, self.w_router, self.w_head = weight(hidden, inputs), weight(experts, hidden), weight(vocab, hidden)
        self.b_in = torch.zeros(hidden, device=device, dtype=torch.bfloat16).requires_grad_()
        self.norm_w = torch.ones(hidden, device=device, requires_grad=True)
        self.norm_b = torch.zeros(hidden, device=device, requires_grad=True)
        self.up = [weight(inner, hidden) for _ in range(experts)]
        self.down = [weight(hidden, inner) for _ in range(experts)]

    def parameters(self):
        return [self.w_in, self.b_in, self.w_router, self.w_head, self.norm_w, self.norm_b, *self.up, *self.down]

    def experts(self, n, scores, top_k, tokens):
        """(the experts' output for each token, the choice): padding goes to no expert."""
        top = scores.float().topk(top_k, dim=1)
        choice = torch.where(tokens[:, None], top.indices, -1)
        order = flp.expert_sort(choice, len(self.up))
        xs = flp.fused_expert_gather(n, order)
        sizes = order.counts.tolist()
        parts = list(xs.split(sizes + [len(xs) - sum(sizes)]))  # the slots without an expert stay as they are
        for i, rows in enumerate(parts[:-1]):
            if len(rows):
                parts[i] = flp.fused_linear(flp.fused_linear(rows, self.up[i], activation="silu"), self.down[i])
        return flp.fused_expert_combine(torch.cat(parts), order, torch.softmax(top.values, 1)), choice

    def logits(self, x, tokens, top_k):
        h = flp.fused_linear(x, self.w_in, self.b_in, "gelu")
        n = flp.fused_layer_norm(h, self.norm_w, self.norm_b)
        scores = n @ self.w_router.t()
        mixed, choice = self.experts(n, scores, top_k, tokens)
        return flp.fused_linear(h + mixed, self.w_head), scores, choice

    def loss(self, x, y, top_k=2, balance=0.01):
        """(loss, token loss, balance loss, tokens per expert, the experts' choice)"""
        tokens = y != -100
        logits, scores, choice = self.logits(x, tokens, top_k)
        logprob, _, _, _ = flp.fused_token_logprob(logits, y, compute_entropy=False)
        nll = -logprob.sum() / tokens.sum()
        even, counts = flp.fused_balance_loss(scores, top_k, experts=choice, mask=tokens, coef=balance)
        return nll + even, nll, even, counts, choice


def batch(rows, inputs, vocab, device="cuda", seed=1):
    g = torch.Generator().manual_seed(seed)
    x = torch.randn(rows, inputs, generator=g).to(device, torch.bfloat16)
    y = torch.randint(0, vocab, (rows,), generator=g)
    y[torch.rand(rows, generator=g) < 0.1] = -100  # padding
    return x, y.to(device)


def train(steps=20, rows=512, inputs=256, hidden=512, inner=384, vocab=4096, experts=8, rate=0.5):
    model = Model(inputs, hidden, inner, vocab, experts)
    x, y = batch(rows, inputs, vocab)
    history = []
    for step in range(steps):
        loss, nll, even, counts, _ = model.loss(x, y)
        loss.backward()
        with torch.no_grad():
            for p in model.parameters():
                if p.grad is not None:  # an expert without tokens has none
                    p -= rate * p.grad
                    p.grad = None
        history.append(float(loss.detach()))
        print(f"step {step:3d}  loss {history[-1]:.4f}  token loss {float(nll.detach()):.4f}  balance {float(even.detach()):.5f}  "
              f"tokens per expert {int(counts.min())}..{int(counts.max())}")
    with torch.no_grad():
        logits, _, _ = model.logits(x[:1], y[:1] != -100, 2)
        logprob, _, entropy, values, index = flp.token_logprob(logits, y[:1], top=5)
    print(f"token {int(y[0])}: log-probability {float(logprob[0]):.3f}, entropy {float(entropy[0]):.3f}, most likely "
          + ", ".join(f"{i} ({v:.2f})" for i, v in zip(index[0].tolist(), values[0].tolist())))
    return history


if __name__ == "__main__":
    ap = argparse.ArgumentParser(description=__doc__.splitlines()[0])
    ap.add_argument("--steps", type=int, default=20)
    build.build()
    train(ap.parse_args().steps)
