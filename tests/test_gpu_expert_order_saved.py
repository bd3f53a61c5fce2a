"""The autograd wrappers of the experts' moves notice an order that was written over
between the forward and the backward pass, as of any tensor that a gradient needs."""
import pytest
import torch

from test_gpu_experts import flp  # noqa: F401 (fixture)

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("which", ["rows", "offsets"])
def test_orders_written_over(flp, which):  # noqa: F811
    e = torch.randint(0, 5, (40, 2), device="cuda")
    x = torch.randn(40, 64, device="cuda", requires_grad=True)
    w = torch.rand(40, 2, device="cuda", requires_grad=True)
    for f in (lambda order: flp.fused_expert_gather(x, order),
              lambda order: flp.fused_expert_combine(torch.cat([x, x]), order, w),
              lambda order: flp.fused_expert_combine(torch.cat([x, x]), order)):
        order = flp.expert_sort(e, 5)
        y = f(order)
        getattr(order, which).copy_(getattr(flp.expert_sort((e + 1) % 6, 5), which))
        with pytest.raises(RuntimeError, match="modified by an inplace operation"):
            y.sum().backward()
        f(flp.expert_sort(e, 5)).sum().backward()


def test_a_step_in_a_graph(flp):  # noqa: F811
    """The wrappers' forward and backward passes captured together, replayed on new inputs."""
    T, H, V, E = 70, 128, 1003, 4
    g = torch.Generator().manual_seed(1)

    def leaf(*shape, scale=1.0):
        return (scale * torch.randn(*shape, generator=g)).cuda().bfloat16().requires_grad_()

    x, W, head, b = leaf(T, H), leaf(H, H, scale=H ** -0.5), leaf(V, H, scale=H ** -0.5), leaf(H)
    gates = torch.rand(T, 2, generator=g).cuda()
    e = torch.randint(-1, E, (T, 2), generator=g).cuda()
    y = torch.randint(0, V, (T,), generator=g).cuda()

    def step():
        order = flp.expert_sort(e, E)
        xs = flp.fused_linear(flp.fused_expert_gather(x, order), W, b, activation="gelu")
        z = flp.fused_linear(x + flp.fused_expert_combine(xs, order, gates), head)
        lp, ent, val, idx = flp.fused_token_logprob(z, y, top=3)
        return [lp, ent, val, idx, *torch.autograd.grad((lp + 0.1 * ent).sum(), (x, W, b, head))]

    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        step()
    s.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=s):
        out = step()
    with torch.no_grad():
        x.mul_(-0.5)
        e.copy_((e + 2) % (E + 1))
        y.copy_((y + 17) % V)
    for _ in range(2):
        graph.replay()
    torch.cuda.synchronize()
    for a, want in zip(out, step()):
        assert torch.equal(a, want)
