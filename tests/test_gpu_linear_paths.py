"""Every way that the linear layer's products of many rows are laid out, with data: tiles
of CTA pairs, wide (256 x 512) and narrow (256 x 256), written directly by bulk stores or
row by row, the last round in halves, and tiles split along the contraction and joined;
forward with every activation, and as the backward pass's dx.

What a GPU of 152 SMs (76 pairs) does with each shape stands beside it.  The tolerances
are those of test_gpu_linear.py.
"""
import pytest
import torch

from test_gpu_linear import ACTS, flp, run_backward, run_forward  # noqa: F401 (flp: fixture)

pytestmark = pytest.mark.gpu

# rows, columns, depth of a product
SHAPES = [(2050, 4104, 1000),   # 152 narrow tiles written directly, one in eight runs
          (4100, 4608, 1000),   # the same of wide tiles
          (2050, 4608, 2048),   # 76 wide tiles, five in halves
          (1030, 8200, 2048),   # 76 wide tiles, nine in halves, some of which hold no column
          (1030, 4104, 128),    # 45 wide tiles, the last of each row with one half
          (2050, 1032, 128)]    # 45 narrow tiles


@pytest.mark.parametrize("M,N,K", SHAPES)
@pytest.mark.parametrize("act", ACTS)
def test_forward(flp, M, N, K, act):  # noqa: F811
    run_forward(flp, M, N, K, act, torch.bfloat16 if act == "silu" else torch.float32, residual=act != "relu", keep=act is not None)


@pytest.mark.parametrize("M,N,K", SHAPES)
def test_forward_at_odd_places(flp, M, N, K):  # noqa: F811
    run_forward(flp, M, N - 1, K, "silu", torch.bfloat16, True, True, (1, 0, 3, 5), (0, 1, 1, 3))


@pytest.mark.parametrize("M,K,N", SHAPES)
@pytest.mark.parametrize("act,dw_dtype", [(None, torch.float32), ("gelu", torch.bfloat16), ("silu", torch.float32)])
def test_gradient_of_the_input(flp, M, K, N, act, dw_dtype):  # noqa: F811
    run_backward(flp, M, N, K, act, dw_dtype)


@pytest.mark.parametrize("M,K,N", SHAPES[:4])
def test_gradient_of_the_input_at_odd_places(flp, M, K, N):  # noqa: F811
    run_backward(flp, M, N + 1, K - 1, "gelu_tanh", torch.bfloat16, (1, 0, 3, 0, 5), (0, 1, 1, 0, 3))


def test_calls_beside_one_another(flp):  # noqa: F811
    """Launches of every layout on several streams give what each gives alone."""
    g = torch.Generator(device="cuda").manual_seed(1)
    jobs = []
    for M, N, K in SHAPES:
        x = torch.randn(M, K, generator=g, device="cuda").bfloat16()
        jobs.append((x, (torch.randn(N, K, generator=g, device="cuda") / K ** 0.5).bfloat16()))
    want = [flp.linear(x, W, activation="gelu") for x, W in jobs]
    streams = [torch.cuda.Stream() for _ in range(4)]
    torch.cuda.synchronize()
    got = [(i % len(jobs), flp.linear(*jobs[i % len(jobs)], activation="gelu", stream=streams[i % 4])) for i in range(24)]
    torch.cuda.synchronize()
    for i, y in got:
        assert torch.equal(y, want[i])
