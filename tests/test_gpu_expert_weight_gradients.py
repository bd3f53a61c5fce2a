"""The gradient of the experts' weights, dw[t, j] = <dy[t], ys[position(t, j)]>, in each of its
kernels, held to the additions that the kernel makes.

A lane takes its elements in pairs, one sum for each half, by fma; then come the halves'
sum, a tree over the lanes that share the row, and in the block kernel one addition a
warp.  The longest chain of roundings is
    a warp a token (2048 tokens or more, or rows of up to two chunks):  H / 64 + 6
    a block a token (fewer tokens):    H / 512 + 8 (chunks of 512 bf16 or 256 fp32) + 6 + 8
    `lanes` of a warp a token (aligned rows of up to 32 vectors):       4 + 6
all below H / 64 + 22, each of at most 2^-24 of the sum of the magnitudes.
"""
import pytest
import torch

from test_gpu_experts import choices, flp, matrix  # noqa: F401 (flp: fixture)

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("T", [5, 300, 2047, 2048, 2100])
@pytest.mark.parametrize("H,pad,offset", [(64, 0, 0), (128, 0, 0), (1024, 0, 0), (5120, 0, 0), (5119, 1, 1), (8192, 0, 0), (333, 0, 0)])
@pytest.mark.parametrize("positive", [False, True])
def test_additions(flp, dtype, T, H, pad, offset, positive):  # noqa: F811
    g = torch.Generator().manual_seed(H + T)
    order = flp.expert_sort(choices(T, 2, 7, seed=T, dropped=0.2).cuda(), 7)
    total = int(order.offsets[-1])
    _, ys = matrix(2 * T, H, dtype, pad, offset, g)
    _, dy = matrix(T, H, dtype, pad, offset, g)
    if positive:
        ys.abs_(), dy.abs_()
    w = torch.rand(T, 2, generator=g).cuda()
    _, dw = flp.expert_combine_backward(dy, ys, order, w)
    rows = order.rows.long()
    for j in range(2):
        live = rows[:, j] < total
        products = dy.double() * ys.double()[rows[:, j]] * live[:, None]
        off = (dw[:, j].double() - products.sum(1)).abs()
        assert bool((off <= (H / 64 + 22) * 2.0 ** -24 * products.abs().sum(1)).all())
        assert bool((dw[~live, j] == 0).all())
