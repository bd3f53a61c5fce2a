"""Alternatives of rows whose first bounds come late: banned beginnings of any length
before ordinary logits, rising logits, few or many left, in one block a row and in
clusters.  Tolerances as in test_gpu_token_logprob.py."""
import math

import pytest
import torch

from test_gpu_token_logprob import check, flp, make  # noqa: F401 (flp: fixture)

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("M,V,k", [(2, 70001, 20), (700, 40001, 5), (2, 151936, 32), (5000, 2500, 8)])
@pytest.mark.parametrize("pad,offset", [(0, 0), (3, 1)])
def test_banned_beginnings(flp, dtype, M, V, k, pad, offset):  # noqa: F811
    x, y = make(M, V, dtype, pad, offset, seed=V)
    n = 24 if M > 24 else M
    for first in (1000, 4096, 8192, 8193, 16384, 20000, 33000, V - 3000, V - 40, V - 3):
        if not 0 < first < V:
            continue
        x[:, :first] = -math.inf
        y.fill_(V - 1)
        got = flp.token_logprob(x, y, top=k)
        part = flp.token_logprob(x[M - n:], y[M - n:], top=k)
        if M < 100:  # the same rows, in the same number of blocks
            for a, b in zip(got, part):
                assert torch.equal(a[M - n:], b)
        assert torch.equal(got[4][M - n:], part[4])
        check(flp, x[M - n:], y[M - n:], k, 1.0)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("V", [9001, 60000])
def test_rising_logits_after_a_banned_beginning(flp, dtype, V):  # noqa: F811
    j = torch.arange(V).float()
    for start in (0, V // 3, V - 2000):
        row = torch.where(j >= start, (j // 7) / 512, -math.inf)
        x = row.repeat(3, 1)
        x[1] = torch.where(j % 5 == 0, x[1], -math.inf)
        x[2, V - 17:] = -math.inf
        x = x.to(dtype).cuda()
        check(flp, x, torch.tensor([V - 1, V - 1 - (V - 1) % 5, V - 18]).cuda(), 20, 1.0)
