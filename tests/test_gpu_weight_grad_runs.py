"""The weight gradient over more than 2048 rows: tiles that are summed in several
runs, whole tiles beside split ones, and split tiles of several runs, each into
new memory and added to a dW.

Tolerances.  Element by element as in test_gpu_checkpoint.py.  In the 2-norm the
kernel's comment states an error of 4.8e-7 of the result for runs of 2048 rows of
centred normal values and 3.0e-6 for one run over 8192; 1e-6 lies between, so a
sum that is not cut into runs fails the cases of 8200 rows.
"""
import pytest
import torch

import step_reference as ref
from test_gpu_checkpoint import check_wgrad, flp, make  # noqa: F401 (flp: fixture)

pytestmark = pytest.mark.gpu

# On 76 pairs (152 SMs): 64-row blocks, tiles written directly / split, splits, runs.
SHAPES = [(8200, 5120, 2048),   # 129, 76 / 4, 10; 5 runs of a whole tile, 1 of a split one
          (8200, 4096, 2348),   # the same with a last half of 44 columns
          (8200, 4096, 2088),   # and with a last tile of one half, 40 columns
          (2113, 5376, 2048),   # 34, 76 / 8, 4: a last block of one row, two runs
          (6200, 5001, 2040),   # 97, 76 / 4, 9: rows of dW, dY and columns that end inside a tile
          (8200, 5120, 2047),   # 129, 0 / 80, 3: no TMA store, split tiles of two runs
          (32768, 1024, 1024)]  # 512, 0 / 8, 9: split tiles of two runs


def error(got, dy, kept, before=None):
    x = torch.from_numpy(ref.unpack(kept.q.cpu().numpy(), kept.scale.cpu().numpy(), kept.cols)).cuda()
    want = dy.double().t() @ x
    if before is not None:
        want += before.double()
    return float((got.double() - want).norm() / want.norm())


@pytest.mark.parametrize("M,N,K", SHAPES)
def test_runs(flp, M, N, K):  # noqa: F811
    dy, kept = make(flp, M, N, K)
    kept = flp.checkpoint_pack((flp.checkpoint_unpack(kept).float() - 0.1).to(torch.bfloat16))  # centred
    dw = flp.checkpoint_weight_grad(dy, kept)
    check_wgrad(flp, dy, kept, dw)
    assert error(dw, dy, kept) <= 1e-6
    assert torch.equal(dw, flp.checkpoint_weight_grad(dy, kept))
    before = 30 * torch.randn(N, K, device="cuda")
    added = before.clone()
    flp.checkpoint_weight_grad(dy, kept, dW=added, accumulate=True)
    check_wgrad(flp, dy, kept, added, before)
    assert error(added, dy, kept, before) <= 1e-6


@pytest.mark.parametrize("M,N,K", [(8200, 5120, 2047), (8200, 4096, 2088)])
def test_bf16_of_many_rows(flp, M, N, K):  # noqa: F811
    dy, kept = make(flp, M, N, K)
    check_wgrad(flp, dy, kept, flp.checkpoint_weight_grad(dy, kept, dw_dtype=torch.bfloat16))


def test_runs_stay_inside_their_buffers(flp):  # noqa: F811
    M, N, K = 4200, 4090, 2348
    dy, kept = make(flp, M, N, K)
    raw = torch.full((N * K * 4 + 8192,), 0xA5, dtype=torch.uint8, device="cuda")
    dw = raw[4096:-4096].view(torch.float32).view(N, K)
    need = flp._workspace_bytes("flp_checkpoint_weight_grad_workspace", 0, dy.data_ptr() % 16, dy.stride(0), M, N, K, 0)
    ws = torch.full((need + 8192,), 0xA5, dtype=torch.uint8, device="cuda")
    flp.checkpoint_weight_grad(dy, kept, dW=dw, workspace=ws[4096:4096 + need])
    check_wgrad(flp, dy, kept, dw)
    for guarded in (raw, ws):
        assert (guarded[:4096] == 0xA5).all() and (guarded[-4096:] == 0xA5).all()
    assert flp.get_error(ws[4096:]) == flp.FLP_OK


def test_bf16_of_very_many_rows_has_no_bias(flp):  # noqa: F811
    """A sum that is truncated at every step comes out too small: over 2^20 rows in
    one run by 1e-3 of itself.  Rounding to bf16 has no direction: 2^-9 of each
    value at most, 64 x 2048 of them, below 1e-4 on average."""
    M, N, K = (1 << 20) - 37, 5120, 2048
    dy = torch.empty(M, N, dtype=torch.bfloat16, device="cuda").normal_()
    kept = flp.checkpoint_pack(torch.empty(M, K, dtype=torch.bfloat16, device="cuda").normal_())
    dw = flp.checkpoint_weight_grad(dy, kept, dw_dtype=torch.bfloat16)
    x = flp.checkpoint_unpack(kept)
    want = sum(dy[i:i + 65536, :64].double().t() @ x[i:i + 65536].double() for i in range(0, M, 65536))
    off = dw[:64].double() - want
    assert abs(float((off * want.sign()).mean() / want.abs().mean())) <= 1e-4
    assert float((off.abs() - 2.0 ** -8 * want.abs()).max()) <= 1e-6 * float(want.abs().max())
