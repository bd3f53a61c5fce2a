"""The layer norm backward's workspace: what the query asks for is what the widest
of the forms uses, and enough for each."""
import pytest
import torch

import step_reference as ref
from test_gpu_norm import check_backward, f64, flp  # noqa: F401 (flp: fixture)

pytestmark = pytest.mark.gpu


def query(flp, M, H):  # noqa: F811
    return flp._workspace_bytes("flp_layer_norm_workspace", 0, M, H)


def test_no_more_than_the_blocks_that_fit(flp):  # noqa: F811
    """Blocks of 256 threads or more: two an SM, above 8192 columns one."""
    sms = torch.cuda.get_device_properties(0).multi_processor_count
    for H, per_sm in ((4096, 2), (5120, 2), (8192, 2), (8200, 1), (16384, 1)):
        assert query(flp, 10 ** 6, H) <= per_sm * sms * 2 * H * 4, H
        assert query(flp, 100, H) <= 100 * 2 * H * 4
    assert query(flp, 10 ** 6, 256) <= 8 * sms * 2 * 256 * 4


@pytest.mark.parametrize("M,H", [(5000, 40), (5000, 300), (3000, 512), (700, 520), (700, 1023), (700, 2048), (650, 4096),
                                 (650, 5120), (400, 8192), (330, 8200), (200, 16384)])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_enough_for_every_form(flp, M, H, dtype):  # noqa: F811
    g = torch.Generator().manual_seed(M + H)
    need = query(flp, M, H)
    ws = torch.full((need + 4096,), 0xA5, dtype=torch.uint8, device="cuda")
    for pitch, offset in ((0, 0), (3, 1)):
        x = ref.rows_of(M, H, dtype, "cuda", pitch, offset, g)
        dy = ref.rows_of(M, H, dtype, "cuda", pitch, offset, g)
        y, mean, rstd, kept = flp.layer_norm(x, checkpoint=True)
        for acts in (x, kept):
            dx, dw, db = flp.layer_norm_backward(dy, acts, None, mean, rstd, workspace=ws[:need])
            values = f64(x) if acts is x else f64(flp.checkpoint_unpack(kept, dtype=torch.float32))
            check_backward(dy, values, None, mean, rstd, dx, dw, db)
    assert (ws[need:] == 0xA5).all()
