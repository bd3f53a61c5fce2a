"""Layer norm where every block takes several rows of a shape: loose rows (odd
widths, pitches and offsets), and both sides of each change of block size.
Formulas and tolerances are those of test_gpu_norm.py."""
import pytest
import torch

import step_reference as ref
from test_gpu_norm import check_backward, check_forward, f64, flp  # noqa: F401 (flp: fixture)

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("M,H,pitch,offset", [(700, 1023, 0, 0), (700, 1023, 2, 1), (700, 4101, 4, 3), (700, 5001, 0, 0),
                                              (640, 4104, 0, 0), (640, 5120, 0, 0), (640, 5128, 0, 0), (640, 6144, 8, 0),
                                              (500, 6001, 0, 1), (340, 8192, 0, 0), (340, 8001, 3, 0), (330, 12345, 2, 1)])
def test_rows_of_one_block(flp, M, H, pitch, offset, dtype):  # noqa: F811
    g = torch.Generator().manual_seed(M + H + pitch)
    x = ref.rows_of(M, H, dtype, "cuda", pitch, offset, g, scale=2.0)
    dy = ref.rows_of(M, H, dtype, "cuda", pitch, offset, g)
    w, b = ((1 + 0.2 * torch.randn(H, generator=g)).to(dtype).cuda() for _ in range(2))
    y, mean, rstd, kept = flp.layer_norm(x, w, b, checkpoint=True)
    check_forward(x, w, b, 1e-5, y, mean, rstd)
    assert torch.equal(y, flp.layer_norm(x, w, b)[0])
    back = flp.checkpoint_unpack(flp.checkpoint_pack(x), dtype=torch.float32)
    assert torch.equal(flp.checkpoint_unpack(kept, dtype=torch.float32), back)
    for acts, values in ((x, f64(x)), (kept, f64(back))):
        dx, dw, db = flp.layer_norm_backward(dy, acts, w, mean, rstd)
        check_backward(dy, values, w, mean, rstd, dx, dw, db)
        assert all(torch.equal(u, v) for u, v in zip((dx, dw, db), flp.layer_norm_backward(dy, acts, w, mean, rstd)))
