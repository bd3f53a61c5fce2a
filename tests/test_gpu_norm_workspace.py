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


@pytest.mark.parametrize("M,H", [(3, 64), (60, 520), (700, 300), (700, 1023), (700, 4096), (330, 16384)])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_sums_that_are_not_wanted(flp, M, H, dtype):  # noqa: F811
    """dx is the same without them, they are the same alone, and without any no
    workspace is needed: neither by the binding nor by the C entry."""
    g = torch.Generator().manual_seed(M + H)
    x, dy = (torch.randn(M, H, generator=g).to(dtype).cuda() for _ in range(2))
    w = torch.rand(H, generator=g).to(dtype).cuda()
    y, mean, rstd, kept = flp.layer_norm(x, w, checkpoint=True)
    for acts in (x, kept):
        dx, dw, db = flp.layer_norm_backward(dy, acts, w, mean, rstd)
        a, none, db1 = flp.layer_norm_backward(dy, acts, w, mean, rstd, want_dweight=False)
        b, dw1, none2 = flp.layer_norm_backward(dy, acts, w, mean, rstd, want_dbias=False)
        tiny = torch.empty(0, dtype=torch.uint8, device="cuda")
        c, none3, none4 = flp.layer_norm_backward(dy, acts, w, mean, rstd, want_dweight=False, want_dbias=False,
                                                  workspace=tiny)
        assert none is none2 is none3 is none4 is None
        assert torch.equal(db, db1) and torch.equal(dw, dw1)
        assert torch.equal(dx, a) and torch.equal(dx, b) and torch.equal(dx, c)


def test_a_frozen_norm_takes_no_sums(flp, monkeypatch):  # noqa: F811
    x = torch.randn(2000, 256, device="cuda", requires_grad=True)
    w, b = torch.rand(256, device="cuda"), torch.rand(256, device="cuda", requires_grad=True)
    seen = []
    real = flp.layer_norm_backward
    monkeypatch.setattr(flp, "layer_norm_backward", lambda *a, **k: seen.append(k) or real(*a, **k))
    flp.fused_layer_norm(x, w, b.detach()).sum().backward()
    flp.fused_layer_norm(x, w, b).sum().backward()
    assert seen[0] == dict(want_dweight=False, want_dbias=False) and seen[1] == dict(want_dweight=False, want_dbias=True)
    assert float((b.grad - 2000).abs().max()) == 0


def test_few_rows_take_one_launch(flp):  # noqa: F811
    """They need no workspace; more rows, whose cluster would take longer, do."""
    for M, H in ((1, 1), (256, 256), (256, 512), (16, 520), (16, 1024), (16, 8192)):
        assert query(flp, M, H) == 0, (M, H)
    for M, H in ((257, 256), (257, 512), (17, 520), (64, 1024), (64, 4096), (17, 8192), (1, 8200)):
        assert query(flp, M, H) > 0, (M, H)


@pytest.mark.parametrize("M,H", [(255, 512), (256, 33), (257, 512), (15, 1023), (16, 5120), (17, 5120), (9, 8192), (18, 8192)])
def test_both_sides_of_the_rule(flp, M, H):  # noqa: F811
    g = torch.Generator().manual_seed(M + H)
    for dtype in (torch.bfloat16, torch.float32):
        x, dy = (torch.randn(M, H, generator=g).to(dtype).cuda() for _ in range(2))
        w = torch.rand(H, generator=g).to(dtype).cuda()
        y, mean, rstd, kept = flp.layer_norm(x, w, checkpoint=True)
        dx, dw, db = flp.layer_norm_backward(dy, x, w, mean, rstd)
        check_backward(dy, f64(x), w, mean, rstd, dx, dw, db)
        dx, dw, db = flp.layer_norm_backward(dy, kept, w, mean, rstd)
        check_backward(dy, f64(flp.checkpoint_unpack(kept, dtype=torch.float32)), w, mean, rstd, dx, dw, db)
