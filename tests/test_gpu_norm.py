"""Layer norm forward and backward on the GPU against the formulas in 64 bits.

Tolerances.  u = 2^-24.  A row sum adds at most 64 elements in one thread and
then 10 tree levels, so its error is below 74 u times the sum of magnitudes:
2^-17 covers it with the few operations around it.  Column sums (dw, db) add
at most M / blocks rows in one thread and 32 + 5 + 8 join steps; for the sizes
here that is also below 128 u = 2^-17.  A bf16 output adds half a unit of its
last place, at most 2^-8 of the value.
"""
import numpy as np
import pytest
import torch

import step_reference as ref

pytestmark = pytest.mark.gpu

R = 2.0 ** -17
ROUND = {torch.bfloat16: 2.0 ** -8, torch.float32: 2.0 ** -22}


@pytest.fixture(scope="module")
def flp():
    if not torch.cuda.is_available():
        pytest.skip("needs a CUDA GPU")
    from entropy_loss_gb300 import build, flp as _flp
    build.build()
    _flp.load()
    return _flp


def f64(t):
    return t.double().cpu().numpy()


def check_forward(x, w, b, eps, y, mean, rstd):
    X = f64(x)
    W, B = (None if t is None else f64(t) for t in (w, b))
    ry, rm, rr = ref.norm_forward(X, W, B, eps)
    size = np.abs(X).mean(1)
    assert np.all(np.abs(f64(mean) - rm) <= R * size + 1e-38)
    assert np.all(np.abs(f64(rstd) - rr) <= rr * (R + (R * size * rr) ** 2))
    aw = 1.0 if W is None else np.abs(W)
    ab = 0.0 if B is None else np.abs(B)
    xh = np.abs((X - rm[:, None]) * rr[:, None])
    tol = R * (xh * aw + (rr * size)[:, None] * aw) + 2.0 ** -21 * ab + ROUND[y.dtype] * np.abs(ry) + 1e-38
    assert np.all(np.abs(f64(y) - ry) <= tol)


def check_backward(dy, X, w, mean, rstd, dx, dw, db):
    """X: the activations' values in 64 bits."""
    D, W = f64(dy), None if w is None else f64(w)
    m, r = f64(mean), f64(rstd)
    rdx, rdw, rdb = ref.norm_backward(D, X, W, m, r)
    g = np.abs(D if W is None else D * W)
    xh = np.abs((X - m[:, None]) * r[:, None])
    tol = R * r[:, None] * (g + g.mean(1, keepdims=True) + xh * (g * xh).mean(1, keepdims=True))
    assert np.all(np.abs(f64(dx) - rdx) <= tol + ROUND[dx.dtype] * np.abs(rdx) + 1e-38)
    assert np.all(np.abs(f64(dw) - rdw) <= R * (np.abs(D) * xh).sum(0) + 1e-38)
    assert np.all(np.abs(f64(db) - rdb) <= R * np.abs(D).sum(0) + 1e-38)


SIZES = [(1, 1), (1, 8), (3, 31), (5, 33), (7, 255), (2, 256), (129, 257), (64, 512), (31, 768), (300, 1000), (33, 1023),
         (400, 1024), (700, 256), (600, 511), (1500, 33), (512, 512), (64, 2048), (65, 2048), (9, 2048), (17, 4096), (700, 4104), (11, 5120), (4, 8192), (5, 12001), (3, 16384)]


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("M,H", SIZES)
def test_forward_and_backward(flp, M, H, dtype):
    g = torch.Generator().manual_seed(M * 7 + H)
    x = (2 * torch.randn(M, H, generator=g) + 0.5).to(dtype).cuda()
    w = (1 + 0.2 * torch.randn(H, generator=g)).to(dtype).cuda()
    b = (0.3 * torch.randn(H, generator=g)).to(dtype).cuda()
    dy = torch.randn(M, H, generator=g).to(dtype).cuda()
    y, mean, rstd = flp.layer_norm(x, w, b, eps=1e-5)
    check_forward(x, w, b, 1e-5, y, mean, rstd)
    dx, dw, db = flp.layer_norm_backward(dy, x, w, mean, rstd)
    check_backward(dy, f64(x), w, mean, rstd, dx, dw, db)
    again = flp.layer_norm_backward(dy, x, w, mean, rstd)
    assert all(torch.equal(a, c) for a, c in zip((dx, dw, db), again))


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("M,H", [(1, 1), (3, 31), (130, 64), (77, 257), (33, 1024), (21, 1023), (260, 4096), (3, 16384), (2, 16383)])
def test_checkpoint_of_the_input(flp, M, H, dtype):
    g = torch.Generator().manual_seed(M + H)
    x = (3 * torch.randn(M, H, generator=g) - 1).to(dtype).cuda()
    w = torch.randn(H, generator=g).to(dtype).cuda()
    dy = torch.randn(M, H, generator=g).to(dtype).cuda()
    y0, mean0, rstd0 = flp.layer_norm(x, w, None)
    y, mean, rstd, kept = flp.layer_norm(x, w, None, checkpoint=True)
    assert torch.equal(y, y0) and torch.equal(mean, mean0) and torch.equal(rstd, rstd0)
    q, scale = ref.pack(x.float().cpu().numpy())
    assert np.array_equal(kept.q.cpu().numpy(), q) and np.array_equal(kept.scale.cpu().numpy(), scale)
    dx, dw, db = flp.layer_norm_backward(dy, kept, w, mean, rstd)
    check_backward(dy, ref.unpack(q, scale, H), w, mean, rstd, dx, dw, db)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("M,H", [(500, 8200), (330, 10001), (460, 12288), (200, 16384), (170, 16383)])
def test_several_wide_rows_a_block(flp, M, H, dtype):
    """Rows whose sums over rows do not all stay in registers, more than the blocks."""
    test_forward_and_backward(flp, M, H, dtype)
    test_checkpoint_of_the_input(flp, M, H, dtype)


@pytest.mark.parametrize("pitch,offset", [(0, 0), (8, 0), (8, 8), (5, 0), (0, 1), (3, 2)])
@pytest.mark.parametrize("H", [64, 1000, 1001])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_pitch_and_alignment(flp, H, pitch, offset, dtype):
    g = torch.Generator().manual_seed(H + pitch)
    M = 37
    x = ref.rows_of(M, H, dtype, "cuda", pitch, offset, g)
    dy = ref.rows_of(M, H, dtype, "cuda", pitch, 0, g)
    out = ref.rows_of(M, H, dtype, "cuda", 0, offset, g)
    dx = ref.rows_of(M, H, dtype, "cuda", pitch, offset, g)
    w, b = ((torch.randn(H + 1, generator=g).to(dtype).cuda())[1 - (offset == 0):][:H] for _ in range(2))
    y, mean, rstd = flp.layer_norm(x, w, b, out=out)
    assert y is out
    check_forward(x, w, b, 1e-5, y, mean, rstd)
    _, dw, db = flp.layer_norm_backward(dy, x, w, mean, rstd, dx=dx)
    check_backward(dy, f64(x), w, mean, rstd, dx, dw, db)


@pytest.mark.parametrize("H", [256, 999, 4096])
def test_parameters_left_out_or_in_fp32(flp, H):
    g = torch.Generator().manual_seed(H)
    x = torch.randn(50, H, generator=g).to(torch.bfloat16).cuda()
    dy = torch.randn(50, H, generator=g).to(torch.bfloat16).cuda()
    w, b = torch.randn(H, generator=g).cuda(), torch.randn(H, generator=g).cuda()
    for weight, bias in ((None, None), (w, None), (None, b), (w, b)):
        y, mean, rstd = flp.layer_norm(x, weight, bias)
        check_forward(x, weight, bias, 1e-5, y, mean, rstd)
        dx, dw, db = flp.layer_norm_backward(dy, x, weight, mean, rstd)
        check_backward(dy, f64(x), weight, mean, rstd, dx, dw, db)


def test_rows_of_one_value_large_means_and_bad_values(flp):
    H = 1024
    x = torch.randn(6, H, device="cuda")
    x[0] = 3.0            # no variance: y is the bias
    x[1] = 0.0
    x[2] += 1.0e4         # a mean far above the spread
    x[3, 5] = float("inf")
    x[4, 7] = float("nan")
    w, b = torch.rand(H, device="cuda") + 0.5, torch.randn(H, device="cuda")
    y, mean, rstd = flp.layer_norm(x, w, b)
    assert torch.equal(y[0], b) and torch.equal(y[1], b)
    fine = [0, 1, 2, 5]
    check_forward(x[fine], w, b, 1e-5, y[fine], mean[fine], rstd[fine])
    assert torch.isnan(y[3]).any() and torch.isnan(y[4]).all()
    # a bad row reaches no other row's dx
    dy = torch.randn_like(x)
    dx, dw, db = flp.layer_norm_backward(dy, x, w, mean, rstd)
    assert torch.isfinite(dx[fine]).all() and torch.isnan(dx[4]).all()
    assert torch.isfinite(db).all()


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_widths_of_one_kernel_in_any_order(flp, dtype):
    """Widths that share a kernel but not a block size, the widest before and after the others."""
    for H in (8192, 5192, 6000, 8192, 4096, 2056, 4096, 16384, 8200, 16384, 5001, 8191):
        x = torch.randn(3, H, device="cuda").to(dtype)
        y, mean, rstd, kept = flp.layer_norm(x, checkpoint=True)
        check_forward(x, None, None, 1e-5, y, mean, rstd)
        dx, dw, db = flp.layer_norm_backward(y, x, None, mean, rstd)
        check_backward(y, f64(x), None, mean, rstd, dx, dw, db)


def test_no_rows(flp):
    x = torch.empty(0, 512, dtype=torch.bfloat16, device="cuda")
    y, mean, rstd, kept = flp.layer_norm(x, checkpoint=True)
    assert y.shape == (0, 512) and mean.numel() == 0 and kept.shape == (0, 512)
    dx, dw, db = flp.layer_norm_backward(x, x, None, mean, rstd)
    assert dx.shape == (0, 512) and not dw.any() and not db.any()


def test_in_place(flp):
    x = torch.randn(99, 2048, device="cuda").to(torch.bfloat16)
    dy = torch.randn(99, 2048, device="cuda").to(torch.bfloat16)
    y, mean, rstd = flp.layer_norm(x)
    dx, dw, db = flp.layer_norm_backward(dy, x, None, mean, rstd)
    keep = x.clone()
    y2, _, _ = flp.layer_norm(keep, out=keep)
    assert y2 is keep and torch.equal(y, keep)
    dx2, dw2, db2 = flp.layer_norm_backward(dy, x, None, mean, rstd, dx=dy)
    assert dx2 is dy and torch.equal(dx, dy) and torch.equal(dw, dw2) and torch.equal(db, db2)


def test_gradient_against_differences(flp):
    """Central differences of L = sum(dy y) in 64 bits.  The difference itself
    is off by O(h^2) = 1e-8 of the third derivative; 1e-5 covers that and the
    fp32 kernel."""
    g = torch.Generator().manual_seed(3)
    M, H, h = 4, 40, 1e-4
    x, dy = torch.randn(M, H, generator=g).cuda(), torch.randn(M, H, generator=g).cuda()
    w, b = (torch.randn(H, generator=g).cuda() for _ in range(2))
    _, mean, rstd = flp.layer_norm(x, w, b)
    dx, dw, db = (f64(t) for t in flp.layer_norm_backward(dy, x, w, mean, rstd))
    X, D, W, B = f64(x), f64(dy), f64(w), f64(b)
    loss = lambda X, W, B: float((D * ref.norm_forward(X, W, B, 1e-5)[0]).sum())
    for i in range(M):
        for j in range(0, H, 7):
            e = np.zeros_like(X)
            e[i, j] = h
            assert abs((loss(X + e, W, B) - loss(X - e, W, B)) / (2 * h) - dx[i, j]) <= 1e-5 * max(1, np.abs(dx).max())
    for j in range(0, H, 5):
        e = np.zeros(H)
        e[j] = h
        assert abs((loss(X, W + e, B) - loss(X, W - e, B)) / (2 * h) - dw[j]) <= 1e-5 * max(1, np.abs(dw).max())
        assert abs((loss(X, W, B + e) - loss(X, W, B - e)) / (2 * h) - db[j]) <= 1e-5 * max(1, np.abs(db).max())


def test_offsets_past_32_bits(flp):
    """More than 2^31 elements: the last rows come out as they do alone."""
    H = 16384
    M = (1 << 31) // H + 40
    x = torch.empty(M, H, dtype=torch.bfloat16, device="cuda")
    x[:-40].fill_(1.0)
    x[-40:] = torch.randn(40, H, device="cuda").to(torch.bfloat16)
    y, mean, rstd, kept = flp.layer_norm(x, checkpoint=True)
    tail = x[-40:].contiguous()
    y1, mean1, rstd1, kept1 = flp.layer_norm(tail, checkpoint=True)
    assert torch.equal(y[-40:], y1) and torch.equal(mean[-40:], mean1) and torch.equal(kept.q[-40:], kept1.q)
    dx, dw, db = flp.layer_norm_backward(y, kept, None, mean, rstd, dx=y)
    dx1, _, _ = flp.layer_norm_backward(y1, kept1, None, mean1, rstd1)
    assert torch.equal(dx[-40:], dx1)


def test_own_stream(flp):
    x = torch.randn(5000, 1024, device="cuda").to(torch.bfloat16)
    y, mean, rstd = flp.layer_norm(x)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    y2, mean2, rstd2 = flp.layer_norm(x, stream=side)
    dx2, dw2, db2 = flp.layer_norm_backward(y2, x, None, mean2, rstd2, stream=side)
    torch.cuda.current_stream().wait_stream(side)
    dx, dw, db = flp.layer_norm_backward(y, x, None, mean, rstd)
    assert torch.equal(y, y2) and torch.equal(dx, dx2) and torch.equal(dw, dw2) and torch.equal(db, db2)


def test_graph_replay(flp):
    x = torch.randn(300, 4096, device="cuda").to(torch.bfloat16)
    ws = torch.empty(flp._workspace_bytes("flp_layer_norm_workspace", 0, 300, 4096), dtype=torch.uint8, device="cuda")
    step = lambda: (lambda r: (r, flp.layer_norm_backward(r[0], r[3], None, r[1], r[2], workspace=ws)))(
        flp.layer_norm(x, checkpoint=True))
    step()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        (y, _, _, _), (dx, dw, _) = step()
    x.copy_(torch.randn(300, 4096, device="cuda").to(torch.bfloat16))
    graph.replay()
    (y1, _, _, _), (dx1, dw1, _) = step()
    assert torch.equal(y, y1) and torch.equal(dx, dx1) and torch.equal(dw, dw1)


def test_refusals(flp):
    x = torch.randn(4, 64, device="cuda")
    w = torch.ones(64, device="cuda")
    y, mean, rstd, kept = flp.layer_norm(x, w, checkpoint=True)
    with pytest.raises(ValueError):
        flp.layer_norm(x.half())
    with pytest.raises(ValueError):
        flp.layer_norm(x.cpu())
    with pytest.raises(ValueError):
        flp.layer_norm(x.t())
    with pytest.raises(ValueError):
        flp.layer_norm(x[:1].expand(4, 64))
    with pytest.raises(ValueError):
        flp.layer_norm(x, w[:63])
    with pytest.raises(ValueError):
        flp.layer_norm(x, w, w.to(torch.bfloat16))
    with pytest.raises(ValueError):
        flp.layer_norm(x, w, out=x.to(torch.bfloat16))
    with pytest.raises(flp.FlpError):
        flp.layer_norm(x, w, eps=-1.0)
    with pytest.raises(flp.FlpError):
        flp.layer_norm(x, w, eps=float("nan"))
    with pytest.raises(flp.FlpError) as e:
        flp.layer_norm(torch.zeros(1, 16385, device="cuda"))
    assert e.value.status == flp.FLP_ERR_UNSUPPORTED
    with pytest.raises(ValueError):
        flp.layer_norm_backward(y, x[:, :63], w, mean, rstd)
    with pytest.raises(ValueError):
        flp.layer_norm_backward(y, x.to(torch.bfloat16), w, mean, rstd)
    with pytest.raises(ValueError):
        flp.layer_norm_backward(y, kept._replace(cols=96), w, mean, rstd)
    with pytest.raises(ValueError):
        flp.layer_norm_backward(y, x, w, mean[:3], rstd)
    x = torch.randn(1000, 64, device="cuda")
    y, mean, rstd = flp.layer_norm(x, w)
    with pytest.raises(flp.FlpError) as e:
        flp.layer_norm_backward(y, x, w, mean, rstd, workspace=torch.empty(16, dtype=torch.uint8, device="cuda"))
    assert e.value.status == flp.FLP_ERR_WORKSPACE
