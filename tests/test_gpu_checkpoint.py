"""8-bit checkpoints on the GPU: bit for bit what the definition gives, and the
weight gradient from one against 64 bits.

The checkpoint has one right answer (dividing by a power of two is exact and
rint rounds once), so bytes and values are compared for equality.

Weight gradient: the products of bf16 values are exact in fp32; adding M of
them 16 at a time rounds at most M / 16 + 32 times (splits and their join
included), each by at most 2^-23 of the sum of magnitudes.  A bf16 dW adds
2^-8 of its value.
"""
import numpy as np
import pytest
import torch

import step_reference as ref

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def flp():
    if not torch.cuda.is_available():
        pytest.skip("needs a CUDA GPU")
    from entropy_loss_gb300 import build, flp as _flp
    build.build()
    _flp.load()
    return _flp


def check(flp, x):
    kept = flp.checkpoint_pack(x)
    q, scale = ref.pack(x.float().cpu().numpy())
    assert kept.shape == tuple(x.shape)
    assert np.array_equal(kept.q.cpu().numpy(), q)
    assert np.array_equal(kept.scale.cpu().numpy(), scale)
    want = ref.unpack(q, scale, x.shape[1])
    for dtype in (torch.float32, torch.bfloat16):
        got = flp.checkpoint_unpack(kept, dtype=dtype)
        assert got.dtype is dtype
        np.testing.assert_array_equal(got.double().cpu().numpy(), want)
    assert flp.checkpoint_unpack(kept).dtype is x.dtype


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("M,H", [(1, 1), (1, 32), (5, 31), (4, 33), (257, 64), (3, 1000), (9, 1023), (64, 520), (1, 20000)])
def test_bytes_and_values(flp, M, H, dtype):
    g = torch.Generator().manual_seed(M * H)
    x = torch.randn(M, H, generator=g) * torch.exp(3 * torch.randn(M, 1, generator=g))
    check(flp, x.to(dtype).cuda())


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_special_blocks(flp, dtype):
    tiny, huge = torch.finfo(dtype).tiny, torch.finfo(dtype).max
    rows = torch.zeros(13, 70)
    rows[1, :32] = -0.0
    rows[2] = torch.arange(70) * tiny / 16              # below the smallest normal number
    rows[3] = huge * torch.linspace(-1, 1, 70)
    rows[4, 3], rows[4, 40] = float("inf"), 1.0
    rows[5, 69] = float("nan")
    rows[6, 31], rows[6, 32] = -float("inf"), 5.0
    rows[7] = torch.tensor([1.9921875, 0.01] * 35)      # 127.5 steps: rounds to 128, kept as 127
    rows[8] = torch.tensor([-1.9921875, 1.0] * 35)
    rows[9] = (torch.arange(70) - 35 + 0.5) / 64        # ties
    rows[9, 0] = rows[9, 32] = rows[9, 64] = 1.0
    rows[10] = 2.0 ** -121 * torch.linspace(-1, 1, 70)  # where the step reaches its floor
    rows[11] = 2.0 ** -120
    rows[12] = 1.9999999
    check(flp, rows.to(dtype).cuda())


@pytest.mark.parametrize("pitch,offset", [(8, 0), (5, 0), (0, 1), (3, 2), (8, 8)])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("H", [64, 100])
def test_pitch_and_alignment(flp, H, pitch, offset, dtype):
    x = ref.rows_of(21, H, dtype, "cuda", pitch, offset, torch.Generator().manual_seed(H))
    check(flp, x)
    kept = flp.checkpoint_pack(x)
    wide = torch.full((21, H + pitch + offset), 7.0, dtype=dtype, device="cuda")
    flp.checkpoint_unpack(kept, out=wide[:, offset:offset + H])
    assert torch.equal(wide[:, offset:offset + H], flp.checkpoint_unpack(kept))
    assert (wide[:, :offset] == 7).all() and (wide[:, offset + H:] == 7).all()


def test_no_rows_and_offsets_past_32_bits(flp):
    kept = flp.checkpoint_pack(torch.empty(0, 40, device="cuda"))
    assert kept.shape == (0, 40) and flp.checkpoint_unpack(kept).shape == (0, 40)
    H = 32768 + 64
    M = (1 << 31) // H + 10
    x = torch.zeros(M, H, dtype=torch.bfloat16, device="cuda")
    x[-9:] = torch.randn(9, H, device="cuda").to(torch.bfloat16)
    kept, tail = flp.checkpoint_pack(x), flp.checkpoint_pack(x[-9:])
    assert torch.equal(kept.q[-9:], tail.q) and torch.equal(kept.scale[-9:], tail.scale)
    assert not kept.q[:-9].any()
    back = flp.checkpoint_unpack(kept, out=x)
    assert torch.equal(back[-9:], flp.checkpoint_unpack(tail))


# ------------------------------------------------------------ weight gradient

def make(flp, M, N, K, seed=0, pitch=0, offset=0):
    g = torch.Generator().manual_seed(seed + M + N + K)
    kept = flp.checkpoint_pack((torch.randn(M, K, generator=g) + 0.1).to(torch.bfloat16).cuda())
    return ref.rows_of(M, N, torch.bfloat16, "cuda", pitch, offset, g), kept


def check_wgrad(flp, dy, kept, dw, before=None):
    M, N = dy.shape
    x = torch.from_numpy(ref.unpack(kept.q.cpu().numpy(), kept.scale.cpu().numpy(), kept.cols)).cuda()
    y = dy.double()
    want = y.t() @ x
    size = y.abs().t() @ x.abs()
    if before is not None:
        want, size = want + before.double(), size + before.double().abs()
    tol = (M / 16 + 32) * 2.0 ** -23 * size + (2.0 ** -8 * want.abs() if dw.dtype is torch.bfloat16 else 0) + 1e-38
    assert bool(((dw.double() - want).abs() <= tol).all())


SHAPES = [(1, 8, 32), (1, 1, 1), (64, 256, 512), (65, 257, 513), (777, 264, 1000), (100, 7, 5), (128, 300, 31),
          (4096, 512, 256), (2048, 1024, 1032), (200, 5120, 2048), (130, 5000, 2040), (3000, 100, 200), (63, 520, 1500)]


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("M,N,K", SHAPES)
def test_weight_gradient(flp, M, N, K, dtype):
    dy, kept = make(flp, M, N, K)
    dw = flp.checkpoint_weight_grad(dy, kept, dw_dtype=dtype)
    assert dw.shape == (N, K) and dw.dtype is dtype
    check_wgrad(flp, dy, kept, dw)
    assert torch.equal(dw, flp.checkpoint_weight_grad(dy, kept, dw_dtype=dtype))


@pytest.mark.parametrize("M,N,K", [(64, 256, 512), (777, 264, 1000), (33, 70, 45), (200, 5120, 2048), (0, 16, 40)])
def test_weight_gradient_accumulates(flp, M, N, K):
    dy, kept = make(flp, M, N, K, seed=5)
    before = torch.randn(N, K, device="cuda")
    dw = before.clone()
    assert flp.checkpoint_weight_grad(dy, kept, dW=dw, accumulate=True) is dw
    check_wgrad(flp, dy, kept, dw, before)
    if M == 0:
        assert torch.equal(dw, before)
        assert not flp.checkpoint_weight_grad(dy, kept).any()


@pytest.mark.parametrize("N,pitch,offset", [(64, 8, 0), (64, 8, 8), (64, 1, 0), (64, 0, 1), (61, 0, 0), (61, 3, 0), (264, 5, 3)])
def test_weight_gradient_pitch_and_alignment(flp, N, pitch, offset):
    dy, kept = make(flp, 150, N, 96, pitch=pitch, offset=offset)
    check_wgrad(flp, dy, kept, flp.checkpoint_weight_grad(dy, kept))


def test_weight_gradient_of_bad_values(flp):
    """A block kept as NaN reaches its own columns, a NaN in dY its own row."""
    x = torch.randn(100, 128, device="cuda")
    x[50, 40] = float("inf")
    dy = torch.randn(100, 48, device="cuda").to(torch.bfloat16)
    dw = flp.checkpoint_weight_grad(dy, flp.checkpoint_pack(x))
    assert torch.isnan(dw[:, 32:64]).all() and torch.isfinite(dw[:, :32]).all() and torch.isfinite(dw[:, 64:]).all()
    dy[3, 5] = float("nan")
    x[50, 40] = 0
    dw = flp.checkpoint_weight_grad(dy, flp.checkpoint_pack(x))
    assert torch.isnan(dw[5]).all() and torch.isfinite(dw[:5]).all() and torch.isfinite(dw[6:]).all()


def test_weight_gradient_against_differences(flp):
    """L = sum(dY (x^ W^T)) is linear in W, so a difference of any width is
    exact: dW_nk = L(W + e_nk) - L(W)."""
    dy, kept = make(flp, 70, 9, 40)
    x = ref.unpack(kept.q.cpu().numpy(), kept.scale.cpu().numpy(), 40)
    D = dy.double().cpu().numpy()
    dw = flp.checkpoint_weight_grad(dy, kept).double().cpu().numpy()
    loss = lambda W: (D * (x @ W.T)).sum()
    for n in range(9):
        for k in (0, 17, 39):
            e = np.zeros((9, 40))
            e[n, k] = 1.0
            assert abs(loss(e) - loss(0 * e) - dw[n, k]) <= 1e-5 * np.abs(D).sum()


def test_weight_gradient_stays_inside_its_buffers(flp):
    M, N, K = 130, 266, 520
    dy, kept = make(flp, M, N, K)
    for dtype in (torch.float32, torch.bfloat16):
        raw = torch.full((N * K * dtype.itemsize + 8192,), 0xA5, dtype=torch.uint8, device="cuda")
        dw = raw[4096:4096 + N * K * dtype.itemsize].view(dtype).view(N, K)
        need = flp._workspace_bytes("flp_checkpoint_weight_grad_workspace", 0, dy.data_ptr(), dy.stride(0), M, N, K,
                                    flp._DTYPE[dtype])
        ws = torch.full((need + 8192,), 0xA5, dtype=torch.uint8, device="cuda")
        flp.checkpoint_weight_grad(dy, kept, dW=dw, workspace=ws[4096:4096 + need])
        check_wgrad(flp, dy, kept, dw)
        for guarded in (raw, ws):
            assert (guarded[:4096] == 0xA5).all() and (guarded[-4096:] == 0xA5).all()
        assert flp.get_error(ws[4096:]) == flp.FLP_OK


def test_own_stream(flp):
    dy, kept = make(flp, 3000, 512, 1024)
    dw = flp.checkpoint_weight_grad(dy, kept)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    dw2 = flp.checkpoint_weight_grad(dy, kept, stream=side)
    back = flp.checkpoint_unpack(kept, stream=side)
    again = flp.checkpoint_pack(back, stream=side)
    torch.cuda.current_stream().wait_stream(side)
    assert torch.equal(dw, dw2)
    assert torch.equal(flp.checkpoint_unpack(again), back)


def test_refusals(flp):
    x = torch.randn(8, 64, device="cuda")
    kept = flp.checkpoint_pack(x)
    dy = torch.randn(8, 16, device="cuda").to(torch.bfloat16)
    with pytest.raises(ValueError):
        flp.checkpoint_pack(x.half())
    with pytest.raises(ValueError):
        flp.checkpoint_pack(x.t())
    with pytest.raises(ValueError):
        flp.checkpoint_unpack(kept._replace(cols=65))
    with pytest.raises(ValueError):
        flp.checkpoint_unpack(kept._replace(q=kept.q.to(torch.int32)))
    with pytest.raises(ValueError):
        flp.checkpoint_unpack(kept, out=torch.empty(8, 63, device="cuda"))
    with pytest.raises(ValueError):
        flp.checkpoint_unpack(kept, dtype=torch.float16)
    with pytest.raises(ValueError):
        flp.checkpoint_weight_grad(dy.float(), kept)
    with pytest.raises(ValueError):
        flp.checkpoint_weight_grad(dy[:7], kept)
    with pytest.raises(ValueError):
        flp.checkpoint_weight_grad(dy, kept, accumulate=True)
    with pytest.raises(ValueError):
        flp.checkpoint_weight_grad(dy, kept, dW=torch.empty(16, 63, device="cuda"))
    with pytest.raises(flp.FlpError) as e:
        flp.checkpoint_weight_grad(dy, kept, dW=torch.zeros(16, 64, dtype=torch.bfloat16, device="cuda"), accumulate=True)
    assert e.value.status == flp.FLP_ERR_UNSUPPORTED
    with pytest.raises(flp.FlpError) as e:
        flp.checkpoint_weight_grad(dy, kept, workspace=torch.empty(1024, dtype=torch.uint8, device="cuda"))
    assert e.value.status == flp.FLP_ERR_WORKSPACE
