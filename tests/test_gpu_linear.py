"""The linear layer with bias, activation and residual, and its gradients.

Tolerances.  A sum of K products of bf16 numbers is exact up to the accumulator's
rounding, toward zero: at most 2^-23 of the partial sums a step of 16 products, so
below (K / 16 + 2) 2^-23 of the sum of the magnitudes (each split adds one rounding).
The activations are Lipschitz with constant below 1.13 (gelu's and silu's slopes lie
between -0.13 and 1.13), their own arithmetic is off by below 2^-18 of their argument's
size (fp32 polynomials, a 2^-22 exponential and quotient; the exponent of gelu_tanh,
up to 90 where its result still counts, is rounded by 2^-24 of it), and y is rounded
to bf16 once: half a step, 2^-8 of the value.  In the backward pass d is rounded to
bf16 (2^-8 of each of its values; for an fp32 dW with an activation it is the sum of two
bf16 numbers, off by 2^-8 of 2^-8 of it) and dx, dW (bf16) once more; dbias sums unrounded d:
2^-24 (rows / 8 + 64) of the sum of the magnitudes at most, the slopes being off by
below 2^-17.
"""
import pytest
import torch

pytestmark = pytest.mark.gpu
ACTS = [None, "relu", "gelu", "gelu_tanh", "silu"]


@pytest.fixture(scope="module")
def flp():
    if not torch.cuda.is_available():
        pytest.skip("needs a CUDA GPU")
    from entropy_loss_gb300 import build, flp as _flp
    build.build()
    _flp.load()
    return _flp


def act64(v, kind):
    """(activation, slope) in 64 bits, from the definitions."""
    if kind is None:
        return v, torch.ones_like(v)
    if kind == "relu":
        return v.clamp(min=0), (v > 0).double()
    if kind == "gelu":
        phi = 0.5 * torch.special.erfc(-v / 2 ** 0.5)
        return v * phi, phi + v * torch.exp(-v * v / 2) / (2 * torch.pi) ** 0.5
    u, du = v, torch.ones_like(v)
    if kind == "gelu_tanh":
        c = (8 / torch.pi) ** 0.5
        u, du = c * (v + 0.044715 * v ** 3), c * (1 + 3 * 0.044715 * v * v)
    p = torch.sigmoid(u)
    return v * p, p + v * p * torch.sigmoid(-u) * du


def matrix(M, N, pad=0, offset=0, gen=None, scale=1.0):
    buf = torch.full((M * (N + pad) + offset + 8,), 7.0, dtype=torch.bfloat16)
    view = buf[offset:offset + M * (N + pad)].view(M, N + pad)[:, :N]
    view.copy_(scale * torch.randn(M, N, generator=gen))
    dev = buf.cuda()
    return dev, dev[offset:offset + M * (N + pad)].view(M, N + pad)[:, :N]


def untouched(buf, view, before):
    ours = torch.zeros_like(buf, dtype=torch.bool)
    torch.as_strided(ours, view.shape, view.stride(), view.storage_offset()).fill_(True)
    assert torch.equal(buf[~ours], before[~ours])


def run_forward(flp, M, N, K, act, bias, residual, keep, pads=(0, 0, 0, 0), offsets=(0, 0, 0, 0)):
    g = torch.Generator().manual_seed(M + N + K)
    _, x = matrix(M, K, pads[0], offsets[0], g)
    _, W = matrix(N, K, pads[1], offsets[1], g, K ** -0.5)
    b = None if bias is None else torch.randn(N + 1, generator=g).cuda().to(bias)[offsets[2] % 2:][:N]
    r = matrix(M, N, pads[2], offsets[2], g)[1] if residual else None
    buf, out = matrix(M, N, pads[3], offsets[3], g)
    before = buf.clone()
    got = flp.linear(x, W, b, activation=act, residual=r, keep=keep, out=out)
    y, pre = got if keep else (got, None)
    assert y is out
    v = x.double() @ W.double().t()
    size = x.double().abs() @ W.double().abs().t()
    if b is not None:
        v, size = v + b.double(), size + b.double().abs()
    off = (K / 16 + 2) * 2.0 ** -23 * size + 2.0 ** -24 * v.abs()
    want = act64(v, act)[0]
    if r is not None:
        want = want + r.double()
    tol = 1.13 * off + 2.0 ** -18 * v.abs() + 2.0 ** -24 * want.abs()
    assert bool(((y.double() - want).abs() <= tol + 2.0 ** -8 * (want.abs() + tol)).all())
    untouched(buf, out, before)
    if keep:
        assert bool(((pre.double() - v).abs() <= off + 2.0 ** -8 * (v.abs() + off)).all())
    # a fresh output and the same numbers from a second call
    again = flp.linear(x, W, b, activation=act, residual=r)
    assert torch.equal(again, y)
    return x, W


SHAPES = [(1, 1, 1), (1, 8, 8), (1, 4096, 4096), (2, 513, 40), (3, 7, 1000), (8, 1000, 64), (9, 520, 65), (33, 256, 128), (128, 512, 264),
          (129, 264, 72), (255, 1023, 63), (256, 512, 64), (257, 513, 129), (300, 2047, 1000), (777, 2047, 100), (1000, 1536, 512), (16, 300, 4096), (17, 4096, 200), (48, 640, 1024), (144, 1000, 328), (600, 1100, 520)]


@pytest.mark.parametrize("M,N,K", SHAPES)
@pytest.mark.parametrize("act", ACTS)
def test_forward(flp, M, N, K, act):
    run_forward(flp, M, N, K, act, torch.bfloat16 if M % 2 else torch.float32, residual=bool(N % 2), keep=act is not None)


@pytest.mark.parametrize("bias", [None, torch.bfloat16, torch.float32])
@pytest.mark.parametrize("residual", [False, True])
@pytest.mark.parametrize("keep", [False, True])
@pytest.mark.parametrize("pads,offsets", [((0, 0, 0, 0), (0, 0, 0, 0)), ((8, 16, 8, 24), (0, 8, 0, 0)), ((1, 0, 0, 0), (0, 1, 0, 0)),
                                          ((0, 0, 3, 0), (0, 0, 1, 0)), ((0, 0, 0, 2), (0, 0, 0, 3)), ((5, 3, 1, 7), (1, 3, 5, 1))])
def test_layouts(flp, bias, residual, keep, pads, offsets):
    run_forward(flp, 200, 296, 136, "silu", bias, residual, keep, pads, offsets)


@pytest.mark.parametrize("M", [1, 2, 80, 128, 129])
@pytest.mark.parametrize("K", [64, 203, 1001])
def test_few_rows_at_odd_places(flp, M, K):
    run_forward(flp, M, 300, K, "gelu_tanh", torch.bfloat16, True, True, (1, 3, 5, 2), (3, 1, 2, 1))
    run_forward(flp, M, 2051, K, "silu", torch.float32, False, False)


def test_few_rows_on_many_streams(flp):
    """Clusters that hold tensor memory beside one another: each launch fits wherever it lands."""
    g = torch.Generator().manual_seed(1)
    x = [matrix(M, 128, gen=g)[1] for M in (16, 80, 128)]
    _, W = matrix(9000, 128, gen=g, scale=0.1)
    want = [flp.linear(v, W) for v in x]
    streams = [torch.cuda.Stream() for _ in range(6)]
    torch.cuda.synchronize()
    got = [(i % 3, flp.linear(x[i % 3], W, stream=streams[i % 6])) for i in range(48)]
    torch.cuda.synchronize()
    for i, y in got:
        assert torch.equal(y, want[i])


@pytest.mark.parametrize("N", [19456, 19457])
def test_more_tiles_than_pairs(flp, N):
    """Whole tiles written directly beside split ones: 3 x 38 tiles on 76 pairs."""
    run_forward(flp, 700, N, 192, "gelu", torch.float32, True, True)


def test_long_sums(flp):
    run_forward(flp, 70, 130, 50000, None, None, False, False)


def test_residual_in_place_and_many_at_once(flp):
    g = torch.Generator().manual_seed(1)
    _, x = matrix(300, 128, gen=g)
    _, W = matrix(304, 128, gen=g, scale=0.1)
    _, r = matrix(300, 304, gen=g)
    want = flp.linear(x, W, residual=r)
    assert torch.equal(flp.linear(x, W, residual=r, out=r), want)
    streams = [torch.cuda.Stream() for _ in range(3)]
    torch.cuda.synchronize()
    outs = [flp.linear(x, W, activation="silu", stream=s) for s in streams]
    torch.cuda.synchronize()
    for o in outs:
        assert torch.equal(o, flp.linear(x, W, activation="silu"))


def test_values_far_out(flp):
    """Arguments where exponentials overflow or vanish, and infinities and NaN in one row alone."""
    v = torch.tensor([0.0, -0.0, 1e-30, 30.0, -30.0, 200.0, -200.0, 1e10, -1e10, 1e30, -1e30, -3.0, -5.0, -8.0, -12.0, 7.0])
    x = torch.zeros(3, 8, dtype=torch.bfloat16, device="cuda")
    x[0, 0] = 1
    x[1, 0] = float("inf")
    x[2, 1] = float("nan")
    W = torch.zeros(16, 8, dtype=torch.bfloat16, device="cuda")
    W[:, 0] = v.to(torch.bfloat16)
    W[:, 1] = 1
    val = W[:, 0].double()
    for act in ACTS:
        y, pre = flp.linear(x, W, activation=act, keep=True)
        want, slope = act64(val, act)
        if act == "gelu_tanh":
            want = torch.where(val.abs() > 20, val.clamp(min=0), want)  # v^3 overflows nothing here
        tol = 2.0 ** -18 * val.abs().clamp(max=40) + 2.0 ** -8 * want.abs() + 1e-38
        assert bool(((y[0].double() - want).abs() <= tol + 2.0 ** -18 * want.abs()).all()), act
        assert bool(torch.isnan(y[2].float()).all()) and bool(torch.isfinite(y[0].float()).all())
        assert torch.equal(pre[0], W[:, 0])
        dy = torch.ones(3, 16, dtype=torch.bfloat16, device="cuda")
        _, _, db = flp.linear_backward(dy[:1], x[:1], W, pre[:1], activation=act, want_dx=False, want_dW=False)
        slope = torch.where(val.abs() > 20, (val > 0).double(), slope) if act else slope
        assert bool(((db.double() - slope).abs() <= 2.0 ** -17).all()), act


def test_empty(flp):
    x = torch.zeros(0, 24, dtype=torch.bfloat16, device="cuda")
    W = torch.ones(40, 24, dtype=torch.bfloat16, device="cuda")
    y, pre = flp.linear(x, W, activation="relu", keep=True)
    assert y.shape == (0, 40) and pre.shape == (0, 40)
    dx, dW, db = flp.linear_backward(y, x, W, pre, activation="relu")
    assert dx.shape == (0, 24) and bool((dW == 0).all()) and bool((db == 0).all())


def run_backward(flp, M, N, K, act, dw_dtype=torch.float32, pads=(0, 0, 0, 0, 0), offsets=(0, 0, 0, 0, 0)):
    g = torch.Generator().manual_seed(M * 3 + N + K)
    _, x = matrix(M, K, pads[0], offsets[0], g)
    _, W = matrix(N, K, pads[1], offsets[1], g, K ** -0.5)
    _, dy = matrix(M, N, pads[2], offsets[2], g)
    pre = matrix(M, N, pads[3], offsets[3], g, 1.5)[1] if act else None
    buf, out = matrix(M, K, pads[4], offsets[4], g)
    before = buf.clone()
    dx, dW, db = flp.linear_backward(dy, x, W, pre, activation=act, dw_dtype=dw_dtype, dx=out)
    assert dx is out and dW.dtype is dw_dtype and db.dtype is torch.float32
    untouched(buf, out, before)
    d = dy.double()
    e = torch.zeros_like(d)
    if act:
        d = d * act64(pre.double(), act)[1]
        e = 2.0 ** -17 * dy.double().abs()
    fine = dw_dtype is torch.float32
    # d as the products see it, and the additions: of one product, or of the two of a sum of two
    off = [e + rounded * (d.abs() + e) if act else e for rounded in (2.0 ** -8, 2.0 ** -16 if fine else 2.0 ** -8)]
    for got, a, b, each, rows, last in ((dx, d, W.double(), off[0], N, 2.0 ** -8),
                                        (dW, d.t(), x.double(), off[1].t(), 2 * M if fine and act else M, 2.0 ** -24 if fine else 2.0 ** -8)):
        want = a @ b
        size = a.abs() @ b.abs()
        slack = each @ b.abs() + (rows / 16 + 2) * 2.0 ** -23 * size * 1.01
        assert bool(((got.double() - want).abs() <= slack + last * (want.abs() + slack)).all())
    want = d.sum(0)
    assert bool(((db.double() - want).abs() <= e.sum(0) + 2.0 ** -24 * (M / 8 + 64) * d.abs().sum(0)).all())
    # each alone, and none
    for want_dx, want_dW, want_db in ((True, False, False), (False, True, False), (False, False, True), (False, False, False)):
        alone = flp.linear_backward(dy, x, W, pre, activation=act, dw_dtype=dw_dtype, want_dx=want_dx, want_dW=want_dW,
                                    want_dbias=want_db)
        for a, b, want in zip(alone, (dx, dW, db), (want_dx, want_dW, want_db)):
            assert torch.equal(a, b) if want else a is None


@pytest.mark.parametrize("act", ["relu", "gelu", "gelu_tanh", "silu"])
@pytest.mark.parametrize("M,N,K", [(1, 72, 64), (1, 1000, 2047), (5, 4096, 1000), (16, 33, 520), (33, 2048, 4096), (64, 264, 136),
                                   (64, 1, 8)])
def test_backward_of_few_rows_rounds_once(flp, M, N, K, act):
    # d is exact to 2^-8 of 2^-8 of it, so that dx and dW in bf16 are the 64-bit ones to
    # half a step, on top of 2^-23 of the magnitudes a step of the accumulator
    g = torch.Generator().manual_seed(M + N + K)
    x, W, dy, pre = (matrix(*shape, 0, 0, g, scale)[1] for shape, scale in (((M, K), 1.0), ((N, K), K ** -0.5), ((M, N), 1.0),
                                                                            ((M, N), 1.5)))
    dx, dW, _ = flp.linear_backward(dy, x, W, pre, activation=act, dw_dtype=torch.bfloat16)
    d = dy.double() * act64(pre.double(), act)[1]
    e = 2.0 ** -17 * dy.double().abs()
    each = e + 2.0 ** -16 * (d.abs() + e)
    for got, a, b, off, terms in ((dx, d, W.double(), each, 2 * N), (dW, d.t(), x.double(), each.t(), 2 * M)):
        want = a @ b
        slack = off @ b.abs() + (terms / 16 + 2) * 2.0 ** -23 * (a.abs() @ b.abs()) * 1.01
        assert bool(((got.double() - want).abs() <= slack + 2.0 ** -8 * (want.abs() + slack)).all())


@pytest.mark.parametrize("M,N,K", SHAPES)
@pytest.mark.parametrize("act", ACTS)
def test_backward(flp, M, N, K, act):
    run_backward(flp, M, N, K, act, torch.bfloat16 if K % 2 else torch.float32)


@pytest.mark.parametrize("act", [None, "gelu"])
@pytest.mark.parametrize("dw_dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("pads,offsets", [((8, 16, 8, 24, 8), (0, 8, 0, 0, 0)), ((1, 0, 0, 0, 0), (0, 1, 0, 0, 0)), ((0, 0, 3, 0, 0), (0, 0, 1, 0, 0)),
                                          ((0, 0, 0, 3, 0), (0, 0, 0, 1, 0)), ((0, 0, 0, 0, 2), (0, 0, 0, 0, 3)), ((5, 3, 1, 7, 9), (1, 3, 5, 1, 7))])
def test_backward_layouts(flp, act, dw_dtype, pads, offsets):
    run_backward(flp, 200, 296, 136, act, dw_dtype, pads, offsets)


def test_backward_of_many_rows(flp):
    run_backward(flp, 5000, 264, 520, "silu")


@pytest.mark.parametrize("act", ACTS)
def test_wrapper_against_64_bit_autograd(flp, act):
    M, N, K = 150, 200, 96
    g = torch.Generator().manual_seed(5)
    x = torch.randn(M, K, generator=g).cuda().bfloat16().requires_grad_()
    W = (torch.randn(N, K, generator=g) / 10).cuda().bfloat16().requires_grad_()
    b = torch.randn(N, generator=g).cuda().bfloat16().requires_grad_()
    r = torch.randn(M, N, generator=g).cuda().bfloat16().requires_grad_()
    up = torch.randn(N, M, generator=g).cuda().bfloat16().t()
    y = flp.fused_linear(x, W, b, act, r)
    y.backward(up)
    ref = [t.detach().double().requires_grad_() for t in (x, W, b, r)]
    z = ref[0] @ ref[1].t() + ref[2]
    f = {None: lambda v: v, "relu": torch.relu, "gelu": torch.nn.functional.gelu, "silu": torch.nn.functional.silu,
         "gelu_tanh": lambda v: torch.nn.functional.gelu(v, approximate="tanh")}[act]
    (f(z) + ref[3]).backward(up.double())
    for got, want in zip((x, W, b, r), ref):
        assert got.grad.dtype is torch.bfloat16
        rel = float((got.grad.double() - want.grad).norm() / want.grad.norm())
        assert rel <= 0.01, rel  # v, d and the result rounded to bf16
    # gradients of some inputs alone, and none recorded
    x2 = x.detach().requires_grad_()
    flp.fused_linear(x2, W.detach(), None, act).sum().backward()
    assert x2.grad is not None
    with torch.no_grad():
        assert torch.equal(flp.fused_linear(x, W, b, act, r), y)
    dx, = torch.autograd.grad(flp.fused_linear(x, W, b, act).float().sum(), x, create_graph=True)
    with pytest.raises(RuntimeError, match="cannot be differentiated again"):
        dx.sum().backward()


@pytest.mark.parametrize("M,N,K", [(4, 600, 512), (300, 257, 100)])
def test_captured_and_replayed(flp, M, N, K):
    g = torch.Generator().manual_seed(3)
    _, x = matrix(M, K, gen=g)
    _, W = matrix(N, K, gen=g, scale=0.1)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())

    def step():
        y, pre = flp.linear(x, W, activation="gelu", keep=True)
        return [y, pre, *flp.linear_backward(y, x, W, pre, activation="gelu")]

    with torch.cuda.stream(s):
        step()
    s.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=s):
        out = step()
    x.copy_(matrix(M, K, gen=g)[1])
    for _ in range(2):
        graph.replay()
    torch.cuda.synchronize()
    for a, b in zip(out, step()):
        assert torch.equal(a, b)


def test_workspaces(flp):
    g = torch.Generator().manual_seed(3)
    _, x = matrix(4, 512, gen=g)
    _, W = matrix(600, 512, gen=g)
    small = torch.empty(64, dtype=torch.uint8, device="cuda")
    with pytest.raises(flp.FlpError) as e:
        flp.linear_backward(flp.linear(x, W), x, W, workspace=small)
    assert e.value.status == flp.FLP_ERR_WORKSPACE
    big = torch.full((1 << 24,), 255, dtype=torch.uint8, device="cuda")  # what it holds does not matter
    y = flp.linear(x, W, workspace=big)
    assert torch.equal(y, flp.linear(x, W))
    for a, b in zip(flp.linear_backward(y, x, W, workspace=big), flp.linear_backward(y, x, W)):
        assert torch.equal(a, b)
    assert flp.get_error(big) == flp.FLP_OK


@pytest.mark.parametrize("form", [0, 1, 2, 3])
@pytest.mark.parametrize("stall", [-1, 0, 1, 2, 3, 4])
def test_bounded_waits(flp, form, stall):
    """Whole tiles, partial tiles, the tiles of few rows, and those of a cluster: two tiles
    (five of few rows) of three blocks, one block a CTA in the last form."""
    ws = torch.empty(flp.SELFTEST_LINEAR_BYTES, dtype=torch.uint8, device="cuda")
    status = flp.selftest_linear_timeout(form, stall, 20_000_000, workspace=ws)
    at = flp.SELFTEST_LINEAR_OUTPUT_OFFSET
    y = ws[at:at + 192 * 520 * 2].view(torch.bfloat16).view(192, 520)
    if stall < 0 or stall >= {0: 6, 1: 6, 2: 3, 3: 1}[form]:
        assert status == flp.FLP_OK and bool((y == 0).all())
        return
    assert status == flp.FLP_ERR_TIMEOUT
    first, second = y[:, :512], y[:, 512:]
    assert bool((first == 0).all() if form < 2 and stall >= 3 else torch.isnan(first.float()).all())
    assert bool(torch.isnan(second.float()).all())
    assert flp.selftest_linear_timeout(form, -1, 10 ** 9, workspace=ws) == flp.FLP_OK
