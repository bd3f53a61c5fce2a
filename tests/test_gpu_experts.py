"""Tokens sorted by expert, their rows brought there and back, and the gradients.

The order is whole numbers and the gather a copy: both exactly equal.  A combine's
sum of k products in fp32 is off by at most (k + 1) 2^-24 of the sum of the
products' magnitudes (each fma rounds once), and is rounded once to the output's
type.  dys is one product, rounded in fp32 and to its type.  dweights, a sum of H
products over 256 threads and then their tree, is off by at most (H / 256 + 16)
2^-24 of the sum of the magnitudes (fewer additions than that in any order it runs).
"""
import pytest
import torch

pytestmark = pytest.mark.gpu
HALF = {torch.bfloat16: 2.0 ** -8, torch.float32: 2.0 ** -24}  # half a step, relative to the value


@pytest.fixture(scope="module")
def flp():
    if not torch.cuda.is_available():
        pytest.skip("needs a CUDA GPU")
    from entropy_loss_gb300 import build, flp as _flp
    build.build()
    _flp.load()
    return _flp


def choices(T, k, E, seed=0, dropped=0.1, skew=True):
    g = torch.Generator().manual_seed(seed)
    e = torch.randint(0, E, (T, k), generator=g)
    if skew and E > 2:
        e = torch.where(torch.rand(T, k, generator=g) < 0.4, e % 2, e)
    out = torch.where(torch.rand(T, k, generator=g) < 0.5, -1 - e, E + 7 * e)
    return torch.where(torch.rand(T, k, generator=g) < dropped, out, e)


def order64(e, E):
    """(rows, slots, counts, offsets) by Python's stable sort."""
    flat = [x if 0 <= x < E else E for x in e.reshape(-1).tolist()]
    slots = sorted(range(len(flat)), key=lambda s: flat[s])
    rows = torch.empty(len(flat), dtype=torch.int32)
    rows[torch.tensor(slots, dtype=torch.long)] = torch.arange(len(flat), dtype=torch.int32)
    counts = torch.bincount(torch.tensor(flat, dtype=torch.long), minlength=E + 1)[:E]
    return (rows.view(e.shape), torch.tensor(slots, dtype=torch.int32), counts,
            torch.cat([torch.zeros(1, dtype=torch.long), counts.cumsum(0)]))


def same_order(got, want):
    for a, b in zip(got, want):
        assert a.dtype is b.dtype and torch.equal(a.cpu(), b)


SIZES = [(0, 3, 5), (1, 1, 1), (1, 8, 8), (3, 2, 1024), (31, 1, 2), (33, 3, 7), (1000, 8, 256), (4096, 2, 8), (4097, 2, 8),
         (2731, 3, 12), (9000, 1, 1), (20001, 3, 33), (70000, 8, 256), (50001, 2, 1024), (12345, 5, 1023)]


@pytest.mark.parametrize("T,k,E", SIZES)
def test_sort(flp, T, k, E):
    e = choices(T, k, E, seed=T + k)
    same_order(flp.expert_sort(e.cuda(), E), order64(e, E))


@pytest.mark.parametrize("T,k", [(5, 2), (9000, 2)])
@pytest.mark.parametrize("what", ["all dropped", "one expert", "extremes"])
def test_sort_of_unusual_choices(flp, T, k, what):
    E = 6
    e = {"all dropped": torch.full((T, k), -1), "one expert": torch.full((T, k), 3),
         "extremes": torch.tensor([2 ** 63 - 1, -2 ** 63, 2 ** 32, 5]).repeat(T * k // 4 + 1)[:T * k].view(T, k)}[what]
    same_order(flp.expert_sort(e.cuda(), E), order64(e, E))


def matrix(M, H, dtype, pad=0, offset=0, gen=None):
    buf = torch.full((M * (H + pad) + offset + 8,), 7.0, dtype=dtype)
    view = buf[offset:offset + M * (H + pad)].view(M, H + pad)[:, :H]
    view.copy_(torch.randn(M, H, generator=gen))
    dev = buf.cuda()
    return dev, dev[offset:offset + M * (H + pad)].view(M, H + pad)[:, :H]


def untouched(buf, view, before):
    """What lies between and around the rows is as it was."""
    ours = torch.zeros_like(buf, dtype=torch.bool)
    torch.as_strided(ours, view.shape, view.stride(), view.storage_offset()).fill_(True)
    assert torch.equal(buf[~ours], before[~ours])


# width, extra pitch and offset of the tokens' matrix and of the slots'
LAYOUTS = [(8, 0, 0, 0, 0), (24, 0, 8, 16, 0), (64, 0, 0, 0, 0), (120, 8, 0, 0, 8), (256, 0, 0, 0, 0), (2048, 0, 0, 8, 0),
           (5120, 0, 8, 0, 0), (1, 0, 0, 0, 0), (7, 1, 0, 0, 0), (33, 0, 1, 5, 3), (257, 0, 0, 2, 1), (1000, 4, 0, 1, 0), (2047, 0, 1, 0, 0), (520, 0, 0, 1, 1)]


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("H,pad1,off1,pad2,off2", LAYOUTS)
def test_gather_is_a_copy(flp, dtype, H, pad1, off1, pad2, off2):
    T, k, E = 37, 3, 5
    g = torch.Generator().manual_seed(H)
    e = choices(T, k, E, seed=H)
    order = flp.expert_sort(e.cuda(), E)
    _, x = matrix(T, H, dtype, pad1, off1, g)
    buf, out = matrix(T * k, H, dtype, pad2, off2, g)
    before = buf.clone()
    assert flp.expert_gather(x, order, out=out) is out
    want = x[order.slots.long() // k]
    want[int(order.offsets[-1]):] = 0
    assert torch.equal(out, want)
    untouched(buf, out, before)
    assert torch.equal(flp.expert_gather(x, order), want)


@pytest.mark.parametrize("weights", [None, torch.float32, torch.bfloat16])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("H,pad1,off1,pad2,off2", LAYOUTS)
def test_combine_and_its_gradient(flp, dtype, weights, H, pad1, off1, pad2, off2):
    for T, k, E in ((29, 3, 5), (6, 9, 9), (2100, 2, 7)):
        g = torch.Generator().manual_seed(H)
        e = choices(T, k, E, seed=H, dropped=0.3)
        e[1] = -1  # a token without an expert
        order = flp.expert_sort(e.cuda(), E)
        total = int(order.offsets[-1])
        rows = order.rows.long()
        live = (rows < total).double()
        w = None if weights is None else torch.randn(T, k, generator=g).cuda().to(weights)
        w64 = live if w is None else w.double() * live
        _, ys = matrix(T * k, H, dtype, pad2, off2, g)
        ys[total:] = float("nan")  # not looked at
        ys64 = torch.nan_to_num(ys.double(), nan=0.0)
        buf, out = matrix(T, H, dtype, pad1, off1, g)
        before = buf.clone()
        got = flp.expert_combine(ys, order, w, out=out)
        terms = w64[..., None] * ys64[rows]
        want, size = terms.sum(1), terms.abs().sum(1)
        tol = (k + 1) * 2.0 ** -24 * size + HALF[dtype] * (want.abs() + (k + 1) * 2.0 ** -24 * size)
        assert bool(((got.double() - want).abs() <= tol).all())
        assert bool((got[1] == 0).all())
        untouched(buf, out, before)
        assert torch.equal(flp.expert_combine(ys, order, w), got)

        _, dy = matrix(T, H, dtype, pad1, off1, g)
        buf, dys_out = matrix(T * k, H, dtype, pad2, off2, g)
        before = buf.clone()
        dys, dw = flp.expert_combine_backward(dy, ys, order, w, out=dys_out)
        want = torch.zeros(T * k, H, dtype=torch.float64, device="cuda")
        want[rows.reshape(-1)] = (w64[..., None] * dy.double()[:, None]).reshape(T * k, H)
        tol = (2.0 ** -24 + HALF[dtype] * (1 + 2.0 ** -24)) * want.abs()
        assert bool(((dys.double() - want).abs() <= tol).all())
        untouched(buf, dys_out, before)
        terms = dy.double()[:, None] * ys64[rows] * live[..., None]
        assert dw.dtype is torch.float32
        assert bool(((dw.double() - terms.sum(2)).abs() <= (H / 256 + 16) * 2.0 ** -24 * terms.abs().sum(2)).all())
        assert bool((dw[live == 0] == 0).all())
        # without the weights' gradient ys is not needed
        alone, none = flp.expert_combine_backward(dy, None, order, w, want_dweights=False)
        assert none is None and torch.equal(alone, dys)


def test_long_rows_and_many_choices(flp):
    """More choices than a warp has lanes, rows longer than a block takes at once."""
    T, k, E, H = 5, 70, 100, 9001
    e = choices(T, k, E, seed=3)
    order = flp.expert_sort(e.cuda(), E)
    x = torch.randn(T, H, device="cuda")
    xs = flp.expert_gather(x, order)
    kept = int(order.offsets[-1])
    assert torch.equal(xs[:kept], x[order.slots[:kept].long() // k]) and bool((xs[kept:] == 0).all())
    w = torch.randn(T, k, device="cuda")
    live = (order.rows.long() < kept).double()
    terms = (w.double() * live)[..., None] * xs.double()[order.rows.long()]
    got = flp.expert_combine(xs, order, w)
    assert bool(((got.double() - terms.sum(1)).abs() <= (k + 3) * 2.0 ** -24 * terms.abs().sum(1)).all())
    dy = torch.randn(T, H, device="cuda")
    dys, dw = flp.expert_combine_backward(dy, xs, order, w)
    want = (dy.double()[:, None] * xs.double()[order.rows.long()]).sum(2) * live
    size = (dy.double()[:, None] * xs.double()[order.rows.long()]).abs().sum(2)
    assert bool(((dw.double() - want).abs() <= (H / 256 + 16) * 2.0 ** -24 * size).all())


def test_infinities_where_they_belong(flp):
    e = torch.tensor([[0, 1], [1, -1], [0, 0]]).cuda()
    order = flp.expert_sort(e, 2)
    ys = torch.ones(6, 16, device="cuda")
    ys[int(order.rows[0, 0])] = float("inf")
    ys[int(order.rows[1, 1])] = float("nan")  # a dropped slot
    y = flp.expert_combine(ys, order, torch.ones(3, 2, device="cuda"))
    assert bool((y[0] == float("inf")).all()) and bool((y[1] == 1).all()) and bool((y[2] == 2).all())


def test_entries_that_are_no_position_are_passed_over(flp):
    e = torch.tensor([[0, 1], [1, 0]]).cuda()
    order = flp.expert_sort(e, 2)
    rows = order.rows.clone()
    rows[0, 1] = 1 << 30
    rows[1, 0] = -5
    bad = order._replace(rows=rows)
    x = torch.randn(2, 8, device="cuda")
    out = torch.zeros(4, 8, device="cuda")
    flp.expert_gather(x, bad, out=out)
    assert torch.equal(out[int(rows[0, 0])], x[0]) and int((out == 0).all(1).sum()) == 2
    assert torch.equal(flp.expert_combine(out, bad), x)
    dys, dw = flp.expert_combine_backward(x, out, bad, out=torch.zeros(4, 8, device="cuda"))
    assert float(dw[0, 1]) == 0 and float(dw[1, 0]) == 0 and int((dys == 0).all(1).sum()) == 2


def test_wrappers_against_64_bit_autograd(flp):
    T, k, E, H = 50, 3, 6, 72
    g = torch.Generator().manual_seed(0)
    e = choices(T, k, E, seed=9).cuda()
    x = torch.randn(T, H, generator=g).cuda().requires_grad_()
    w = torch.rand(T, k, generator=g).cuda().requires_grad_()
    up = torch.randn(H, T, generator=g).cuda().t()  # an upstream gradient that is not contiguous
    order = flp.expert_sort(e, E)
    flp.fused_expert_combine(torch.sin(flp.fused_expert_gather(x, order)), order, w).backward(up)
    xr, wr = x.detach().double().requires_grad_(), w.detach().double().requires_grad_()
    live = ((e >= 0) & (e < E)).double()
    ((torch.sin(xr)[:, None] * (wr * live)[..., None]).sum(1) * up).sum().backward()
    assert torch.allclose(x.grad.double(), xr.grad, rtol=1e-5, atol=1e-5)
    assert torch.allclose(w.grad.double(), wr.grad, rtol=1e-5, atol=1e-5)
    # bf16 weights get a bf16 gradient; none is taken where none is wanted
    wb = w.detach().to(torch.bfloat16).requires_grad_()
    flp.fused_expert_combine(x.detach()[:1].expand(T * k, H).contiguous(), order, wb).sum().backward()
    assert wb.grad.dtype is torch.bfloat16
    x2 = x.detach().clone().requires_grad_()
    flp.fused_expert_combine(flp.fused_expert_gather(x2, order), order).sum().backward()
    assert torch.equal(x2.grad, live.sum(1, keepdim=True).float().expand(T, H))
    y = flp.fused_expert_gather(x2, order)
    dx, = torch.autograd.grad(y.square().sum(), x2, create_graph=True)
    with pytest.raises(RuntimeError, match="cannot be differentiated again"):
        dx.sum().backward()


def test_captured_and_replayed_on_another_stream(flp):
    T, k, E, H = 9000, 2, 16, 264
    e = choices(T, k, E, seed=1).cuda()
    x = torch.randn(T, H, device="cuda")
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())

    def step():
        order = flp.expert_sort(e, E)
        xs = flp.expert_gather(x, order)
        return order, xs, flp.expert_combine(xs, order)

    with torch.cuda.stream(s):
        step()
    s.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=s):
        order, xs, y = step()
    e.copy_(choices(T, k, E, seed=2).cuda())
    x.normal_()
    graph.replay()
    torch.cuda.synchronize()
    same_order(order, order64(e.cpu(), E))
    assert torch.equal(xs, flp.expert_gather(x, order)) and torch.equal(y, flp.expert_combine(xs, order))
    # the caller's stream argument and workspace
    ws = torch.empty(1 << 20, dtype=torch.uint8, device="cuda")
    with_ws = flp.expert_sort(e, E, workspace=ws, stream=s)
    s.synchronize()
    same_order(with_ws, [t.cpu() for t in order])
