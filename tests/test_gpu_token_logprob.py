"""Log-probabilities of given tokens from logits, entropy, top alternatives, gradient.

Tolerances, for rows of V logits z = s x with largest M and S = sum exp(z - M):
every term of S is off by its exponent's rounding, at most 3 2^-24 |z - M| (difference,
factor, product), and by 2^-22 of itself (the exponential), so S is off by at most
2^-22 + 3 2^-24 E|z - M| of itself, the mean taken over the distribution, which is at
most 2^-22 + 3 2^-24 (H + 1) with the entropy H (E(M - z) <= H as M - z <= lse - z),
and adding terms of one sign in any order by at most another n 2^-24, n the additions a
term passes through: at most 16 a chunk in pairs and one per chunk, so below
V / 1024 + 64 here; the errors' signs alternate, but the bound stands.  Call the sum r.
logprob and lse carry r, ln's own 2^-23 |ln S| and the roundings of s (x_y - M), lse and
the difference: 2^-22 |z_y - M| + 2^-23 |lse|.  The entropy carries r (H + 2) twice.
The gradient: p carries the exponent's error 2^-23 (|z| + |lse| + |z - lse|) and 2^-22;
the rest are a few fp32 roundings and the rounding to its type.
"""
import math

import pytest
import torch

pytestmark = pytest.mark.gpu
IGNORE = -100
HALF = {torch.bfloat16: 2.0 ** -8, torch.float32: 2.0 ** -24}


@pytest.fixture(scope="module")
def flp():
    if not torch.cuda.is_available():
        pytest.skip("needs a CUDA GPU")
    from entropy_loss_gb300 import build, flp as _flp
    build.build()
    _flp.load()
    return _flp


def make(M, V, dtype, pad=0, offset=0, seed=0, spread=2.0):
    g = torch.Generator().manual_seed(seed)
    buf = torch.full((M * (V + pad) + offset + 8,), float("nan"), dtype=dtype)  # nothing between the rows is read
    view = buf[offset:offset + M * (V + pad)].view(M, V + pad)[:, :V]
    view.copy_(spread * torch.randn(M, V, generator=g) + torch.randn(V, generator=g))
    dev = buf.cuda()
    y = torch.randint(0, V, (M,), generator=g)
    y[torch.rand(M, generator=g) < 0.1] = IGNORE
    return dev[offset:offset + M * (V + pad)].view(M, V + pad)[:, :V], y.cuda()


def order_of(x, k):
    """Columns of the k largest above -inf, equal ones by column, from the definition."""
    out = []
    for row in x.float().cpu():
        keep = torch.nonzero(row > -math.inf)[:, 0].tolist()
        vals = row.tolist()
        first = sorted(keep, key=lambda j: (-vals[j], j))[:k]
        out.append(first + [-1] * (k - len(first)))
    return torch.tensor(out)


def check(flp, x, y, k, scale, **kw):
    lp, lse, ent, val, idx = flp.token_logprob(x, y, top=k, scale=scale, ignore_index=IGNORE, **kw)
    V = x.shape[1]
    z = x.double() * float(torch.tensor(scale, dtype=torch.float32))
    lse64 = torch.logsumexp(z, 1)
    p = torch.exp(z - lse64[:, None])
    ent64 = torch.special.entr(p).sum(1)
    live = y != IGNORE
    r = 2.0 ** -22 + 3 * 2.0 ** -24 * (ent64 + 1) + (V / 1024 + 64) * 2.0 ** -24
    top = z.amax(1)
    base = r + 2.0 ** -23 * ((lse64 - top).abs() + lse64.abs())
    assert bool(((lse.double() - lse64).abs() <= base).all())
    zy = z.gather(1, y.clamp(min=0)[:, None])[:, 0]
    want = torch.where(live, zy - lse64, 0)
    assert bool(((lp.double() - want).abs() <= base + 2.0 ** -22 * (zy - top).abs()).all())
    if ent is not None:
        want = torch.where(live, ent64, 0)
        assert bool(((ent.double() - want).abs() <= 2 * r * (ent64 + 2)).all())
    if k:
        want = order_of(x, k).cuda()
        assert idx.dtype is torch.int64 and torch.equal(idx, want)
        zt = z.gather(1, want.clamp(min=0))
        wv = torch.where(want >= 0, zt - lse64[:, None], -math.inf)
        same = torch.isinf(wv) & (val.double() == wv)
        assert bool((same | ((val.double() - wv).abs() <= base[:, None] + 2.0 ** -22 * (zt - top[:, None]).abs())).all())
    return lp, lse, ent


SIZES = [(1, 1, 1), (3, 2, 2), (5, 7, 3), (4, 33, 32), (2, 255, 5), (3, 256, 32), (7, 1000, 20), (5, 4096, 1), (3, 4097, 20),
         (2, 5000, 32), (1, 16384, 20), (1, 16385, 8), (3, 50257, 20), (1, 131072, 32), (40, 32000, 2), (200, 9001, 5), (400, 8192, 0)]


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("M,V,k", SIZES)
@pytest.mark.parametrize("pad,offset,scale", [(0, 0, 1.0), (3, 1, 0.7)])
def test_forward(flp, dtype, M, V, k, pad, offset, scale):
    x, y = make(M, V, dtype, pad, offset, seed=V + M)
    check(flp, x, y, k, scale)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("kind", ["all equal", "two values", "ascending", "descending", "zeros of both signs", "one peak",
                                  "largest at the end"])
def test_rows_that_fill_the_list(flp, dtype, kind):
    M, V, k = 2, 40001, 20
    j = torch.arange(V).float()
    row = {"all equal": torch.full((V,), 3.25), "two values": torch.where(torch.rand(V) < 0.5, 1.0, 1.5),
           "ascending": j / 4096, "descending": -j / 4096,
           "zeros of both signs": torch.where(torch.rand(V) < 0.5, 0.0, -0.0), "one peak": torch.where(j == 30000, 90.0, -90.0),
           "largest at the end": torch.where(j >= V - 3000, 5.0, -5.0)}[kind]
    x = row.repeat(M, 1).to(dtype).cuda()
    y = torch.tensor([V - 1, 5]).cuda()
    check(flp, x, y, k, 1.0)
    check(flp, x[:, :3000].contiguous(), torch.tensor([2999, 5]).cuda(), k, 1.0)
    many = x[:1].expand(700, V).contiguous()  # one block a row
    check(flp, many, y[:1].expand(700).contiguous(), 5, 1.0) if kind in ("all equal", "ascending") else None


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("V", [40, 3000, 60000])
def test_masked_rows(flp, dtype, V):
    low = torch.finfo(dtype).min
    x, y = make(6, V, dtype, seed=V)
    y[:] = 3
    x[0, 10:] = -math.inf            # ten left: fewer than the alternatives asked for
    x[1] = -math.inf                 # nothing left
    x[2, ::2] = -math.inf
    x[3] = low                       # the type's lowest value throughout
    x[4, 1:] = low                   # and in all places but one
    y[5] = IGNORE
    lp, lse, ent, val, idx = flp.token_logprob(x, y, top=16)
    assert float(lp[1]) == -math.inf and float(lse[1]) == -math.inf and float(ent[1]) == 0
    assert bool((val[1] == -math.inf).all()) and bool((idx[1] == -1).all())
    assert bool((idx[0, 10:] == -1).all()) and sorted(idx[0, :10].tolist()) == list(range(10))
    keep = torch.tensor([0, 2, 5]).cuda()
    check(flp, x[keep].contiguous(), y[keep].contiguous(), 16, 1.0)
    assert abs(float(lp[3]) + math.log(V)) < 1e-5 and abs(float(ent[3]) - math.log(V)) < 1e-5
    assert idx[3].tolist() == list(range(16))
    assert float(lp[4]) == -math.inf or float(lp[4]) < -1e30
    assert float(ent[4]) == 0 and float(val[4, 0]) == 0 and int(idx[4, 0]) == 0
    assert float(lp[5]) == 0 and float(ent[5]) == 0
    # and the gradient: zeros for the empty row, no NaN for the masked ones
    g = torch.ones(6, device="cuda")
    dz = flp.token_logprob_backward(x, y, lse, ent, g, g)
    assert bool(torch.isfinite(dz.float()).all())
    assert bool((dz[1] == 0).all()) and bool((dz[5] == 0).all()) and bool((dz[0, 10:] == 0).all())


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("what", [math.nan, math.inf])
@pytest.mark.parametrize("V", [100, 70000])
def test_nan_and_infinity(flp, dtype, what, V):
    x, y = make(4, V, dtype, seed=1)
    y[:] = 2
    x[1, V - 1] = what
    x[2] = what
    y[3] = IGNORE
    x[3, 5] = what
    lp, lse, ent, val, idx = flp.token_logprob(x, y, top=4)
    for t in (lp, lse, ent):
        assert bool(torch.isfinite(t[0])) and bool(torch.isnan(t[1:3]).all())
    assert bool(torch.isnan(val[1:]).all()) and bool((idx[1:] == -1).all())
    assert float(lp[3]) == 0 and float(ent[3]) == 0
    dz = flp.token_logprob_backward(x, y, lse, ent, torch.ones(4, device="cuda"))
    assert bool(torch.isnan(dz[1:3].float()).all()) and bool((dz[3] == 0).all()) and bool(torch.isfinite(dz[0].float()).all())


def test_targets_outside_the_vocabulary(flp):
    x, y = make(4, 500, torch.float32)
    y.copy_(torch.tensor([-1, 500, 2 ** 40, 7]))
    lp, lse, ent, _, _ = flp.token_logprob(x, y)
    assert bool(torch.isnan(lp[:3]).all()) and bool(torch.isfinite(lp[3])) and bool(torch.isfinite(lse).all())
    dz = flp.token_logprob_backward(x, y, lse, ent, torch.ones(4, device="cuda"))
    p = torch.softmax(x[:3].double(), 1)
    assert torch.allclose(dz[:3].double(), -p, rtol=1e-5, atol=1e-9)


def test_without_entropy_and_empty(flp):
    x, y = make(3, 100, torch.bfloat16)
    lp, lse, ent, val, idx = flp.token_logprob(x, y, compute_entropy=False)
    assert ent is None and val is None and idx is None
    full = flp.token_logprob(x, y, top=3)
    assert torch.equal(lp, full[0]) and torch.equal(lse, full[1])
    got = flp.token_logprob(x[:0], y[:0], top=2)
    assert got[0].shape == (0,) and got[3].shape == (0, 2)
    assert flp.token_logprob_backward(x[:0], y[:0], lse[:0], None, None).shape == (0, 100)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("M,V,pad,offset", [(1, 1, 0, 0), (3, 7, 0, 0), (5, 1000, 0, 0), (4, 1024, 8, 0), (6, 5001, 2, 1), (2, 131072, 0, 0),
                                            (3, 4099, 1, 3)])
def test_backward(flp, dtype, M, V, pad, offset):
    scale = 0.7
    x, y = make(M, V, dtype, pad, offset, seed=V)
    lp, lse, ent, _, _ = flp.token_logprob(x, y, scale=scale)
    g = torch.Generator().manual_seed(2)
    g_lp, g_ent = torch.randn(M, generator=g).cuda(), torch.randn(M, generator=g).cuda()
    s = float(torch.tensor(scale, dtype=torch.float32))
    z = x.double() * s
    l64, e64 = lse.double()[:, None], ent.double()[:, None]
    live = (y != IGNORE).double()[:, None]
    for a, b in ((g_lp, g_ent), (g_lp, None), (None, g_ent), (None, None)):
        dz = flp.token_logprob_backward(x, y, lse, ent, a, b, scale=scale, ignore_index=IGNORE)
        a64 = torch.zeros(M, 1, dtype=torch.float64, device="cuda") if a is None else a.double()[:, None]
        b64 = torch.zeros_like(a64) if b is None else b.double()[:, None]
        p = torch.exp(z - l64)
        hit = torch.zeros_like(z).scatter_(1, y.clamp(min=0)[:, None], 1.0)
        want = s * live * (a64 * (hit - p) - b64 * p * (z - l64 + e64))
        size = s * live * (a64.abs() * (hit + p) + b64.abs() * p * ((z - l64).abs() + e64.abs()))
        rel = 2.0 ** -22 + 2.0 ** -23 * (z.abs() + l64.abs() + (z - l64).abs()) + 8 * 2.0 ** -24
        # sums below the normal range of fp32 flush to 0
        assert bool(((dz.double() - want).abs() <= rel * size + HALF[dtype] * (want.abs() + rel * size) + 2.0 ** -125).all())
    wide = torch.full((M, V + 5), 9.0, dtype=dtype, device="cuda")
    out = flp.token_logprob_backward(x, y, lse, ent, g_lp, g_ent, scale=scale, out=wide[:, 2:V + 2])
    assert torch.equal(out, flp.token_logprob_backward(x, y, lse, ent, g_lp, g_ent, scale=scale))
    assert bool((wide[:, :2] == 9).all()) and bool((wide[:, V + 2:] == 9).all())
    inplace = x.clone()
    assert torch.equal(flp.token_logprob_backward(inplace, y, lse, ent, g_lp, g_ent, scale=scale, out=inplace), out)


def test_gradient_against_differences(flp):
    """The wrapper's gradient along random directions against central differences in 64 bits."""
    M, V, scale = 5, 300, 1.3
    x, y = make(M, V, torch.float32, seed=4)
    x = x.clone().requires_grad_()
    lp, ent, val, idx = flp.fused_token_logprob(x, y, top=3, scale=scale)
    a, b = torch.randn(M, device="cuda"), torch.randn(M, device="cuda")
    (lp * a + ent * b).sum().backward()

    def f(z):
        logp = torch.log_softmax(z * float(torch.tensor(scale)), 1)
        live = (y != IGNORE).double()
        e = -(torch.exp(logp) * logp).sum(1)
        return (live * (a.double() * logp.gather(1, y.clamp(min=0)[:, None])[:, 0] + b.double() * e)).sum()

    for seed in range(3):
        d = torch.randn(M, V, dtype=torch.float64, generator=torch.Generator().manual_seed(seed)).cuda()
        x64 = x.detach().double()
        want = (f(x64 + 1e-5 * d) - f(x64 - 1e-5 * d)) / 2e-5
        got = (x.grad.double() * d).sum()
        assert abs(float(got - want)) <= 1e-5 * float((x.grad.double() * d).abs().sum())
    assert not val.requires_grad and not idx.requires_grad
    x.grad = None
    flp.fused_token_logprob(x, y, scale=scale, compute_entropy=False)[0].sum().backward()
    p = torch.softmax(x.detach().double() * scale, 1)
    hit = torch.zeros_like(p).scatter_(1, y.clamp(min=0)[:, None], 1.0)
    assert torch.allclose(x.grad.double(), scale * (hit - p) * (y != IGNORE)[:, None], rtol=1e-4, atol=1e-7)
    dz, = torch.autograd.grad(flp.fused_token_logprob(x, y)[0].sum(), x, create_graph=True)
    with pytest.raises(RuntimeError, match="cannot be differentiated again"):
        dz.sum().backward()


def test_captured_and_replayed(flp):
    x, y = make(3, 60000, torch.bfloat16, seed=8)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        flp.token_logprob(x, y, top=5)
    s.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=s):
        out = flp.token_logprob(x, y, top=5)
        dz = flp.token_logprob_backward(x, y, out[1], out[2], out[0])
    x.copy_(make(3, 60000, torch.bfloat16, seed=9)[0])
    graph.replay()
    torch.cuda.synchronize()
    again = flp.token_logprob(x, y, top=5, stream=s)
    s.synchronize()
    for a, b in zip(out, again):
        assert torch.equal(a, b)
    assert torch.equal(dz, flp.token_logprob_backward(x, y, again[1], again[2], again[0]))
