"""Cases of the training-step operators beside the fused head, and their plain forms.

Operators: layer norm forward and backward (from the activations or from their
8-bit checkpoint), the 8-bit checkpoint itself (written and read back), the
weight gradient of a linear layer from its input's 8-bit checkpoint, and the
router balance loss with per-expert counts and the gradient.

``run`` computes the plain form (elementary torch operations in 32 bits) or,
with ``own`` set, calls the framework's operators; ``exact`` computes the same
outputs from the definitions in 64 bits.
"""
import math

import torch

own = False

EPS = 1e-5
BLOCK = 32            # columns of a checkpoint block (one shared power-of-two step)
DTYPES = {"bf16": torch.bfloat16, "fp32": torch.float32}


# ------------------------------------------------------------------- cases

def listed():
    return [
        # one decoded position through a model's last norm: launch latency
        dict(name="norm_forward_one_row", op="norm_forward", rows=1, cols=4096, dtype="bf16", extra=0, checkpoint=False),
        # odd sizes in full precision, rows cut out of a wider activation (a small research model)
        dict(name="norm_forward_odd_fp32", op="norm_forward", rows=777, cols=2047, dtype="fp32", extra=9, checkpoint=False),
        # a training micro-batch whose norm also writes its input's checkpoint
        dict(name="norm_forward_checkpoint", op="norm_forward", rows=20001, cols=4096, dtype="bf16", extra=0, checkpoint=True),
        # the tiny model of the unit tests: launch latency of the two-output backward
        dict(name="norm_backward_tiny", op="norm_backward", rows=256, cols=256, dtype="bf16", extra=0, checkpoint=False),
        # an ordinary micro-batch, activations kept in bf16
        dict(name="norm_backward_ordinary", op="norm_backward", rows=8192, cols=4096, dtype="bf16", extra=0, checkpoint=False),
        # the largest micro-batch, activations kept as 8-bit checkpoints
        dict(name="norm_backward_checkpoint", op="norm_backward", rows=32768, cols=5120, dtype="bf16", extra=0, checkpoint=True),
        # a short odd-width activation: the last block of every row is cut
        dict(name="checkpoint_short", op="checkpoint", rows=300, cols=1023, dtype="fp32", extra=0),
        # one layer's activation of a large micro-batch, written and read back
        dict(name="checkpoint_large", op="checkpoint", rows=20001, cols=7168, dtype="bf16", extra=0),
        # a narrow projection over a short batch: latency and little parallel work
        dict(name="weight_grad_small", op="weight_grad", rows=777, outs=264, ins=1000, dtype="bf16"),
        # a full-width projection of a training micro-batch
        dict(name="weight_grad_large", op="weight_grad", rows=8192, outs=8192, ins=5120, dtype="fp32"),
        # few tokens, few experts: launch latency
        dict(name="balance_small", op="balance", rows=64, experts=8, top_k=2, dtype="bf16", masked=False),
        # a global batch through a wide router, padding masked
        dict(name="balance_large", op="balance", rows=65536, experts=256, top_k=8, dtype="fp32", masked=True),
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def _width(rng, lo, hi):
    """A width: multiples of 64 as models have them, or any number."""
    w = _log(rng, lo, hi)
    w = max(64, w // 64 * 64) if rng.random() < 0.6 and hi >= 64 else w
    return w + 64 if w == 3072 else w


def draw(rng):
    op = rng.choice(["norm_forward", "norm_backward", "checkpoint", "weight_grad", "balance"])
    dtype = rng.choice(["bf16", "fp32"])
    if op in ("norm_forward", "norm_backward", "checkpoint"):
        cols = _width(rng, 32, 8192)
        # within the largest listed case's bytes
        rows = _log(rng, 1, min(65536, 32768 * 5120 // cols // (1 if dtype == "bf16" else 2)))
        extra = rng.choice([0, 0, 8, 5])
        c = dict(op=op, rows=rows, cols=cols, dtype=dtype, extra=extra)
        if op != "checkpoint":
            c["checkpoint"] = rng.random() < 0.5
        return c
    if op == "weight_grad":
        outs, ins = _width(rng, 64, 8192), _width(rng, 64, 8192)
        rows = _log(rng, 1, min(32768, 8192 * 8192 * 5120 // (outs * ins)))
        return dict(op=op, rows=rows, outs=outs, ins=ins, dtype=dtype)
    experts = _log(rng, 2, 256)
    return dict(op=op, rows=_log(rng, 1, 65536), experts=experts, top_k=rng.randint(1, min(8, experts)), dtype=dtype,
                masked=rng.random() < 0.5)


def _size(dtype):
    return 2 if dtype == "bf16" else 4


def work(case):
    op, rows, e = case["op"], case["rows"], _size(case["dtype"])
    if op in ("norm_forward", "norm_backward", "checkpoint"):
        cols = case["cols"]
        n = rows * cols
        packed = rows * (-(-cols // BLOCK)) * (BLOCK + 1)
        if op == "checkpoint":  # written, then read back
            return {"bytes": n * e + packed + packed + n * e, "flops": 4 * n}
        if op == "norm_forward":
            back = packed + packed + n * e if case["checkpoint"] else 0
            return {"bytes": 2 * n * e + 8 * rows + 2 * cols * e + back, "flops": 8 * n}
        x = packed if case["checkpoint"] else n * e
        return {"bytes": x + 2 * n * e + 8 * rows + cols * e + 8 * cols, "flops": 14 * n}
    if op == "weight_grad":
        outs, ins = case["outs"], case["ins"]
        packed = rows * (-(-ins // BLOCK)) * (BLOCK + 1)
        return {"bytes": 2 * rows * outs + packed + outs * ins * e, "flops": 2 * rows * outs * ins}
    n = rows * case["experts"]
    return {"bytes": 2 * n * e + (rows if case["masked"] else 0) + 8 * case["experts"], "flops": 12 * n}


# ------------------------------------------------------------------ inputs

def _gen(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def _normal(g, *shape):
    return torch.randn(*shape, generator=g, device="cuda", dtype=torch.float32)


def _activations(g, rows, cols, dtype, extra=0):
    """Hidden states: a channel-dependent size and offset, a few large channels."""
    size = (1 + 0.5 * _normal(g, cols).abs()) * (1 + 15 * (torch.rand(cols, generator=g, device="cuda") < 0.003))
    wide = torch.zeros(rows, cols + extra, device="cuda", dtype=DTYPES[dtype])
    wide[:, :cols] = _normal(g, rows, cols).mul_(size).add_(0.3 * _normal(g, cols))
    return wide[:, :cols]


def _step_of(scale_byte):
    """2^(byte - 127) as fp32, NaN for byte 255."""
    step = (scale_byte.to(torch.int32) << 23).view(torch.float32)
    return torch.where(scale_byte == 255, float("nan"), step)


def _pack(x):
    """(q int8 [rows, padded], scale uint8 [rows, padded / 32]) of x."""
    rows, cols = x.shape
    blocks = -(-cols // BLOCK)
    v = torch.zeros(rows, blocks * BLOCK, device=x.device, dtype=torch.float32)
    v[:, :cols] = x.float()
    v = v.view(rows, blocks, BLOCK)
    top = v.abs().amax(-1)
    fine = torch.isfinite(top)
    exponent = (torch.where(fine, top, 0).view(torch.int32) >> 23) - 127  # floor(log2(top))
    byte = (exponent - 6 + 127).clamp(min=1)
    inverse = ((254 - byte) << 23).view(torch.float32)
    q = torch.round(v * inverse[..., None]).clamp(-127, 127)
    q = torch.where(fine[..., None], q, 0).to(torch.int8)
    return q.view(rows, blocks * BLOCK), torch.where(fine, byte, 255).to(torch.uint8)


def _unpack(q, scale, cols):
    rows = q.shape[0]
    v = q.view(rows, -1, BLOCK).float() * _step_of(scale)[..., None]
    return v.view(rows, -1)[:, :cols]


def prepare(case, seed):
    g = _gen(seed)
    op, rows = case["op"], case["rows"]
    s = dict(case)
    if op in ("norm_forward", "norm_backward", "checkpoint"):
        cols, dt = case["cols"], DTYPES[case["dtype"]]
        s["x"] = _activations(g, rows, cols, case["dtype"], case["extra"])
        if op != "checkpoint":
            s["weight"] = (1 + 0.1 * _normal(g, cols)).to(dt)
            s["bias"] = (0.1 * _normal(g, cols)).to(dt)
        if op == "norm_backward":
            x = s["x"].double() if rows * cols < 1 << 24 else s["x"].float()
            s["mean"] = x.mean(1).float()
            s["rstd"] = torch.rsqrt(x.var(1, unbiased=False) + EPS).float()
            del x
            s["dy"] = (1e-2 * _normal(g, rows, cols)).to(dt)
            if case["checkpoint"]:
                s["q"], s["scale"] = _pack(s.pop("x"))
    elif op == "weight_grad":
        s["q"], s["scale"] = _pack(_activations(g, rows, case["ins"], "bf16"))
        s["dy"] = (1e-2 * _normal(g, rows, case["outs"])).to(torch.bfloat16)
    else:
        experts = case["experts"]
        logits = 1.5 * _normal(g, rows, experts) + 0.7 * _normal(g, experts)
        s["logits"] = logits.to(DTYPES[case["dtype"]])
        s["mask"] = torch.rand(rows, generator=g, device="cuda") < 0.9 if case["masked"] else None
    return s


# --------------------------------------------------------------------- run

def _plain(s):
    op = s["op"]
    if op == "norm_forward":
        x = s["x"].float()
        mean = x.mean(1)
        centred = x - mean[:, None]
        rstd = torch.rsqrt((centred * centred).mean(1) + EPS)
        y = centred * rstd[:, None] * s["weight"].float() + s["bias"].float()
        out = [y.to(s["x"].dtype), mean, rstd]
        if s["checkpoint"]:
            out.append(_unpack(*_pack(x), s["cols"]).to(s["x"].dtype))
        return out
    if op == "norm_backward":
        x = _unpack(s["q"], s["scale"], s["cols"]) if s["checkpoint"] else s["x"].float()
        dy = s["dy"].float()
        xhat = (x - s["mean"][:, None]) * s["rstd"][:, None]
        gy = dy * s["weight"].float()
        dx = s["rstd"][:, None] * (gy - gy.mean(1, keepdim=True) - xhat * (gy * xhat).mean(1, keepdim=True))
        return [dx.to(s["dy"].dtype), (dy * xhat).sum(0), dy.sum(0)]
    if op == "checkpoint":
        return _unpack(*_pack(s["x"]), s["cols"]).to(s["x"].dtype)
    if op == "weight_grad":
        x = _unpack(s["q"], s["scale"], s["ins"])
        return (s["dy"].float().t() @ x).to(DTYPES[s["dtype"]])
    z = s["logits"].float()
    experts, k = s["experts"], s["top_k"]
    live = z.amax(1) > -math.inf
    if s["mask"] is not None:
        live = live & s["mask"]
    z = torch.where(live[:, None], z, 0)
    e = torch.exp(z - z.amax(1, keepdim=True))
    p = torch.where(live[:, None], e / e.sum(1, keepdim=True), 0)
    order = torch.sort(z, dim=1, descending=True, stable=True).indices[:, :k]  # ties: the lowest index first
    chosen = live[:, None].expand(-1, k) & (z.gather(1, order) > -math.inf)
    counts = torch.zeros(experts, dtype=torch.int64, device=z.device)
    counts.scatter_add_(0, order.reshape(-1), chosen.reshape(-1).to(torch.int64))
    rows = live.sum().clamp(min=1).float()
    load = experts * counts.float() / counts.sum().clamp(min=1).float()
    loss = (load * (p.sum(0) / rows)).sum()
    grad = p * (load - (p * load).sum(1, keepdim=True)) / rows
    return [loss, grad.to(s["logits"].dtype), counts]


def _own(s):
    from entropy_loss_gb300 import flp
    op = s["op"]
    if op == "norm_forward":
        if s["checkpoint"]:
            y, mean, rstd, kept = flp.layer_norm(s["x"], s["weight"], s["bias"], eps=EPS, checkpoint=True)
            return [y, mean, rstd, flp.checkpoint_unpack(kept)]
        return list(flp.layer_norm(s["x"], s["weight"], s["bias"], eps=EPS))
    if op == "norm_backward":
        x = flp.Checkpoint8(s["q"], s["scale"], s["cols"], s["dy"].dtype) if s["checkpoint"] else s["x"]
        return list(flp.layer_norm_backward(s["dy"], x, s["weight"], s["mean"], s["rstd"]))
    if op == "checkpoint":
        return flp.checkpoint_unpack(flp.checkpoint_pack(s["x"]))
    if op == "weight_grad":
        x = flp.Checkpoint8(s["q"], s["scale"], s["ins"], torch.bfloat16)
        return flp.checkpoint_weight_grad(s["dy"], x, dw_dtype=DTYPES[s["dtype"]])
    loss, grad, counts = flp.balance_loss(s["logits"], s["top_k"], mask=s["mask"])
    return [loss[0], grad, counts]


def run(state):
    return _own(state) if own else _plain(state)


# ------------------------------------------------------------------- exact

def _power64(e):
    """2^e in 64 bits for integers e, exactly: a step that is off by one bit would break ties another way."""
    return ((e.long() + 1023) << 52).view(torch.float64)


def _blocks64(x):
    """The values an 8-bit checkpoint of x (64-bit) stands for, block by block from the definition."""
    rows, cols = x.shape
    pad = -cols % BLOCK
    b = torch.nn.functional.pad(x, (0, pad)).reshape(rows, -1, BLOCK)
    _, e = torch.frexp(b.abs().amax(-1, keepdim=True))       # top = m 2^e, 1/2 <= m < 1
    step = _power64((e - 7).clamp(min=-126))
    kept = torch.round(b / step).clamp(-127, 127) * step
    return kept.reshape(rows, cols + pad)[:, :cols]


def _kept64(s, cols):
    exponent = s["scale"].long().repeat_interleave(BLOCK, dim=1)[:, :cols] - 127
    return s["q"][:, :cols].double() * _power64(exponent)


def exact(case, seed):
    s = prepare(case, seed)
    op = s["op"]
    if op == "checkpoint":
        return _blocks64(s["x"].double())
    if op == "norm_forward":
        x = s["x"].double()
        var, mean = torch.var_mean(x, dim=1, unbiased=False)
        rstd = 1 / torch.sqrt(var + EPS)
        y = torch.addcmul(s["bias"].double(), (x - mean[:, None]) / torch.sqrt(var + EPS)[:, None], s["weight"].double())
        return [y, mean, rstd] + ([_blocks64(x)] if s["checkpoint"] else [])
    if op == "norm_backward":
        x = _kept64(s, s["cols"]) if s["checkpoint"] else s["x"].double()
        dy, n, rstd = s["dy"].double(), s["cols"], s["rstd"].double()[:, None]
        xhat = (x - s["mean"].double()[:, None]) * rstd
        del x
        a = dy * s["weight"].double()
        along, level = torch.einsum("mh,mh->m", a, xhat)[:, None] / n, a.sum(1, keepdim=True) / n
        db, dw = dy.sum(0), torch.einsum("mh,mh->h", dy, xhat)
        return [(a - level - xhat * along) * rstd, dw, db]
    if op == "weight_grad":
        return torch.einsum("mn,mk->nk", s["dy"].double(), _kept64(s, s["ins"]))
    z, k, experts = s["logits"].double(), s["top_k"], s["experts"]
    keep = torch.ones(s["rows"], dtype=torch.bool, device=z.device) if s["mask"] is None else s["mask"]
    keep = keep & (z > -math.inf).any(1)
    if not bool(keep.any()):
        return [torch.zeros((), dtype=torch.float64, device=z.device), torch.zeros_like(z), None]
    zk = z[keep]
    p = torch.softmax(zk, 1)
    # an expert is chosen if fewer than k experts come before it: larger logits, or equal ones of a lower index
    rank = torch.argsort(torch.argsort(-zk, dim=1, stable=True), dim=1)
    c = ((rank < k) & (zk > -math.inf)).double().sum(0)
    f, n = c / c.sum(), zk.shape[0]
    loss = experts * (f * p.mean(0)).sum()
    grad = torch.zeros_like(z)
    grad[keep] = experts / n * p * (f - (p @ f)[:, None])
    return [loss, grad, None]
