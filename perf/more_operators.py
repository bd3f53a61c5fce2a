"""Cases of the operators for mixtures of experts, linear layers and given logits, and their plain forms.

Operators: tokens sorted by expert and their rows brought there (dispatch) and
back with weights (combine), each with its gradient; a linear layer with bias,
activation and residual in its epilogue, with its gradients; log-probabilities
of given tokens from logits, with entropy and top alternatives, and the gradient
by the logits.

``run`` computes the plain form (elementary torch operations in 32 bits) or,
with ``own`` set, calls the framework's operators; ``exact`` computes the same
outputs from the definitions in 64 bits.
"""
import math

import torch

own = False

IGNORE = -100
DTYPES = {"bf16": torch.bfloat16, "fp32": torch.float32}
ACTIVATIONS = [None, "relu", "gelu", "gelu_tanh", "silu"]
CHUNK = 1 << 27       # logits that the plain and exact forms hold in a wide type at a time


# ------------------------------------------------------------------- cases

def listed():
    return [
        # a few decoded tokens on their way to the experts: launch latency
        dict(name="dispatch_decode", op="dispatch", tokens=16, experts=8, top_k=2, width=4096, dtype="bf16", dropped=False),
        # a global batch through a wide router
        dict(name="dispatch_large", op="dispatch", tokens=65536, experts=256, top_k=8, width=2048, dtype="bf16", dropped=False),
        # odd sizes in full precision, some slots over the experts' capacity (a small research model)
        dict(name="combine_odd", op="combine", tokens=777, experts=12, top_k=3, width=2047, dtype="fp32", dropped=True),
        # the backward pass of a large micro-batch
        dict(name="combine_backward_large", op="combine_backward", tokens=32768, experts=64, top_k=4, width=5120, dtype="bf16",
             dropped=True),
        # one decoded token through the first half of a feed-forward block
        dict(name="linear_one_token", op="linear", rows=1, ins=4096, outs=16384, activation="silu", bias=False, residual=False,
             keep=False),
        # a short ragged batch, odd output width, into the residual stream
        dict(name="linear_ragged", op="linear", rows=777, ins=1000, outs=2047, activation="gelu", bias=True, residual=True,
             keep=False),
        # a training micro-batch through the first half of a feed-forward block, ready for the backward pass
        dict(name="linear_large", op="linear", rows=8192, ins=4096, outs=16384, activation="gelu_tanh", bias=True, residual=False,
             keep=True),
        # the backward pass of an ordinary micro-batch: all three gradients through the activation
        dict(name="linear_backward_large", op="linear_backward", rows=8192, ins=5120, outs=8192, activation="gelu_tanh", bias=True,
             dtype="bf16"),
        # one decoded token: its log-probability and the alternatives that a server shows
        dict(name="logprob_one_token", op="logprob", rows=1, vocab=151936, dtype="bf16", extra=0, top=20, scale=1.25, masked=False),
        # a short batch in full precision, rows cut out of wider ones, banned tokens at minus infinity
        dict(name="logprob_odd", op="logprob", rows=300, vocab=50257, dtype="fp32", extra=3, top=5, scale=1.0, masked=True),
        # a rollout scored in one pass
        dict(name="logprob_large", op="logprob", rows=8192, vocab=131072, dtype="bf16", extra=0, top=8, scale=1.0, masked=False),
        # the gradient by the logits of a training micro-batch
        dict(name="logprob_backward_large", op="logprob_backward", rows=4096, vocab=152064, dtype="bf16", extra=0, scale=1.25,
             masked=False),
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def _width(rng, lo, hi):
    """A width: multiples of 64 as models have them, or any number."""
    w = _log(rng, lo, hi)
    return max(64, w // 64 * 64) if rng.random() < 0.6 else w


def draw(rng):
    op = rng.choice(["dispatch", "dispatch_backward", "combine", "combine_backward", "linear", "linear", "linear_backward",
                     "logprob", "logprob", "logprob_backward"])
    dtype = rng.choice(["bf16", "fp32"])
    e = _size(dtype)
    if op in ("linear", "linear_backward"):
        ins, outs = _width(rng, 64, 8192), _width(rng, 64, 8192)
        rows = _log(rng, 1, min(8192, 8192 * 8192 * 5120 // (ins * outs)))
        c = dict(op=op, rows=rows, ins=ins, outs=outs, activation=rng.choice(ACTIVATIONS), bias=rng.random() < 0.6)
        if op == "linear":
            c.update(residual=rng.random() < 0.5, keep=c["activation"] is not None and rng.random() < 0.5)
        else:
            c.update(dtype=dtype)
        return c
    if op in ("logprob", "logprob_backward"):
        vocab = _log(rng, 1000, 202048)
        rows = _log(rng, 1, min(16384, (1 << 29) // (vocab * e // 2)))
        c = dict(op=op, rows=rows, vocab=vocab, dtype=dtype, extra=rng.choice([0, 0, 0, 8, 3]), scale=rng.choice([1.0, 0.75, 1.25]),
                 masked=rng.random() < 0.4)
        if op == "logprob":
            c["top"] = rng.choice([0, 1, 2, 5, 8, 20])
        return c
    experts = _log(rng, 2, 256)
    top_k = rng.randint(1, min(8, experts))
    width = _width(rng, 32, 8192)
    tokens = _log(rng, 1, min(65536, (1 << 29) // (top_k * width * e // 2)))
    return dict(op=op, tokens=tokens, experts=experts, top_k=top_k, width=width, dtype=dtype, dropped=rng.random() < 0.5)


def _size(dtype):
    return 2 if dtype == "bf16" else 4


def work(case):
    op = case["op"]
    if op in ("linear", "linear_backward"):
        rows, ins, outs = case["rows"], case["ins"], case["outs"]
        n = rows * outs
        if op == "linear":
            full = 1 + case["residual"] + case["keep"]
            return {"bytes": 2 * (rows * ins + ins * outs + full * n + case["bias"] * outs), "flops": 2 * rows * ins * outs}
        read = n * (2 if case["activation"] else 1) + rows * ins + ins * outs
        written = 2 * rows * ins + _size(case["dtype"]) * ins * outs + (4 * outs if case["bias"] else 0)
        return {"bytes": 2 * read + written, "flops": 4 * rows * ins * outs}
    if op in ("logprob", "logprob_backward"):
        rows = case["rows"]
        n = rows * case["vocab"]
        if op == "logprob":
            return {"bytes": n * _size(case["dtype"]) + rows * (8 + 12 + 12 * case["top"]), "flops": 6 * n}
        return {"bytes": 2 * n * _size(case["dtype"]) + 24 * rows, "flops": 8 * n}
    tokens, slots, e = case["tokens"], case["tokens"] * case["top_k"], _size(case["dtype"])
    one, many = tokens * case["width"] * e, slots * case["width"] * e
    if op == "dispatch":  # choices read; positions, slots, counts and offsets written
        return {"bytes": one + many + 16 * slots + 16 * case["experts"] + 8, "flops": 0}
    if op == "dispatch_backward":
        return {"bytes": one + many + 4 * slots, "flops": slots * case["width"]}
    if op == "combine":
        return {"bytes": one + many + 8 * slots, "flops": 2 * slots * case["width"]}
    return {"bytes": one + 2 * many + 12 * slots, "flops": 3 * slots * case["width"]}


# ------------------------------------------------------------------ inputs

def _gen(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def _normal(g, *shape):
    return torch.randn(*shape, generator=g, device="cuda", dtype=torch.float32)


def _hidden(g, rows, cols, dtype):
    """Hidden states: a channel-dependent size, a few large channels."""
    size = (1 + 0.5 * _normal(g, cols).abs()) * (1 + 7 * (torch.rand(cols, generator=g, device="cuda") < 0.003))
    return (_normal(g, rows, cols) * size).to(dtype)


def _parts(rows, cols):
    step = max(1, CHUNK // cols)
    return [slice(i, min(rows, i + step)) for i in range(0, rows, step)]


def _order(experts, n):
    """Tokens' slots sorted by expert, slots without one last: (position of each slot,
    slot at each position, tokens of each expert, where each expert begins)."""
    flat = experts.reshape(-1)
    key = torch.where((flat >= 0) & (flat < n), flat, n)
    slots = torch.sort(key, stable=True).indices
    rows = torch.empty_like(slots)
    rows[slots] = torch.arange(len(slots), device=slots.device)
    counts = torch.zeros(n + 1, dtype=torch.int64, device=slots.device).scatter_add_(0, key, torch.ones_like(key))[:n]
    offsets = torch.zeros(n + 1, dtype=torch.int64, device=slots.device)
    offsets[1:] = torch.cumsum(counts, 0)
    return rows.view(experts.shape).to(torch.int32), slots.to(torch.int32), counts, offsets


def prepare(case, seed):
    g = _gen(seed)
    op = case["op"]
    s = dict(case)
    if op in ("linear", "linear_backward"):
        rows, ins, outs = case["rows"], case["ins"], case["outs"]
        s["x"] = _hidden(g, rows, ins, torch.bfloat16)
        s["W"] = (_normal(g, outs, ins) / ins ** 0.5).to(torch.bfloat16)
        s["b"] = (0.2 * _normal(g, outs)).to(torch.bfloat16) if case["bias"] else None
        if op == "linear":
            s["r"] = _hidden(g, rows, outs, torch.bfloat16) if case["residual"] else None
        else:
            s["dy"] = (1e-2 * _normal(g, rows, outs)).to(torch.bfloat16)
            s["pre"] = (1.5 * _normal(g, rows, outs)).to(torch.bfloat16) if case["activation"] else None
        return s
    if op in ("logprob", "logprob_backward"):
        rows, vocab, dt = case["rows"], case["vocab"], DTYPES[case["dtype"]]
        wide = torch.zeros(rows, vocab + case["extra"], device="cuda", dtype=dt)
        common = 1.5 * _normal(g, vocab)
        allowed = vocab - vocab // 16 if case["masked"] else vocab
        for part in _parts(rows, vocab):
            wide[part, :vocab] = _normal(g, part.stop - part.start, vocab).mul_(2).add_(common).to(dt)
        if case["masked"]:
            wide[:, allowed:vocab] = -math.inf
        s["logits"] = wide[:, :vocab]
        y = torch.randint(0, allowed, (rows,), generator=g, device="cuda")
        s["y"] = torch.where(torch.rand(rows, generator=g, device="cuda") < 0.06, IGNORE, y)
        if op == "logprob_backward":
            s["lse"], s["entropy"] = torch.empty(rows, device="cuda"), torch.empty(rows, device="cuda")
            for part in _parts(rows, vocab):
                lse, ent = _statistics(s["logits"][part].float() * case["scale"])
                s["lse"][part], s["entropy"][part] = lse, torch.where(s["y"][part] == IGNORE, 0, ent)
            s["g_lp"] = -torch.rand(rows, generator=g, device="cuda") / rows
            s["g_ent"] = 0.01 * _normal(g, rows) / rows
        return s
    tokens, experts, top_k, width, dt = case["tokens"], case["experts"], case["top_k"], case["width"], DTYPES[case["dtype"]]
    score = _normal(g, tokens, experts) + 0.7 * _normal(g, experts)
    top = torch.topk(score, top_k, dim=1)
    s["choice"] = top.indices
    if case["dropped"]:  # slots over the experts' capacity
        s["choice"] = torch.where(torch.rand(tokens, top_k, generator=g, device="cuda") < 0.04, -1, s["choice"])
    if op == "dispatch":
        s["x"] = _hidden(g, tokens, width, dt)
        return s
    s["weights"] = torch.softmax(top.values, 1)
    s["rows"], s["slots"], s["counts"], s["offsets"] = _order(s["choice"], experts)
    if op == "dispatch_backward":
        s["dxs"] = (1e-2 * _normal(g, tokens * top_k, width)).to(dt)
        return s
    s["ys"] = _hidden(g, tokens * top_k, width, dt)
    if op == "combine_backward":
        s["dy"] = (1e-2 * _normal(g, tokens, width)).to(dt)
    return s


# --------------------------------------------------------------------- run

def _act(v, kind):
    if kind == "relu":
        return v.clamp(min=0)
    if kind == "gelu":
        return 0.5 * v * (1 + torch.erf(v * 0.5 ** 0.5))
    if kind == "gelu_tanh":
        return 0.5 * v * (1 + torch.tanh((2 / math.pi) ** 0.5 * (v + 0.044715 * v * v * v)))
    if kind == "silu":
        return v / (1 + torch.exp(-v))
    return v


def _slope(v, kind):
    if kind == "relu":
        return (v > 0).float()
    if kind == "gelu":
        return 0.5 * (1 + torch.erf(v * 0.5 ** 0.5)) + v * torch.exp(-0.5 * v * v) / (2 * math.pi) ** 0.5
    if kind == "gelu_tanh":
        c = (2 / math.pi) ** 0.5
        t = torch.tanh(c * (v + 0.044715 * v * v * v))
        return 0.5 * (1 + t) + 0.5 * v * (1 - t * t) * c * (1 + 3 * 0.044715 * v * v)
    p = 1 / (1 + torch.exp(-v))
    return p * (1 + v * (1 - p))


def _statistics(z):
    """(log-sum-exp, entropy) of rows of scaled logits."""
    top = z.amax(1, keepdim=True)
    e = torch.exp(z - top)
    total = e.sum(1)
    lse = top[:, 0] + torch.log(total)
    mean = (e * torch.where(e > 0, z, 0)).sum(1) / total
    return lse, lse - mean


def _first(z, k):
    """Columns of the k largest values of each row, equal ones by their column."""
    bits = torch.where(z == 0, 0.0, z).view(torch.int32).long()
    rank = torch.where(bits < 0, -(bits & 0x7FFFFFFF), bits)
    key = (rank << 32) + (z.shape[1] - 1 - torch.arange(z.shape[1], device=z.device))
    return z.shape[1] - 1 - (torch.topk(key, k, dim=1, sorted=True).values & 0xFFFFFFFF)


def _plain_logprob(s):
    rows, top = s["rows"], s["top"]
    out = [torch.empty(rows, device="cuda") for _ in range(3)]
    if top:
        out += [torch.empty(rows, top, device="cuda"), torch.empty(rows, top, device="cuda", dtype=torch.int64)]
    for part in _parts(rows, s["vocab"]):
        raw = s["logits"][part].float()
        z, y = raw * s["scale"], s["y"][part]
        lse, ent = _statistics(z)
        skip = y == IGNORE
        picked = z.gather(1, torch.where(skip, 0, y)[:, None])[:, 0]
        out[0][part], out[1][part], out[2][part] = torch.where(skip, 0, picked - lse), lse, torch.where(skip, 0, ent)
        if top:
            at = _first(raw, top)
            out[3][part], out[4][part] = z.gather(1, at) - lse[:, None], at
    return out


def _plain_logprob_backward(s):
    logits = s["logits"]
    grad = torch.empty(logits.shape, dtype=logits.dtype, device="cuda")
    for part in _parts(s["rows"], s["vocab"]):
        z, y, lse = logits[part].float() * s["scale"], s["y"][part], s["lse"][part, None]
        live = (y != IGNORE).float()[:, None]
        g_lp, g_ent = s["g_lp"][part, None] * live, s["g_ent"][part, None] * live
        p = torch.exp(z - lse)
        away = torch.where(p > 0, lse - s["entropy"][part, None] - z, 0)
        hit = (torch.arange(z.shape[1], device="cuda") == y[:, None]).float()
        grad[part] = (s["scale"] * (g_lp * (hit - p) + g_ent * p * away)).to(logits.dtype)
    return grad


def _plain_expert(s):
    op, k, tokens = s["op"], s["top_k"], s["tokens"]
    if op == "dispatch":
        rows, slots, counts, offsets = _order(s["choice"], s["experts"])
        xs = s["x"][slots.long() // k]
        kept = torch.arange(tokens * k, device="cuda") < offsets[-1]
        return [torch.where(kept[:, None], xs, 0), rows, slots, counts, offsets]
    rows = s["rows"].long()
    live = (rows < s["offsets"][-1]).float()
    if op == "combine_backward":
        dy = s["dy"].float()
        dys = torch.empty_like(s["ys"])
        dw = torch.empty(tokens, k, device="cuda")
        for j in range(k):
            dys[rows[:, j]] = (dy * (s["weights"][:, j] * live[:, j])[:, None]).to(dys.dtype)
            dw[:, j] = (dy * s["ys"][rows[:, j]].float()).sum(1) * live[:, j]
        return [dys, dw]
    many = s["ys"] if op == "combine" else s["dxs"]
    total = torch.zeros(tokens, s["width"], device="cuda")
    for j in range(k):
        w = s["weights"][:, j] * live[:, j] if op == "combine" else live[:, j]
        total += w[:, None] * many[rows[:, j]].float()
    return total.to(many.dtype)


def _plain(s):
    op = s["op"]
    if op == "linear":
        pre = s["x"].float() @ s["W"].float().t()
        if s["b"] is not None:
            pre += s["b"].float()
        y = _act(pre, s["activation"])
        if s["r"] is not None:
            y = y + s["r"].float()
        y = y.to(torch.bfloat16)
        return [y, pre.to(torch.bfloat16)] if s["keep"] else y
    if op == "linear_backward":
        d = s["dy"].float()
        if s["activation"]:
            d = d * _slope(s["pre"].float(), s["activation"])
        out = [(d @ s["W"].float()).to(torch.bfloat16), (d.t() @ s["x"].float()).to(DTYPES[s["dtype"]])]
        return out + [d.sum(0)] if s["bias"] else out
    if op == "logprob":
        return _plain_logprob(s)
    if op == "logprob_backward":
        return _plain_logprob_backward(s)
    return _plain_expert(s)


def _own(s):
    from entropy_loss_gb300 import flp
    op = s["op"]
    if op == "linear":
        out = flp.linear(s["x"], s["W"], s["b"], activation=s["activation"], residual=s["r"], keep=s["keep"])
        return list(out) if s["keep"] else out
    if op == "linear_backward":
        dx, dW, db = flp.linear_backward(s["dy"], s["x"], s["W"], s["pre"], activation=s["activation"],
                                         dw_dtype=DTYPES[s["dtype"]], want_dbias=s["bias"])
        return [dx, dW, db] if s["bias"] else [dx, dW]
    if op == "logprob":
        out = flp.token_logprob(s["logits"], s["y"], top=s["top"], scale=s["scale"], ignore_index=IGNORE)
        return list(out) if s["top"] else list(out[:3])
    if op == "logprob_backward":
        return flp.token_logprob_backward(s["logits"], s["y"], s["lse"], s["entropy"], s["g_lp"], s["g_ent"], scale=s["scale"],
                                          ignore_index=IGNORE)
    if op == "dispatch":
        order = flp.expert_sort(s["choice"], s["experts"])
        return [flp.expert_gather(s["x"], order), order.rows, order.slots, order.counts, order.offsets]
    order = flp.ExpertOrder(s["rows"], s["slots"], s["counts"], s["offsets"])
    if op == "combine":
        return flp.expert_combine(s["ys"], order, s["weights"])
    if op == "dispatch_backward":
        return flp.expert_combine(s["dxs"], order)
    return list(flp.expert_combine_backward(s["dy"], s["ys"], order, s["weights"]))


def run(state):
    return _own(state) if own else _plain(state)


# ------------------------------------------------------------------- exact

def _act64(v, kind):
    """(activation, slope) in 64 bits."""
    if kind is None:
        return v, torch.ones_like(v)
    if kind == "relu":
        return torch.relu(v), (v > 0).double()
    if kind == "gelu":
        phi = torch.special.ndtr(v)
        return v * phi, phi + v * torch.exp(-v * v / 2) / math.sqrt(2 * math.pi)
    # both are v sigmoid(u)
    if kind == "silu":
        u, du = v, torch.ones_like(v)
    else:
        c = math.sqrt(8 / math.pi)
        u, du = c * (v + 0.044715 * v ** 3), c * (1 + 0.134145 * v ** 2)
    p = torch.sigmoid(u)
    return v * p, p + v * p * torch.sigmoid(-u) * du


def _exact_logits(s, op):
    out = []
    for part in _parts(s["rows"], 2 * s["vocab"]):
        z, y = s["logits"][part].double() * s["scale"], s["y"][part]
        live = y != IGNORE
        if op == "logprob":
            logp = torch.log_softmax(z, 1)
            lse = torch.logsumexp(z, 1)
            ent = torch.special.entr(torch.exp(logp)).sum(1)
            lp = logp[torch.arange(len(y), device=y.device), y.clamp(min=0)]
            out.append([torch.where(live, lp, 0), lse, torch.where(live, ent, 0)]
                       + ([torch.topk(logp, s["top"], dim=1).values] if s["top"] else []))
        else:
            away = z - s["lse"][part].double()[:, None]          # log p
            p = torch.exp(away)
            a, b = s["g_lp"][part].double()[:, None], s["g_ent"][part].double()[:, None]
            grad = -p * (a + b * torch.where(p > 0, away + s["entropy"][part].double()[:, None], 0))
            grad[live, y[live]] += a[live, 0]
            out.append([s["scale"] * grad * live[:, None]])
    whole = [torch.cat(c) for c in zip(*out)]
    if op == "logprob_backward":
        return whole[0]
    return whole + ([None] if s["top"] else [])


def exact(case, seed):
    s = prepare(case, seed)
    op = s["op"]
    if op == "linear":
        pre = torch.einsum("mk,nk->mn", s["x"].double(), s["W"].double())
        pre = pre if s["b"] is None else pre + s["b"].double()
        y = _act64(pre, s["activation"])[0]
        y = y if s["r"] is None else y + s["r"].double()
        return [y, pre] if s["keep"] else y
    if op == "linear_backward":
        d = s["dy"].double()
        if s["activation"]:
            d = d * _act64(s["pre"].double(), s["activation"])[1]
        out = [torch.einsum("mn,nk->mk", d, s["W"].double()), torch.einsum("mn,mk->nk", d, s["x"].double())]
        return out + [torch.einsum("mn->n", d)] if s["bias"] else out
    if op in ("logprob", "logprob_backward"):
        return _exact_logits(s, op)
    tokens, k, n = s["tokens"], s["top_k"], s["experts"]
    # a slot's row: how many slots come before it, by expert and then by slot
    choice = s["choice"].reshape(-1)
    inside = (choice >= 0) & (choice < n)
    live = torch.nonzero(inside)[:, 0]
    source = live[torch.argsort(choice[live] * (tokens * k) + live)]  # slot of each row that holds a token
    token, total = source // k, len(source)
    if op == "dispatch":
        xs = torch.zeros(tokens * k, s["width"], dtype=torch.float64, device="cuda")
        xs[:total] = s["x"].double()[token]
        return [xs, None, None, None, None]
    w = s["weights"].double().reshape(-1)[source]
    if op == "combine_backward":
        dy, ys = s["dy"].double()[token], s["ys"][:total].double()
        dw = torch.zeros(tokens * k, dtype=torch.float64, device="cuda")
        dw[source] = torch.einsum("ph,ph->p", dy, ys)
        dys = torch.zeros(tokens * k, s["width"], dtype=torch.float64, device="cuda")
        dys[:total] = dy.mul_(w[:, None])
        return [dys, dw.view(tokens, k)]
    many = s["ys"][:total].double() * w[:, None] if op == "combine" else s["dxs"][:total].double()
    return torch.zeros(tokens, s["width"], dtype=torch.float64, device="cuda").index_add_(0, token, many)
