"""Plain 64-bit implementations of the training-step operators, written from
their formulas for the tests (numpy and torch on the CPU, no library code)."""
import numpy as np
import torch

BLOCK = 32


def norm_forward(x, w, b, eps):
    """x float64 [M, H] -> (y, mean, rstd)."""
    mean = x.mean(1)
    c = x - mean[:, None]
    rstd = 1 / np.sqrt((c * c).mean(1) + eps)
    y = c * rstd[:, None]
    if w is not None:
        y = y * w
    if b is not None:
        y = y + b
    return y, mean, rstd


def norm_backward(dy, x, w, mean, rstd):
    H = x.shape[1]
    xh = (x - mean[:, None]) * rstd[:, None]
    g = dy if w is None else dy * w
    dx = rstd[:, None] * (g - g.sum(1, keepdims=True) / H - xh * (g * xh).sum(1, keepdims=True) / H)
    return dx, (dy * xh).sum(0), dy.sum(0)


def pack(x):
    """x float32 or float64 numpy [M, H] -> (q int8 [M, Hp], scale uint8 [M, Hp / 32])."""
    M, H = x.shape
    nb = -(-H // BLOCK)
    v = np.zeros((M, nb * BLOCK))
    v[:, :H] = x
    v = v.reshape(M, nb, BLOCK)
    q = np.zeros(v.shape, np.int8)
    scale = np.zeros((M, nb), np.uint8)
    for i in range(M):
        for j in range(nb):
            blk = v[i, j]
            if not np.all(np.isfinite(blk)):
                scale[i, j] = 255
                continue
            top = np.max(np.abs(blk))
            e = -126 if top == 0 else max(int(np.frexp(top)[1]) - 1 - 6, -126)
            scale[i, j] = e + 127
            q[i, j] = np.clip(np.rint(np.ldexp(blk, -e)), -127, 127).astype(np.int8)
    return q.reshape(M, nb * BLOCK), scale


def unpack(q, scale, H):
    M = q.shape[0]
    with np.errstate(over="ignore"):
        step = np.where(scale == 255, np.nan, np.ldexp(1.0, scale.astype(np.int64) - 127))
    return (q.reshape(M, scale.shape[1], BLOCK).astype(np.float64) * step[:, :, None]).reshape(q.shape)[:, :H]


def balance(z, k, coef=1.0, mask=None, experts=None):
    """z float64 [T, E] -> (loss, grad, counts, a, p, n, live)."""
    T, E = z.shape
    keep = np.ones(T, bool) if mask is None else np.asarray(mask)
    counts = np.zeros(E, np.int64)
    p = np.zeros((T, E))
    live = np.zeros(T, bool)
    for t in range(T):
        if not keep[t] or np.all(z[t] == -np.inf):
            continue
        live[t] = True
        odd = bool(np.any(np.isnan(z[t])) or np.any(z[t] == np.inf))
        if odd:
            p[t] = np.nan
        else:
            e = np.exp(z[t] - z[t].max())
            p[t] = e / e.sum()
        if experts is not None:
            for e in experts[t]:
                if 0 <= e < E:
                    counts[e] += 1
        elif not odd:
            order = sorted(range(E), key=lambda j: (-z[t, j], j))[:k]
            for j in order:
                if z[t, j] > -np.inf:
                    counts[j] += 1
    n, c = int(live.sum()), int(counts.sum())
    if n == 0 or c == 0:
        return 0.0, np.zeros((T, E)), counts, np.zeros(E), p, n, live
    a = (E * counts - c) / c
    loss = coef * E * np.sum(counts / c * (p[live].sum(0) / n))
    grad = np.zeros((T, E))
    # E c_e / C less 1 (sum p = 1): an even load's gradient is 0, not the rounding of 1 - sum p
    grad[live] = coef / n * p[live] * (a - (p[live] * a).sum(1, keepdims=True))
    return loss, grad, counts, a, p, n, live


def rows_of(M, H, dtype, device, pitch=0, offset=0, gen=None, scale=1.0):
    """A [M, H] view with the given extra pitch and element offset, filled with normals."""
    buf = torch.zeros(M * (H + pitch) + offset + 64, dtype=dtype, device=device)
    view = buf[offset:offset + M * (H + pitch)].view(M, H + pitch)[:, :H] if M else buf[:0].view(0, H)
    view.copy_((scale * torch.randn(M, H, generator=gen)).to(dtype))
    return view
