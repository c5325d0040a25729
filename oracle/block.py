"""The layer around the experts in fp64: residual addition and root-mean-square
norm, routing, tokens in expert order and back, and the gradients -- TEST
INFRASTRUCTURE ONLY (see oracle/__init__).

The pages (arXiv 2607.15810, section 3) take the layer's input and its routes as
given; these are the forms that an MoE layer commonly has.  Conventions:
  * h = x + residual is formed in fp32 and rounded to the residual's type;
  * experts rank by logit, equal logits by lower index; a masked expert (-inf)
    has weight 0, and a token with nothing else has weights 0 and no gradient;
  * a slot whose position is outside [0, rows) is left out.
"""

import numpy as np

from . import mx


def bf16_round(v):
    """fp32 (or exactly held) values rounded to the nearest bf16, ties to even, as fp64."""
    f = np.asarray(v, np.float32)
    b = f.view(np.uint32).astype(np.uint64)
    up = (b + 0x7FFF + ((b >> 16) & 1)) >> 16 << 16
    up = np.where(np.isnan(f), 0x7FC00000, up).astype(np.uint32)
    return up.view(np.float32).astype(np.float64)


def add(x, residual, bf16):
    """h of exactly held x and residual; bf16: the residual's type."""
    s = np.asarray(x, np.float32) + np.asarray(residual, np.float32)
    return bf16_round(s) if bf16 else s.astype(np.float64)


def rmsnorm(h, weight, eps):
    """(y, r) of rows h [T, H]: y = h r w, r = 1 / sqrt(mean h^2 + eps) [T, 1]."""
    h = np.asarray(h, np.float64)
    r = 1.0 / np.sqrt((h * h).mean(axis=1, keepdims=True) + eps)
    return h * r * (1.0 if weight is None else np.asarray(weight, np.float64)), r


def rmsnorm_mx(h, weight, eps):
    """(codes, scale bytes) of the norm's exact output in MX FP8."""
    return mx.quantize(rmsnorm(h, weight, eps)[0], "fp8")


def rmsnorm_grad(g, h, weight, eps, g_sum=None):
    """(dh, dweight) of sum(g y) + sum(g_sum h)."""
    g, h = np.asarray(g, np.float64), np.asarray(h, np.float64)
    w = 1.0 if weight is None else np.asarray(weight, np.float64)
    r = rmsnorm(h, None, eps)[1]
    n = h * r
    dh = r * (w * g - n * (n * w * g).mean(axis=1, keepdims=True))
    if g_sum is not None:
        dh = dh + np.asarray(g_sum, np.float64)
    return dh, (g * n).sum(axis=0)


def softmax(z):
    """p [T, E]; 0 where masked, and in a row with nothing else."""
    z = np.asarray(z, np.float64)
    m = z.max(axis=1, keepdims=True)
    e = np.exp(z - np.where(np.isneginf(m), 0.0, m))
    s = e.sum(axis=1, keepdims=True)
    return e / np.where(s == 0, 1.0, s)


def route(z, topk, renorm):
    """(ids int32, w) [T, topk]."""
    z = np.asarray(z, np.float64)
    ids = np.argsort(-z, axis=1, kind="stable")[:, :topk]
    w = np.take_along_axis(softmax(z), ids, axis=1)
    if renorm:
        w = softmax(np.take_along_axis(z, ids, axis=1))
    return ids.astype(np.int32), w


def route_grad(z, ids, g, renorm):
    """d(sum g w) / dz for the given ids."""
    z, g = np.asarray(z, np.float64), np.asarray(g, np.float64)
    ids = np.asarray(ids, np.int64)
    p = softmax(z)
    w = np.take_along_axis(p, ids, axis=1)
    if renorm:
        w = softmax(np.take_along_axis(z, ids, axis=1))
    a = g * w
    total = a.sum(axis=1, keepdims=True)
    out = np.zeros_like(p) if renorm else -p * total
    for t in range(z.shape[0]):
        for i, e in enumerate(ids[t]):
            out[t, e] += a[t, i] - (w[t, i] * total[t, 0] if renorm else 0.0)
    return out


def _slots(pos, topk, rows):
    pos = np.asarray(pos, np.int64).reshape(-1, topk)
    return [(t, s, int(pos[t, s])) for t in range(pos.shape[0]) for s in range(topk)
            if 0 <= pos[t, s] < rows]


def sort(x, pos, topk, rows, fill=0.0):
    """[rows, H]: row pos[t, s] is x[t]; `fill` where no slot points."""
    x = np.asarray(x, np.float64)
    out = np.full((rows, x.shape[1]), fill)
    for t, _, p in _slots(pos, topk, rows):
        out[p] = x[t]
    return out


def unsort(y, pos, topk, w=None):
    """(out [T, H], sum |w y|) in slot order."""
    y = np.asarray(y, np.float64)
    out = np.zeros((np.asarray(pos).size // topk, y.shape[1]))
    size = np.zeros_like(out)
    for t, s, p in _slots(pos, topk, y.shape[0]):
        v = y[p] * (1.0 if w is None else float(w[t, s]))
        out[t] += v
        size[t] += np.abs(v)
    return out, size


def unsort_grad(g, y, pos, topk, w, fill=0.0):
    """(dy, dw, sum |g y| per slot)."""
    g, y = np.asarray(g, np.float64), np.asarray(y, np.float64)
    dy = np.full(y.shape, fill)
    dw = np.zeros((g.shape[0], topk))
    size = np.zeros_like(dw)
    for t, s, p in _slots(pos, topk, y.shape[0]):
        dy[p] = g[t] * (1.0 if w is None else float(w[t, s]))
        dw[t, s] = (g[t] * y[p]).sum()
        size[t, s] = np.abs(g[t] * y[p]).sum()
    return dy, dw, size
