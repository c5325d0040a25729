"""The output head in fp64: W4A16 product, token log-probabilities with
entropy and top alternatives, distillation from a teacher's alternatives, and
the gradients -- TEST INFRASTRUCTURE ONLY (see oracle/__init__).

The W4A16 product is the learner's side of arXiv 2607.15810, Eq. (12): bf16
activations times the NVFP4 weights.  Log-probabilities are what the pages
compare between rollout and learner (Table 3).  The loss forms are readings;
with y = it z, p = softmax(y), the conventions are
  * masked entries are -inf; a row of nothing but -inf has entropy 0, log-sum
    0 and a zero gradient;
  * alternatives rank by value, equal values by lower index;
  * a teacher's list leaves out ids outside [0, V); an id may stand twice.
"""

import numpy as np

from .nvfp4 import dequantize_unscaled


def row_stats(z, it):
    """(m, s) per row: m = max z, s = ln sum exp(it (z - m)); (-inf, 0) for an empty row."""
    z = np.asarray(z, np.float64)
    m = z.max(axis=1)
    base = np.where(np.isneginf(m), 0.0, m)
    with np.errstate(divide="ignore"):
        s = np.log(np.exp(it * (z - base[:, None])).sum(axis=1))
    return m, np.where(np.isneginf(m), 0.0, s)


def log_softmax(z, it):
    """ln p; -inf where masked."""
    z = np.asarray(z, np.float64)
    m, s = row_stats(z, it)
    base = np.where(np.isneginf(m), 0.0, m)
    return it * (z - base[:, None]) - s[:, None]


def _plogp(lp):
    p = np.exp(lp)
    return p * np.where(p > 0, lp, 0.0)


def token_logprob(z, ids, it=1.0, topk=0):
    """dict of logp (if ids), entropy, stats [T, 2], top_logp, top_id (if topk)."""
    z = np.asarray(z, np.float64)
    t, v = z.shape
    m, s = row_stats(z, it)
    lp = log_softmax(z, it)
    out = dict(entropy=-_plogp(lp).sum(axis=1), stats=np.stack([m, s], axis=1))
    if ids is not None:
        ids = np.asarray(ids, np.int64)
        have = (ids >= 0) & (ids < v)
        out["logp"] = np.where(have, lp[np.arange(t), np.where(have, ids, 0)], 0.0)
    if topk:
        order = np.argsort(-z, axis=1, kind="stable")[:, :topk]
        out["top_id"] = order.astype(np.int32)
        out["top_logp"] = np.take_along_axis(lp, order, axis=1)
    return out


def token_logprob_grad(z, ids, g_logp, g_entropy, it=1.0):
    """d(sum g_logp logp + g_entropy H) / dz; either gradient may be None."""
    z = np.asarray(z, np.float64)
    t, v = z.shape
    lp = log_softmax(z, it)
    p = np.exp(lp)
    out = np.zeros((t, v))
    if g_logp is not None:
        ids = np.asarray(ids, np.int64)
        have = (ids >= 0) & (ids < v)
        g = np.where(have, np.asarray(g_logp, np.float64), 0.0)
        out -= g[:, None] * p
        out[np.arange(t), np.where(have, ids, 0)] += g
    if g_entropy is not None:
        pl = _plogp(lp)
        out -= np.asarray(g_entropy, np.float64)[:, None] * (pl - p * pl.sum(axis=1)[:, None])
    out[np.isneginf(z.max(axis=1))] = 0.0
    return it * out


def teacher(t_val, t_id, v, it=1.0, renorm=True):
    """(q, ln q) [T, topk] of the teacher's list: 0 and -inf where left out."""
    y = np.asarray(t_val, np.float64)
    have = (np.asarray(t_id) >= 0) & (np.asarray(t_id) < v)
    y = np.where(have, it * y if renorm else y, -np.inf)
    if renorm:
        m = y.max(axis=1, keepdims=True)
        m = np.where(np.isneginf(m), 0.0, m)
        with np.errstate(divide="ignore", invalid="ignore"):
            y = y - m - np.log(np.exp(y - m).sum(axis=1, keepdims=True))
        y = np.where(have & ~np.isnan(y), y, -np.inf)    # a list of probability 0 stays 0
    return np.exp(y), y


def distill(z, t_val, t_id, weight=None, it=1.0, renorm=True):
    """loss [T] = w sum_i q_i (ln q_i - ln p_{id_i})."""
    z = np.asarray(z, np.float64)
    t, v = z.shape
    q, lq = teacher(t_val, t_id, v, it, renorm)
    at = np.where(q > 0, np.asarray(t_id, np.int64), 0)
    lp = np.take_along_axis(log_softmax(z, it), at, axis=1)
    with np.errstate(invalid="ignore"):
        loss = np.where(q > 0, q * (lq - lp), 0.0).sum(axis=1)
        if weight is not None:
            w = np.asarray(weight, np.float64)
            loss = np.where(w == 0, 0.0, w * loss)
    return loss


def distill_grad(z, t_val, t_id, g, weight=None, it=1.0, renorm=True):
    """d(sum g loss) / dz."""
    z = np.asarray(z, np.float64)
    t, v = z.shape
    q, _ = teacher(t_val, t_id, v, it, renorm)
    out = q.sum(axis=1, keepdims=True) * np.exp(log_softmax(z, it))
    for i in range(t):
        for j in range(q.shape[1]):
            if q[i, j] > 0:
                out[i, int(t_id[i][j])] -= q[i, j]
    w = np.asarray(g, np.float64) * it * (1.0 if weight is None else np.asarray(weight, np.float64))
    out[np.isneginf(z.max(axis=1))] = 0.0
    return w[:, None] * out


def w4a16(x, w, offsets, row_token=None):
    """Y [rows, N] = s_tW[e] x w_e^T over the packed rows, and sum |x w| per output.

    x float64 [Tx, K] (bf16 values), w = (packed, scales, s_tW) as oracle.nvfp4 gives them."""
    w_nib, w_sc, w_ts = w
    offsets = np.asarray(offsets, np.int64)
    rows = int(offsets[-1])
    row_token = np.arange(rows) if row_token is None else np.asarray(row_token, np.int64)
    y = np.zeros((rows, w_nib.shape[1]))
    bound = np.zeros_like(y)
    for e in range(len(offsets) - 1):
        sl = slice(int(offsets[e]), int(offsets[e + 1]))
        if sl.start == sl.stop:
            continue
        xa = np.asarray(x, np.float64)[row_token[sl]]
        wh = dequantize_unscaled(w_nib[e], w_sc[e]) * np.float64(np.float32(w_ts[e]))
        y[sl] = xa @ wh.T
        bound[sl] = np.abs(xa) @ np.abs(wh).T
    return y, bound
