"""The steps around the experts in float64: the residual norm and its gradient,
token rows sorted by expert and back with their gradients.

Readings: the norm divides by the root of the mean square plus eps and has a
weight and no bias; the residual stream is normed as it is stored (the caller
rounds it).  Written from the formulas; no code is shared with the library.
"""
from __future__ import annotations

import numpy as np


def norm_forward(s, weight, eps):
    """(y, rstd) of the stream s [T, cols]."""
    s = np.asarray(s, dtype=np.float64)
    rstd = (np.mean(s * s, axis=1) + eps) ** -0.5
    return s * rstd[:, None] * np.asarray(weight, dtype=np.float64), rstd


def norm_backward(dy, s, weight, rstd, d_next=None):
    """(gradient of s, gradient of weight).  rstd as the forward left it; the
    mean square is 1 / rstd^2."""
    dy, s, rstd = (np.asarray(a, dtype=np.float64) for a in (dy, s, rstd))
    n = s * rstd[:, None]
    a = dy * np.asarray(weight, dtype=np.float64)
    d = rstd[:, None] * (a - n * np.mean(a * n, axis=1, keepdims=True))
    return d if d_next is None else d + np.asarray(d_next, dtype=np.float64), (dy * n).sum(0)


def local_pairs(pair_pos, M):
    """[(token, slot, row)] of the pairs that have a row."""
    return [(t, j, int(p)) for t, row in enumerate(np.asarray(pair_pos)) for j, p in enumerate(row) if 0 <= p < M]


def sort_rows(x, pair_pos, out):
    """out with the rows of local pairs replaced by their tokens'."""
    out = np.array(out, dtype=np.float64)
    for t, _, p in local_pairs(pair_pos, len(out)):
        out[p] = x[t]
    return out


def combine_rows(y, pair_pos, topk_w):
    y = np.asarray(y, dtype=np.float64)
    out = np.zeros((len(pair_pos), y.shape[1]))
    for t, j, p in local_pairs(pair_pos, len(y)):
        out[t] += (1.0 if topk_w is None else float(topk_w[t][j])) * y[p]
    return out


def combine_rows_backward(d_out, y, pair_pos, topk_w, dy):
    """(dy with the rows of local pairs replaced, d_topk_w)."""
    d_out, y, dy = (np.array(a, dtype=np.float64) for a in (d_out, y, dy))
    d_w = np.zeros(np.shape(pair_pos))
    for t, j, p in local_pairs(pair_pos, len(y)):
        d_w[t, j] = d_out[t] @ y[p]
        dy[p] = (1.0 if topk_w is None else float(topk_w[t][j])) * d_out[t]
    return dy, d_w
