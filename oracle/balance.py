"""The router's balance loss and the gradient of the router logits, written
out in float64 one token at a time (oracle side, test infrastructure only).

For the n live tokens of a sequence, s = sigmoid(z), p = s / sum s:
loss = E / (k n) * sum_e counts[e] * mean_t p[t][e].  The counts carry no
gradient.  Readings:

* a token whose logits are all -inf has p = 0;
* a sequence without live tokens has loss 0;
* masked tokens and tokens outside every sequence have zero gradient rows;
* ids outside [0, E) are neither counted nor weighted.
"""
from __future__ import annotations

import numpy as np


def log_sigmoid(z: np.ndarray) -> np.ndarray:
    """log(1 / (1 + e^-z)), exact far below zero as well."""
    z = np.asarray(z, dtype=np.float64)
    with np.errstate(over="ignore"):
        return np.where(z >= 0, -np.log1p(np.exp(-np.abs(z))), z - np.log1p(np.exp(-np.abs(z))))


def _probs(z: np.ndarray) -> np.ndarray:
    """p of one token."""
    ls = log_sigmoid(z)
    top = ls.max()
    if top == -np.inf:
        return np.zeros_like(ls)
    t = np.exp(ls - top)
    return t / t.sum()


def _tokens(T, seq_offsets, mask):
    """Live token indices of each sequence."""
    bounds = [0, T] if seq_offsets is None else [int(b) for b in seq_offsets]
    return [[t for t in range(lo, hi) if mask is None or mask[t]] for lo, hi in zip(bounds[:-1], bounds[1:])]


def balance_forward(z, ids, E: int, k: int, seq_offsets=None, mask=None):
    """dict(counts int64 [S, E], live int64 [S], probs [S, E], loss [S])."""
    z = np.asarray(z, dtype=np.float64)
    seqs = _tokens(z.shape[0], seq_offsets, mask)
    S = len(seqs)
    counts, live = np.zeros((S, E), np.int64), np.zeros(S, np.int64)
    probs, loss = np.zeros((S, E)), np.zeros(S)
    for s, toks in enumerate(seqs):
        live[s] = len(toks)
        for t in toks:
            probs[s] += _probs(z[t])
            for e in ids[t]:
                if 0 <= e < E:
                    counts[s, e] += 1
        if toks:
            probs[s] /= len(toks)
            loss[s] = E / (k * len(toks)) * float(counts[s] @ probs[s])
    return dict(counts=counts, live=live, probs=probs, loss=loss)


def gate(z, ids, E: int, norm: bool, scale: float):
    """Gate weights of one token's slots (0 for an id outside [0, E))."""
    ls = np.array([log_sigmoid(z[e]) if 0 <= e < E else -np.inf for e in ids])
    if not norm:
        return scale * np.exp(ls)
    top = ls.max()
    if top == -np.inf:
        return np.zeros(len(ids))
    w = np.exp(ls - top)
    return scale * w / w.sum()


def balance_backward(z, ids, fwd: dict, d_loss, E: int, k: int, seq_offsets=None, mask=None, d_w=None,
                     norm: bool = True, scale: float = 1.0):
    """(dz [T, E], size [T, E]): the gradient and, next to it, the sum of the
    magnitudes of its terms (what rounding errors scale with)."""
    z = np.asarray(z, dtype=np.float64)
    dz, size = np.zeros_like(z), np.zeros_like(z)
    for s, toks in enumerate(_tokens(z.shape[0], seq_offsets, mask)):
        n = len(toks)
        if n == 0:
            continue
        g = float(d_loss[s]) * E / (k * n * n) * fwd["counts"][s]
        for t in toks:
            p, c = _probs(z[t]), np.exp(log_sigmoid(-z[t]))
            dot = float(g @ p)
            dz[t] = p * c * (g - dot)
            size[t] = p * c * (np.abs(g) + float(np.abs(g) @ p))
            if d_w is None:
                continue
            w = gate(z[t], ids[t], E, norm, 1.0)
            dw = np.asarray(d_w[t], dtype=np.float64)
            mean = float(dw @ w) if norm else 0.0
            span = float(np.abs(dw) @ w) if norm else 0.0
            for j, e in enumerate(ids[t]):
                if 0 <= e < E:
                    dz[t, e] += scale * w[j] * c[e] * (dw[j] - mean)
                    size[t, e] += abs(scale) * w[j] * c[e] * (abs(dw[j]) + span)
    return dz, size


def balance_loss(z, ids, d_loss, E: int, k: int, counts, seq_offsets=None, mask=None, d_w=None, norm: bool = True,
                 scale: float = 1.0) -> float:
    """The scalar whose gradient balance_backward returns, the counts held
    fixed: sum_s d_loss[s] loss[s] + sum of d_w * gate weights over live tokens."""
    z = np.asarray(z, dtype=np.float64)
    total = 0.0
    for s, toks in enumerate(_tokens(z.shape[0], seq_offsets, mask)):
        n = len(toks)
        for t in toks:
            total += float(d_loss[s]) * E / (k * n * n) * float(counts[s] @ _probs(z[t]))
            if d_w is not None:
                total += float(np.asarray(d_w[t], dtype=np.float64) @ gate(z[t], ids[t], E, norm, scale))
    return total
