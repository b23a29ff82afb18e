"""The router's load-balance loss and its gradient in NumPy float64.

Per sequence s with n_s kept tokens: f = counts E / (k n_s), P = mean of the
tokens' shares p, loss = coeff / S' sum_s <f, P> over the S' sequences that
have tokens.  p is the softmax of the logits, or sigma(logits) / sum.
"""
from __future__ import annotations

import numpy as np


def shares(logits: np.ndarray, score: str) -> np.ndarray:
    """p [T, E]; an all -inf row has p = 0."""
    l = np.asarray(logits, np.float64)
    z = l if score == "softmax" else -np.logaddexp(0.0, -l)       # log sigma
    with np.errstate(invalid="ignore"):
        e = np.exp(z - z.max(axis=1, keepdims=True))
    e = np.where(np.isneginf(l), 0.0, e)
    t = e.sum(axis=1, keepdims=True)
    return np.divide(e, t, out=np.zeros_like(e), where=t != 0)


def balance_loss(logits, topk_idx, coeff, score, mask=None, seq_offsets=None, grad_loss=1.0):
    """dict(loss, counts [S, E], tokens [S + 1], probs [S, E], dlogits)."""
    l = np.asarray(logits, np.float64)
    T, E = l.shape
    k = topk_idx.shape[1]
    keep = np.ones(T, bool) if mask is None else np.asarray(mask, bool)
    off = np.array([0, T]) if seq_offsets is None else np.asarray(seq_offsets)
    S = len(off) - 1
    p = np.zeros((T, E))
    p[keep] = shares(l[keep], score)
    counts = np.zeros((S, E), np.int64)
    probs = np.zeros((S, E))
    tokens = np.zeros(S + 1, np.int64)
    d = np.zeros((T, E))
    rows = [np.arange(off[s], off[s + 1])[keep[off[s]:off[s + 1]]] for s in range(S)]
    full = sum(len(r) > 0 for r in rows)
    loss = 0.0
    for s, r in enumerate(rows):
        tokens[s] = n = len(r)
        if n == 0:
            continue
        idx = topk_idx[r].reshape(-1)
        counts[s] = np.bincount(idx[(idx >= 0) & (idx < E)], minlength=E)
        probs[s] = p[r].sum(axis=0) / n
        f = counts[s] * E / (k * n)
        loss += coeff / full * (f @ probs[s])
        g = grad_loss * coeff / (full * n) * p[r] * (f - (p[r] @ f)[:, None])
        if score == "sigmoid":
            g = g * np.exp(-np.logaddexp(0.0, l[r]))              # sigma(-l)
        d[r] = np.where(p[r] == 0, 0.0, g)
    tokens[S] = full
    return dict(loss=loss, counts=counts, tokens=tokens, probs=probs, dlogits=d)
