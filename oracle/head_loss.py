"""Oracle of the head's loss and its gradient: numpy in 64 bits, from the
definition, row by row of the logit matrix it materialises.

  x = hidden @ weight.T,  lse = log sum exp x,  loss = lse - x[target]
  G = g (exp(x - lse) - onehot),  grad_hidden = G weight,  grad_weight = G^T hidden

A row whose target is ``ignore`` has loss 0 and lse 0; any other target
outside the vocabulary gives NaN in both; neither has a gradient.
"""
from __future__ import annotations

import numpy as np


def _sides(target: np.ndarray, vocab: int, ignore: int):
    target = np.asarray(target, dtype=np.int64)
    ignored = target == ignore
    return ignored, ~ignored & (target >= 0) & (target < vocab)


def loss(hidden, weight, target, ignore: int = -100):
    """(loss, lse), float64 [rows]."""
    h, w = np.asarray(hidden, np.float64), np.asarray(weight, np.float64)
    ignored, counts = _sides(target, len(w), ignore)
    out_loss, out_lse = np.full(len(h), np.nan), np.full(len(h), np.nan)
    out_loss[ignored] = out_lse[ignored] = 0.0
    for r in np.flatnonzero(counts):
        x = w @ h[r]
        top = x.max()
        out_lse[r] = top + np.log(np.exp(x - top).sum()) if np.isfinite(top) else top
        others = np.delete(x, target[r]) - x[target[r]]
        # log(1 + sum over the others): exact also where it is nearly 0
        m = others.max() if len(others) else -np.inf
        if m <= 0:
            out_loss[r] = np.log1p(np.exp(others).sum())
        else:
            out_loss[r] = m + np.log(np.exp(-m) + np.exp(others - m).sum())
    return out_loss, out_lse


def grad(hidden, weight, target, g, ignore: int = -100):
    """(grad_hidden, grad_weight, G), float64; G is [rows, vocab]."""
    h, w = np.asarray(hidden, np.float64), np.asarray(weight, np.float64)
    _, counts = _sides(target, len(w), ignore)
    G = np.zeros((len(h), len(w)))
    for r in np.flatnonzero(counts):
        x = w @ h[r]
        p = np.exp(x - x.max())
        p /= p.sum()
        p[target[r]] -= 1.0
        G[r] = p * np.float64(g[r])
    h = np.where(counts[:, None], h, 0.0)
    return G @ w, G.T @ h, G
