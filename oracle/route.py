"""Oracle of expert routing and its gradient: numpy in 64 bits, token by token,
from the definition.

  score s = sigmoid(x) or softmax(x) over the experts within reach (logit not
  NaN, not -inf; +inf stands for the largest finite float); choice c = s +
  bias; the best groups by the sum of their best choices; the k largest
  choices, ties to the lower index (without a bias: by the logits); weight =
  scale * s, renormalised over the chosen.
"""
from __future__ import annotations

import numpy as np

LARGEST = float(np.finfo(np.float32).max)


def scores(x, score: str):
    """(scores float64 [experts], within reach) of one token."""
    x = np.asarray(x, np.float64)
    reach = ~np.isnan(x) & (x > -np.inf)
    y = np.minimum(np.where(reach, x, 0.0), LARGEST)
    s = np.zeros(len(x))
    if score == "sigmoid":
        e = np.exp(-np.abs(y))
        s = np.where(y >= 0, 1 / (1 + e), e / (1 + e))
    elif reach.any():
        p = np.where(reach, np.exp(np.where(reach, y - y[reach].max(), 0.0)), 0.0)
        s = p / p.sum()
    return np.where(reach, s, 0.0), reach


def shares(x, chosen, score: str):
    """The chosen experts' scores over their sum, without underflow."""
    y = np.minimum(np.asarray(x, np.float64)[chosen], LARGEST)
    log_s = y if score == "softmax" else np.minimum(y, 0) - np.log1p(np.exp(-np.abs(y)))
    q = np.exp(log_s - log_s.max())
    return q / q.sum()


def _best(rank, n):
    """Indices of the n largest finite-or-+inf entries, descending, ties to the lower."""
    order = sorted((i for i in range(len(rank)) if rank[i] > -np.inf), key=lambda i: (-rank[i], i))
    return order[:n]


def route(logits, k: int, bias=None, score: str = "softmax", groups: int = 1, kept: int | None = None, best: int = 2,
          renorm: bool = True, scale: float = 1.0):
    """(idx int32 [tokens, k], weight float64 [tokens, k], load int32 [experts])."""
    logits = np.asarray(logits, np.float64)
    t, e = logits.shape
    idx, weight = np.full((t, k), -1, np.int32), np.zeros((t, k))
    load = np.zeros(e, np.int32)
    kept = groups if kept is None else kept
    for r in range(t):
        s, reach = scores(logits[r], score)
        with np.errstate(invalid="ignore"):
            c = s + (0.0 if bias is None else np.asarray(bias, np.float64))
        c = np.where(reach & ~np.isnan(c), c, -np.inf)
        rank = c if bias is not None else np.where(reach, np.minimum(np.where(reach, logits[r], 0), LARGEST), -np.inf)
        if kept < groups:
            per = e // groups
            value = np.full(groups, -np.inf)
            for g in range(groups):
                top = [c[g * per + i] for i in _best(c[g * per: (g + 1) * per], best)]
                if top:
                    value[g] = sum(top)
            keep = set(sorted(range(groups), key=lambda g: (-value[g], g))[:kept])
            rank = np.where([i // per in keep for i in range(e)], rank, -np.inf)
        chosen = _best(rank, k)
        if not chosen:
            continue
        idx[r, : len(chosen)] = chosen
        weight[r, : len(chosen)] = scale * (shares(logits[r], chosen, score) if renorm else s[chosen])
        load[chosen] += 1
    return idx, weight, load


def grad(logits, idx, grad_weight, score: str = "softmax", renorm: bool = True, scale: float = 1.0):
    """(gradient float64 [tokens, experts], magnitude of its terms, for error bounds)."""
    logits = np.asarray(logits, np.float64)
    out, size = np.zeros(logits.shape), np.zeros(logits.shape)
    for r in range(len(logits)):
        s, reach = scores(logits[r], score)
        places = [i for i, e in enumerate(idx[r]) if 0 <= e < len(s) and reach[e]]
        if not places:
            continue
        chosen = [int(idx[r, i]) for i in places]
        g = scale * np.asarray(grad_weight, np.float64)[r, places]
        y = np.minimum(logits[r], LARGEST)
        below = 1 / (1 + np.exp(np.minimum(y, 700))) if score == "sigmoid" else np.ones(len(s))
        if renorm:
            q = shares(logits[r], chosen, score)
            dot, total = (g * q).sum(), (np.abs(g) * q).sum()
            for j, e in enumerate(chosen):
                out[r, e] += q[j] * (g[j] - dot) * below[e]
                size[r, e] += q[j] * (abs(g[j]) + total) * below[e]
        elif score == "sigmoid":
            for j, e in enumerate(chosen):
                out[r, e] += g[j] * s[e] * below[e]
                size[r, e] += abs(g[j]) * s[e] * below[e]
        else:
            dot, total = (g * s[chosen]).sum(), (np.abs(g) * s[chosen]).sum()
            out[r] = -s * dot
            size[r] = s * total
            for j, e in enumerate(chosen):
                out[r, e] += s[e] * g[j]
                size[r, e] += s[e] * abs(g[j])
    return out, size
