"""Penalties, biases and masks on logits in float64: the oracle."""
from __future__ import annotations

import numpy as np


def penalize(logits, tokens=None, lengths=None, prompts=None, repetition=None, presence=None, frequency=None,
             bias_tokens=None, bias_values=None, allowed=None):
    """(logits, size): the changed logits, and the largest magnitude each went through."""
    x = np.array(logits, np.float64)
    rows, cols = x.shape
    size = np.abs(x)
    with np.errstate(invalid="ignore"):
        for r in range(rows):
            if tokens is not None:
                width = tokens.shape[1]
                n = width if lengths is None else min(max(int(lengths[r]), 0), width)
                p = 0 if prompts is None else min(max(int(prompts[r]), 0), n)
                said = tokens[r, :n].astype(np.int64)
                ok = (said >= 0) & (said < cols)
                seen = np.unique(said[ok])
                rep = 1.0 if repetition is None else float(repetition[r])
                x[r, seen] = np.where(x[r, seen] > 0, x[r, seen] / rep, x[r, seen] * rep)
                size[r, seen] = np.maximum(size[r, seen], np.abs(x[r, seen]))
                c, n = np.unique(said[p:][ok[p:]], return_counts=True)
                f = 0.0 if frequency is None else float(frequency[r])
                s = 0.0 if presence is None else float(presence[r])
                x[r, c] -= f * n + s
                size[r, c] += np.abs(f * n) + abs(s)
            if bias_tokens is not None:
                last = {int(c): float(v) for c, v in zip(bias_tokens[r], bias_values[r]) if 0 <= c < cols}
                for c, v in last.items():
                    x[r, c] += v
                    size[r, c] += abs(v)
            if allowed is not None:
                bits = (allowed[r].astype(np.int64)[:, None] >> np.arange(32)) & 1
                x[r, bits.reshape(-1)[:cols] == 0] = -np.inf
    return x, size
