"""Tokens sorted by expert and back in float64, and rows in 8 bits: the oracle.

The order is a stable sort of the choices by expert; gathering, combining with
weights and the gradients follow it.  Rows in 8 bits: the scale and the quotient
are defined in 32 bits, the rounding to e4m3 is written out.
"""
from __future__ import annotations

import numpy as np

BLOCK = 128


def order(idx, experts):
    """(slot, source, offsets): choices outside [0, experts) take no part."""
    idx = np.asarray(idx)
    flat = idx.reshape(-1).astype(np.int64)
    valid = (flat >= 0) & (flat < experts)
    used = np.flatnonzero(valid)
    used = used[np.argsort(flat[used], kind="stable")]
    source = np.full(flat.size, -1, np.int64)
    source[:used.size] = used
    slot = np.full(flat.size, -1, np.int64)
    slot[used] = np.arange(used.size)
    offsets = np.concatenate([[0], np.cumsum(np.bincount(flat[valid], minlength=experts))])
    return slot.reshape(idx.shape), source, offsets


def gather(x, source, k):
    """A row for each place, zeros where there is none."""
    x, source = np.asarray(x, np.float64), np.asarray(source)
    out = np.zeros((source.size, x.shape[1]))
    out[source >= 0] = x[source[source >= 0] // k]
    return out


def combine(rows, slot, weight=None):
    """(out, size): the weighted sums, and the sums of the terms' magnitudes."""
    rows, slot = np.asarray(rows, np.float64), np.asarray(slot)
    out = np.zeros((slot.shape[0], rows.shape[1]))
    size = np.zeros_like(out)
    for j in range(slot.shape[1]):
        have = slot[:, j] >= 0
        part = rows[slot[have, j]]
        if weight is not None:
            part = part * np.asarray(weight, np.float64)[have, j, None]
        out[have] += part
        size[have] += np.abs(part)
    return out, size


def combine_grad(grad, rows, slot, weight):
    """(gradient of the rows, of the weights, sums of the latter's magnitudes)."""
    grad, rows = np.asarray(grad, np.float64), np.asarray(rows, np.float64)
    slot, weight = np.asarray(slot), np.asarray(weight, np.float64)
    d_rows, d_weight = np.zeros_like(rows), np.zeros(slot.shape)
    size = np.zeros(slot.shape)
    for j in range(slot.shape[1]):
        have = np.flatnonzero(slot[:, j] >= 0)
        at = slot[have, j]
        d_rows[at] = grad[have] * weight[have, j, None]
        d_weight[have, j] = (grad[have] * rows[at]).sum(1)
        size[have, j] = np.abs(grad[have] * rows[at]).sum(1)
    return d_rows, d_weight, size


def e4m3(v):
    """Nearest e4m3 values (ties to even), at most 448 in magnitude; NaN stays NaN."""
    v = np.asarray(v, np.float64)
    with np.errstate(invalid="ignore"):
        step = np.ldexp(1.0, np.maximum(np.frexp(np.where(np.isfinite(v), v, 0.0))[1] - 4, -9))
        return np.where(np.isnan(v), np.nan, np.clip(np.rint(v / step) * step, -448.0, 448.0))


def quantize(x):
    """(values as e4m3 holds them, scales float32) of float32 rows."""
    x = np.asarray(x, np.float32)
    rows, dim = x.shape
    blocks = -(-dim // BLOCK)
    q, scale = np.empty((rows, dim)), np.empty((rows, blocks), np.float32)
    with np.errstate(all="ignore"):
        for b in range(blocks):
            part = x[:, b * BLOCK:(b + 1) * BLOCK]
            most = np.abs(part).max(1)  # NaN where there is one
            unit = np.where(most < np.float32(2.0 ** -100), np.float32(2.0 ** -100), most) * np.float32(1 / 448)
            scale[:, b] = unit
            q[:, b * BLOCK:(b + 1) * BLOCK] = e4m3((part / unit[:, None]).astype(np.float32))
    return q, scale


def product(q, scale, weight, weight_scale, offsets=None):
    """(y, size) of rows and weights as e4m3 holds them: [groups, cols, dim] weights over the groups' rows."""
    q, weight = np.asarray(q, np.float64), np.asarray(weight, np.float64)
    if offsets is None:
        offsets, weight, weight_scale = [0, len(q)], weight[None], np.asarray(weight_scale)[None]
    groups, cols, dim = weight.shape

    def spread(s, axis):
        return np.repeat(np.asarray(s, np.float64), BLOCK, axis)

    a = q * spread(scale, 1)[:, :dim]
    y, size = np.zeros((len(q), cols)), np.zeros((len(q), cols))
    for g in range(groups):
        rows = slice(int(offsets[g]), int(offsets[g + 1]))
        b = weight[g] * spread(spread(weight_scale[g], 0)[:cols], 1)[:, :dim]
        y[rows] = a[rows] @ b.T
        size[rows] = np.abs(a[rows]) @ np.abs(b).T
    return y, size
