"""Plain reference of slots sorted by expert, and of rows brought there and
back, in fp64.

TEST INFRASTRUCTURE.  Only the test suite and the smoke check may use this
module; it shares nothing with the GPU library.
"""

from __future__ import annotations

import numpy as np


def sort(experts, n_experts):
    """(offsets, position, order) of [tokens, slots] experts."""
    flat = np.asarray(experts).reshape(-1)
    order = [i for e in range(n_experts) for i in np.flatnonzero(flat == e)]
    offsets = np.concatenate([[0], np.cumsum([(flat == e).sum() for e in range(n_experts)])]).astype(np.int64)
    position = np.full(flat.shape, -1, np.int32)
    position[order] = np.arange(len(order))
    return offsets, position.reshape(np.shape(experts)), np.array(order, np.int32)


def slots(position, rows_len):
    """(token, slot, place) of every slot that has a row."""
    return [(t, j, p) for t, row in enumerate(position) for j, p in enumerate(row) if 0 <= p < rows_len]


def gather(x, position, rows, weights=None):
    out = np.array(rows, np.float64)
    for t, j, p in slots(position, len(rows)):
        out[p] = x[t] * (1.0 if weights is None else weights[t, j])
    return out


def combine(rows, position, weights=None, residual=None):
    """(y, mag): mag = the sums of absolute terms."""
    T, C = position.shape[0], rows.shape[1]
    y = np.zeros((T, C)) if residual is None else np.array(residual, np.float64)
    mag = np.abs(y)
    for t, j, p in slots(position, len(rows)):
        v = rows[p] * (1.0 if weights is None else weights[t, j])
        y[t] += v
        mag[t] += np.abs(v)
    return y, mag


def combine_backward(dy, position, rows, weights=None):
    """(drows, dweights, mag of dweights); rows without a slot are NaN in drows."""
    drows = np.full(rows.shape, np.nan)
    dw, mag = np.zeros(position.shape), np.zeros(position.shape)
    for t, j, p in slots(position, len(rows)):
        drows[p] = dy[t] * (1.0 if weights is None else weights[t, j])
        dw[t, j] = dy[t] @ rows[p]
        mag[t, j] = np.abs(dy[t]) @ np.abs(rows[p])
    return drows, dw, mag
