"""Embedding lookup with a scale and the gradient of its table, float64 (oracle).

    out[t] = scale * table[ids[t]];   dtable[v] = scale * sum over t with ids[t] = v of dy[t]
An id outside the table reads a zero row and takes no part in the gradient, nor does
``padding_idx``.
"""

from __future__ import annotations

import numpy as np


def forward(table, ids, scale: float):
    table = np.asarray(table, dtype=np.float64)
    out = np.zeros((len(ids), table.shape[1]))
    for t, i in enumerate(ids):
        if 0 <= i < table.shape[0]:
            out[t] = scale * table[i]
    return out


def backward(ids, dy, scale: float, vocab: int, padding_idx: int = -1, start=None):
    """The gradient, added to ``start`` where given."""
    dy = np.asarray(dy, dtype=np.float64)
    grad = np.zeros((vocab, dy.shape[1])) if start is None else np.array(start, dtype=np.float64)
    for t, i in enumerate(ids):
        if 0 <= i < vocab and i != padding_idx:
            grad[i] += scale * dy[t]
    return grad
