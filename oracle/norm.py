"""Layer norm and RMS norm of the rows of a matrix, forward and backward, float64 (oracle).

Per row x of n elements (an RMS norm has mu = 0 and no bias):
    mu = sum(x) / n,  r = 1 / sqrt(sum((x - mu)^2) / n + eps),  z = (x - mu) r,  y = z w + b
    g = dy w,  dx = r (g - [layer] mean(g) - z mean(g z)),  dw = sum_rows dy z,  db = sum_rows dy
"""

from __future__ import annotations

import numpy as np


def f64(a):
    return np.asarray(a, dtype=np.float64)


def forward(x, w, b, eps: float, layer: bool):
    """(y, mean, rstd); ``w`` and ``b`` may be None (1 and 0)."""
    x = f64(x)
    mu = x.mean(axis=1) if layer else np.zeros(x.shape[0])
    c = x - mu[:, None]
    r = 1.0 / np.sqrt((c * c).mean(axis=1) + eps)
    y = c * r[:, None]
    if w is not None:
        y = y * f64(w)
    if b is not None:
        y = y + f64(b)
    return y, mu, r


def backward(dy, x, w, mean, rstd, layer: bool):
    """(dx, dw, db) with the statistics given."""
    dy, x, mean, rstd = f64(dy), f64(x), f64(mean), f64(rstd)
    z = (x - mean[:, None]) * rstd[:, None] if layer else x * rstd[:, None]
    g = dy * f64(w) if w is not None else dy
    dx = g - z * (g * z).mean(axis=1, keepdims=True)
    if layer:
        dx = dx - g.mean(axis=1, keepdims=True)
    return dx * rstd[:, None], (dy * z).sum(axis=0), dy.sum(axis=0)
