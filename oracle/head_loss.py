"""Softmax cross entropy of an output head and its gradients, float64 (oracle).

    z = H W^T,  lse_t = log sum_v exp z_tv,  loss_t = lse_t - z_{t, label_t}
    G_tv = (exp(z_tv - lse_t) - [v = label_t]) dloss_t,  dH = G W,  dW = G^T H
A token whose label is ``ignore`` (or lies outside the vocabulary) has loss = lse = 0 and no
part in the gradients, whatever its hidden row holds.
"""

from __future__ import annotations

import numpy as np


def live_rows(labels, vocab: int, ignore: int) -> np.ndarray:
    lab = np.asarray(labels)
    return np.nonzero((lab != ignore) & (lab >= 0) & (lab < vocab))[0]


def forward(hidden, weight, labels, ignore: int = -100):
    """(loss, lse)."""
    h, w = np.asarray(hidden, np.float64), np.asarray(weight, np.float64)
    loss, lse = np.zeros(h.shape[0]), np.zeros(h.shape[0])
    rows = live_rows(labels, w.shape[0], ignore)
    z = h[rows] @ w.T
    top = z.max(axis=1) if len(rows) else np.zeros(0)
    lse[rows] = top + np.log(np.exp(z - top[:, None]).sum(axis=1))
    loss[rows] = lse[rows] - z[np.arange(len(rows)), np.asarray(labels)[rows]]
    return loss, lse


def logit_gradient(hidden, weight, labels, dloss, ignore: int = -100):
    """(rows, G of those rows)."""
    h, w = np.asarray(hidden, np.float64), np.asarray(weight, np.float64)
    rows = live_rows(labels, w.shape[0], ignore)
    z = h[rows] @ w.T
    _, lse = forward(h, w, labels, ignore)
    g = np.exp(z - lse[rows][:, None])
    g[np.arange(len(rows)), np.asarray(labels)[rows]] -= 1.0
    return rows, g * np.asarray(dloss, np.float64)[rows][:, None]


def backward(hidden, weight, labels, dloss, ignore: int = -100):
    """(dH, dW)."""
    h, w = np.asarray(hidden, np.float64), np.asarray(weight, np.float64)
    rows, g = logit_gradient(h, w, labels, dloss, ignore)
    dh = np.zeros(h.shape)
    dh[rows] = g @ w
    return dh, g.T @ h[rows]
