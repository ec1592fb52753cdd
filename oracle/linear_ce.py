"""Float64 CPU reference of the cross entropy of a linear output layer
(include/linear_ce.h), with numpy.  Test infrastructure only; the package never
imports it."""
from __future__ import annotations

import numpy as np

from .losses import log_softmax


def linear_cross_entropy(h, w, y, weights=None, z_loss=0.0, temperature=1.0, ignore=-100, grad_scale=1.0):
    """(loss, grad_hidden, grad_weight, logp, lse) for h [tokens, dim], w [vocab, dim], y [tokens]."""
    h, w = np.asarray(h, dtype=np.float64), np.asarray(w, dtype=np.float64)
    n, vocab = len(y), w.shape[0]
    keep = y != ignore
    share = np.full(n, 1.0 / max(1, int(keep.sum()))) if weights is None else np.asarray(weights, dtype=np.float64)
    logp, lse, dx = np.zeros(n), np.zeros(n), np.zeros((n, vocab))
    loss = 0.0
    for t in range(n):
        if not keep[t]:
            continue
        z = w @ h[t] / temperature
        lq = log_softmax(z)
        with np.errstate(invalid="ignore"):
            lse[t] = (z - lq)[np.argmax(z)] if np.isfinite(z).all() else np.nan
        if not 0 <= y[t] < vocab:
            logp[t], dx[t] = np.nan, np.nan
        else:
            logp[t] = lq[y[t]]
            dx[t] = share[t] / temperature * np.exp(lq) * (1 + 2 * z_loss * lse[t])
            dx[t, y[t]] -= share[t] / temperature
        loss += share[t] * (z_loss * lse[t] ** 2 - logp[t])
    dx *= grad_scale
    return loss, dx @ w, dx.T @ h, logp, lse
