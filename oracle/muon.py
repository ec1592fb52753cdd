"""Float64 CPU reference of the Muon step (include/muon.h): the formulas, one
matrix at a time, with numpy.  Test infrastructure only; the package never
imports it."""
from __future__ import annotations

import numpy as np

COEFFICIENTS = ((3.4445, -4.7750, 2.0315),) * 5


def orthogonalize(u, coefficients=COEFFICIENTS, eps=1e-7):
    x = np.asarray(u, dtype=np.float64)
    x = x / max(np.sqrt(np.sum(x * x)), eps)
    for a, b, c in coefficients:
        # the singular values go through a s + b s^3 + c s^5
        g = x @ x.T if x.shape[0] <= x.shape[1] else x.T @ x
        q = b * g + c * (g @ g)
        x = a * x + (q @ x if x.shape[0] <= x.shape[1] else x @ q)
    return x


def by_singular_values(u, coefficients=COEFFICIENTS, eps=1e-7):
    """The same from the singular value decomposition: another route to it."""
    left, s, right = np.linalg.svd(np.asarray(u, dtype=np.float64), full_matrices=False)
    s = s / max(np.sqrt(np.sum(s * s)), eps)
    for a, b, c in coefficients:
        s = a * s + b * s ** 3 + c * s ** 5
    return (left * s) @ right


def step(p, g, m, lr=1e-3, momentum=0.95, nesterov=True, weight_decay=0.0, adjust="original", coefficients=COEFFICIENTS,
         eps=1e-7):
    """(p, m) after one step, for one matrix."""
    m = momentum * m + g
    u = g + momentum * m if nesterov else m
    h, w = p.shape
    s = np.sqrt(max(1.0, h / w)) if adjust == "original" else 0.2 * np.sqrt(max(h, w))
    return p - lr * weight_decay * p - lr * s * orthogonalize(u, coefficients, eps), m
