"""Pins of the Muon oracle: closed forms that a slip in it would miss."""
import numpy as np
import pytest

from oracle import muon as O

A, B, C = 3.4445, -4.7750, 2.0315


def poly(s, steps=5):
    for _ in range(steps):
        s = A * s + B * s ** 3 + C * s ** 5
    return s


@pytest.mark.parametrize("h,w", [(1, 1), (1, 9), (9, 1), (5, 5), (4, 11), (11, 4)])
def test_two_routes_agree(h, w):
    u = np.random.default_rng(h * 100 + w).standard_normal((h, w))
    assert np.allclose(O.orthogonalize(u), O.by_singular_values(u), rtol=0, atol=1e-12)
    assert np.allclose(O.orthogonalize(u.T), O.orthogonalize(u).T, rtol=0, atol=1e-12)
    assert np.allclose(O.orthogonalize(7 * u), O.orthogonalize(u), rtol=0, atol=1e-12)


def test_closed_forms():
    # a single row keeps its direction: length p(1)
    u = np.array([[3.0, 0.0, 4.0]])
    assert np.allclose(O.orthogonalize(u), poly(1.0) * u / 5, atol=1e-13)
    # equal singular values: each 1 / sqrt(n) before the steps
    assert np.allclose(O.orthogonalize(2 * np.eye(4)), poly(0.5) * np.eye(4), atol=1e-13)
    # diag(3, 4): 0.6 and 0.8
    assert np.allclose(O.orthogonalize(np.diag([3.0, 4.0])), np.diag([poly(0.6), poly(0.8)]), atol=1e-13)
    # eps is a floor of the norm
    assert np.allclose(O.orthogonalize(np.diag([3.0, 4.0]), eps=10.0), np.diag([poly(0.3), poly(0.4)]), atol=1e-13)
    assert np.all(O.orthogonalize(np.zeros((3, 5))) == 0)


def test_step_closed_form():
    p, g, m = np.ones((1, 4)), np.array([[0.0, 2.0, 0.0, 0.0]]), np.array([[4.0, 0.0, 0.0, 0.0]])
    # m = 2 + g on the first axis, u = g + m / 2: directions (1, 3) / sqrt(10)
    q, n = O.step(p, g, m, lr=0.1, momentum=0.5, weight_decay=0.5)
    assert np.allclose(n, [[2, 2, 0, 0]])
    d = np.array([1.0, 3.0, 0, 0]) / np.sqrt(10)
    assert np.allclose(q, 1 - 0.05 - 0.1 * poly(1.0) * d)
    q, _ = O.step(p, g, m, lr=0.1, momentum=0.5, nesterov=False, adjust="match_rms")
    assert np.allclose(q, 1 - 0.1 * 0.2 * 2 * poly(1.0) * np.array([1.0, 1.0, 0, 0]) / np.sqrt(2))
    # taller than wide: the update is scaled by sqrt(rows / cols)
    q, _ = O.step(np.zeros((4, 1)), g.T, 0 * m.T, lr=0.1)
    assert np.allclose(q[:, 0], [0, -0.1 * 2 * poly(1.0), 0, 0])


def test_singular_values_end_near_one():
    s = np.linspace(0.01, 1, 500)
    assert poly(s).min() > 0.65 and poly(s).max() < 1.21
