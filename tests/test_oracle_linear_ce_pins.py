"""Pins of the oracle of the linear output layer's cross entropy."""
import numpy as np

from oracle import linear_ce as O


def problem(n=5, d=4, v=7, seed=0):
    g = np.random.default_rng(seed)
    return g.standard_normal((n, d)), g.standard_normal((v, d)), g.integers(0, v, n)


def test_closed_forms():
    # equal logits: logp = -ln v, lse = ln v; the gradient of the logits is 1/v - onehot
    w, h = np.zeros((4, 2)), np.ones((3, 2))
    y = np.array([0, 3, -100])
    loss, gh, gw, logp, lse = O.linear_cross_entropy(h, w, y)
    assert np.isclose(loss, np.log(4)) and np.allclose(logp, [-np.log(4), -np.log(4), 0])
    assert np.allclose(lse, [np.log(4), np.log(4), 0]) and np.all(gh == 0)
    assert np.allclose(gw[:, 0], np.array([0.25 - 0.5, 0.25, 0.25, 0.25 - 0.5]))
    # two words, one dimension: logits 0 and 1, at half temperature 0 and 2
    loss, gh, gw, logp, lse = O.linear_cross_entropy(np.array([[1.0]]), np.array([[0.0], [1.0]]), np.array([0]), temperature=0.5)
    q = 1 / (1 + np.exp(-2.0))
    assert np.isclose(loss, np.log1p(np.exp(2.0))) and np.isclose(gh[0, 0], 2 * q) and np.allclose(gw[:, 0], [-2 * q, 2 * q])


def test_gradients_against_differences():
    h, w, y = problem()
    y[1] = -100
    share = np.array([0.3, 0.2, -0.1, 0.5, 0.7])
    kw = dict(weights=share, z_loss=0.2, temperature=0.7)
    _, gh, gw, _, _ = O.linear_cross_entropy(h, w, y, **kw)
    f = lambda a, b: O.linear_cross_entropy(a, b, y, **kw)[0]
    for x, g, at in ((h, gh, 0), (w, gw, 1)):
        for i in np.ndindex(x.shape):
            d = np.zeros_like(x)
            d[i] = 1e-5
            both = (f(h + d, w) - f(h - d, w)) if at == 0 else (f(h, w + d) - f(h, w - d))
            assert abs(both / 2e-5 - g[i]) < 1e-8


def test_shift_and_scale():
    h, w, y = problem()
    a = O.linear_cross_entropy(h, w, y)
    b = O.linear_cross_entropy(h, w + np.ones(4), y)      # every logit of a token moves alike
    assert np.isclose(a[0], b[0]) and np.allclose(a[3], b[3]) and np.allclose(b[4] - a[4], h.sum(1))
    c = O.linear_cross_entropy(h, w, y, grad_scale=3.0)
    assert np.isclose(a[0], c[0]) and np.allclose(3 * a[1], c[1]) and np.allclose(3 * a[2], c[2])
    assert np.allclose(a[2].sum(0), 0)                     # the words' shares of a token's gradient cancel


def test_bad_target_and_no_tokens():
    h, w, y = problem()
    loss, gh, gw, logp, _ = O.linear_cross_entropy(h, w, np.array([0, 7, 1, 2, -1]))
    assert np.isnan(loss) and np.isnan(logp[[1, 4]]).all() and np.isnan(gw).all() and np.isfinite(gh[[0, 2, 3]]).all()
    loss, gh, gw, _, _ = O.linear_cross_entropy(h, w, np.full(5, -100))
    assert loss == 0 and not gh.any() and not gw.any()
