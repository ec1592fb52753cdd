"""The float64 oracle of the losses at the edges of their formulas: words of
probability 0."""
import numpy as np
import pytest

from oracle import losses as o

INF = float("inf")


def masked(t):
    """Four tokens in two sequences; the target of token t has probability 0."""
    r = np.random.default_rng(5)
    x, y = r.normal(size=(4, 9)), np.array([1, 2, 3, 4])
    x[t, y[t]] = -INF
    return x, y


@pytest.mark.parametrize("t,smooth,want", [(3, 0.0, 0.0), (3, 0.1, INF), (0, 0.0, INF), (0, 0.1, INF)])
def test_preference_with_a_side_of_probability_zero(t, smooth, want):
    x, y = masked(t)
    loss, pair, rewards, _, grad, d = o.preference(x, y, [(0, 2), (2, 4)], beta=0.3, label_smoothing=smooth)
    assert loss == want and pair[0] == want
    assert rewards[0 if t < 2 else 1] == -INF and np.isfinite(grad).all()
    # the limit of the derivative beta (e - 1 + s(beta h)) at h = -inf, +inf
    assert d[0] == pytest.approx(0.3 * (smooth - 1 if t < 2 else smooth)) and d[2] == -d[0]


def test_policy_first_step_on_a_word_of_probability_zero():
    x, y = masked(2)
    loss, token, logp, grad, d = o.policy(x, y, [1.0, 1.0, -2.0, 3.0])
    assert logp[2] == -INF and np.array_equal(token, [-1.0, -1.0, 2.0, -3.0]) and loss == pytest.approx(-0.75)
    assert np.isfinite(grad).all() and np.array_equal(d * 4, token)
    # a target outside the vocabulary is no word: NaN
    y[0] = 9
    assert np.isnan(o.policy(x, y, [1.0] * 4)[1][0])


def test_policy_kl_term_of_a_word_of_probability_zero():
    x, y = masked(2)
    ref = np.array([-1.0, -INF, -2.0, -3.0])
    token = o.policy(x, y, [1.0] * 4, ref=ref, kl_coef=0.1)[1]
    assert token[1] == INF and token[2] == INF and np.isfinite(token[[0, 3]]).all()
