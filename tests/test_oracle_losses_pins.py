"""The float64 oracle of the losses: gradients against central differences, and
closed forms.  Differences with a step of 1e-6 on values of order 1 are good to
about 1e-9; the bar is 1e-7."""
import numpy as np
import pytest

from oracle import losses as o


def differences(f, x, eps=1e-6):
    g = np.zeros_like(x)
    for i in np.ndindex(x.shape):
        a, b = x.copy(), x.copy()
        a[i] += eps
        b[i] -= eps
        g[i] = (f(a) - f(b)) / (2 * eps)
    return g


@pytest.fixture
def case():
    r = np.random.default_rng(3)
    x = r.normal(size=(8, 11)) * 2
    y = r.integers(0, 11, 8)
    y[2] = y[7] = -100
    return r, x, y


@pytest.mark.parametrize("tau", [1.0, 0.6, 2.0])
def test_logprobs_gradient(case, tau):
    r, x, y = case
    d = r.normal(size=8)
    got = o.logprobs_grad(x, y, d, tau)
    np.testing.assert_allclose(got, differences(lambda v: np.sum(d * o.token_logprobs(v, y, tau)), x), atol=1e-7)
    assert not got[2].any() and not got[7].any()


@pytest.mark.parametrize("kl", [0.0, 0.1])
@pytest.mark.parametrize("weighted", [False, True])
def test_policy_gradient(case, kl, weighted):
    r, x, y = case
    logp = o.token_logprobs(x, y, 1.3)
    old = logp - np.array([0.0, 0.5, 0, -0.6, 0.1, -0.1, 0.9, 0])
    kw = dict(adv=r.normal(size=8), old=old, ref=logp + 0.4 * r.normal(size=8), kl_coef=kl, clip_high=0.28,
              weights=r.random(8) if weighted else None, temperature=1.3)
    np.testing.assert_allclose(o.policy(x, y, **kw)[3], differences(lambda v: o.policy(v, y, **kw)[0], x), atol=1e-7)


def test_policy_clip_takes_the_lower_side():
    x = np.log(np.array([[0.5, 0.5]]))
    y = np.array([0])
    for ratio, adv, loss, moves in [(1.5, 1.0, -1.2, False), (1.5, -1.0, 1.5, True), (0.5, 1.0, -0.5, True),
                                    (0.5, -1.0, 0.8, False), (1.1, 2.0, -2.2, True)]:
        got = o.policy(x, y, adv=[adv], old=np.log([0.5 / ratio]))
        assert got[0] == pytest.approx(loss)
        assert bool(np.any(got[3])) == moves


@pytest.mark.parametrize("kind,smooth,margin", [("sigmoid", 0.0, 0.0), ("sigmoid", 0.1, 0.3), ("hinge", 0.0, 0.2),
                                                ("squared", 0.0, 0.1)])
@pytest.mark.parametrize("average", [False, True])
def test_preference_gradient(case, kind, smooth, margin, average):
    r, x, y = case
    kw = dict(sequences=[(0, 3), (3, 4), (4, 7), (7, 8)], ref=r.normal(size=8) - 2, beta=0.4, label_smoothing=smooth,
              kind=kind, margin=margin, average=average)
    got = o.preference(x, y, **kw)
    np.testing.assert_allclose(got[4], differences(lambda v: o.preference(v, y, **kw)[0], x), atol=1e-7)


def test_preference_of_equal_sequences_is_log_two(case):
    _, x, y = case
    got = o.preference(np.concatenate([x, x]), np.concatenate([y, y]), [(0, 8), (8, 16)])
    assert got[0] == pytest.approx(np.log(2))


@pytest.mark.parametrize("rest", [False, True])
@pytest.mark.parametrize("tau", [1.0, 2.0])
def test_distill_gradient(case, rest, tau):
    r, x, _ = case
    ids = np.stack([r.permutation(11)[:4] for _ in range(8)])
    ids[1, 2] = -1
    ids[4] = -1
    t = r.normal(size=(8, 4))
    kw = dict(ids=ids, t=t, lse=np.log(np.exp(t / tau).sum(1)) + 0.5 if rest else None, mask=np.arange(8) != 6,
              temperature=tau)
    got = o.distill(x, **kw)
    np.testing.assert_allclose(got[2], differences(lambda v: o.distill(v, **kw)[0], x), atol=1e-7)
    assert got[1][6] == 0 and (rest or got[1][4] == 0)


def test_distill_of_the_teacher_itself_is_zero(case):
    r, x, _ = case
    ids = np.stack([r.permutation(11)[:5] for _ in range(8)])
    lse = np.log(np.exp(x / 2).sum(1))
    got = o.distill(x, ids, np.take_along_axis(x, ids, 1), lse, temperature=2.0)
    assert abs(got[0]) < 1e-13 and np.abs(got[2]).max() < 1e-15


def test_distill_with_every_word_listed_is_plain_kl(case):
    r, x, _ = case
    ids = np.tile(np.arange(11), (8, 1))
    t = r.normal(size=(8, 11))
    p = np.exp(t - np.log(np.exp(t).sum(1, keepdims=True)))
    q = np.exp(x - np.log(np.exp(x).sum(1, keepdims=True)))
    want = np.sum(p * np.log(p / q), 1)
    for lse in (None, np.log(np.exp(t).sum(1))):
        got = o.distill(x, ids, t, lse)
        np.testing.assert_allclose(got[1], want, rtol=1e-12)
        np.testing.assert_allclose(got[2] * 8, q - p, atol=1e-14)
