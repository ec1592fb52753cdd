"""GPU parity of the losses (include/losses.h) at the edges of their formulas
and of their arguments, and what one call may see of another.  The bars are
those of test_gpu_losses.py, which derives them."""
import numpy as np
import pytest
import torch

import memory_efficient_optimizer_gb300 as meo
from oracle import losses as o
from test_gpu_losses import (BF16, DTYPES, FP32, U, _built, check, check_grad, check_logp, ds, f64, flat, make,  # noqa: F401
                             per_token)

pytestmark = pytest.mark.gpu
INF = float("inf")


# ---- words of probability 0 -----------------------------------------------------

def two_sides(vocab, dtype, masked):
    """A chosen and a rejected sequence of three tokens; one target of the
    `masked` side has probability 0."""
    x, y = make(6, vocab, dtype, vocab + 3)
    t = 1 if masked == "chosen" else 4
    x[t, y[t]] = -INF
    return x, y


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("vocab", [7, 1000, 50257])
@pytest.mark.parametrize("masked", ["chosen", "rejected"])
@pytest.mark.parametrize("smooth", [0.0, 0.1])
def test_preference_with_a_side_of_probability_zero(masked, smooth, vocab, dtype):
    """h = -inf or +inf: -(1 - e) ln s(beta h) is inf or 0, the other side's
    term 0 or inf where e > 0 and nothing where e = 0; the derivative is finite."""
    x, y = two_sides(vocab, dtype, masked)
    at = torch.tensor([0, 3, 6]).cuda()
    out = meo.preference_loss(x, y, seq_offsets=at, beta=0.3, label_smoothing=smooth)
    want, pair, rewards, lp, grad, d = o.preference(f64(x), y.cpu().numpy(), [(0, 3), (3, 6)], beta=0.3,
                                                    label_smoothing=smooth)
    assert want == (0.0 if masked == "rejected" and smooth == 0 else INF)
    check("loss", f64(out.loss), want, 0.0)
    check("pair_loss", f64(out.pair_loss), pair, 0.0)
    e = 3 * (ds(vocab) + 4 * U * 60)
    check("rewards", f64(out.rewards), rewards, 0.3 * e, 4 * U)
    # the logistic function is 0 or 1 there, so the coefficient beta (e - 1), beta e is one rounding off
    check_grad(f64(out.grad), grad, d, vocab, dtype)


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("vocab", [7, 1000, 50257])
def test_policy_first_step_on_a_word_of_probability_zero(vocab, dtype):
    """Without old_logp the ratio is 1, whatever the target's probability is."""
    x, y = make(5, vocab, dtype, vocab + 4)
    x[1, y[1]] = -INF
    x[2, y[2]] = -INF
    adv = torch.tensor([1.0, 0.7, -1.5, 0.4, -1.0]).cuda()
    out = meo.policy_loss(x, y, adv)
    want, token, lp, grad, d = o.policy(f64(x), y.cpu().numpy(), f64(adv))
    assert np.isneginf(lp[1:3]).all() and np.array_equal(token, -f64(adv))
    check_logp(f64(out.logp), lp, vocab)
    check("token_loss", f64(out.token_loss), token, 0.0, 2 * U)
    check("loss", f64(out.loss), want, 0.0, 8 * U)
    check_grad(f64(out.grad), grad, d, vocab, dtype)
    # a row without a distribution still answers NaN
    y[3] = vocab
    x[4, 0] = float("nan")
    out = meo.policy_loss(x, y, adv)
    assert out.token_loss[3:].isnan().all() and out.grad[3:].isnan().all() and out.grad[:3].isfinite().all()
    assert out.token_loss[:3].isfinite().all()


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("vocab", [7, 1000, 50257])
def test_policy_kl_term_of_a_word_of_probability_zero(vocab, dtype):
    """exp(d) - d - 1 grows without bound on both sides: inf where the policy
    gives the word probability 0, and where the reference does."""
    x, y = make(4, vocab, dtype, vocab + 5)
    x[1, y[1]] = -INF
    lp = o.token_logprobs(f64(x), y.cpu().numpy())
    ref = torch.tensor(np.float32(np.where(np.isfinite(lp), lp, -5) - 0.3)).cuda()
    ref[2] = -INF
    old = torch.tensor(np.float32(np.where(np.isfinite(lp), lp, -5) + 0.1)).cuda()
    adv = torch.tensor([1.0, 1.0, -1.0, 0.5]).cuda()
    for args in ((None, ref), (old, ref)):
        out = meo.policy_loss(x, y, adv, *args, kl_coef=0.05)
        want, token, _, grad, d = o.policy(f64(x), y.cpu().numpy(), f64(adv), *(None if a is None else f64(a) for a in args),
                                           kl_coef=0.05)
        assert want == INF and np.isposinf(token[1:3]).all()
        err = 4 * (6 * ds(vocab) + 8 * U * 40)
        check("token_loss", f64(out.token_loss), token, err, err)
        check("loss", f64(out.loss), want, 0.0)
        keep = [0, 2, 3]     # (the derivative of token 1 is infinite)
        check("grad", f64(out.grad)[keep], grad[keep], 3 * ds(vocab) * np.abs(d[keep])[:, None] + 1e-37,
              err + (2 ** -8 if dtype is BF16 else 0))


# ---- state between rows and between calls ---------------------------------------------

def ring_case(op, tokens, vocab, k, dtype):
    from test_gpu_losses import distill_inputs
    x, y = make(tokens, vocab, dtype, 7, ignore=range(3, tokens, 7))
    if op == "policy":
        adv = per_token(tokens, 5)
        return lambda **kw: meo.policy_loss(x, y, adv, **kw), lambda: o.policy(f64(x), y.cpu().numpy(), f64(adv))
    ids, t = distill_inputs(tokens, vocab, k, 8)
    lse = torch.logsumexp(t, 1) + 0.2
    mask = y != -100
    return (lambda **kw: meo.distill_loss(x, ids, t, lse, mask=mask, **kw),
            lambda: o.distill(f64(x), ids.cpu().numpy(), f64(t), f64(lse), mask.cpu().numpy()))


@pytest.mark.parametrize("op,tokens,vocab,k,dtype", [
    ("distill", 2400, 20001, 300, FP32), ("distill", 2400, 9001, 319, FP32), ("distill", 1200, 50257, 500, BF16),
    ("distill", 800, 128256, 1000, BF16), ("policy", 2400, 20001, 0, FP32), ("policy", 1200, 50257, 0, BF16)])
def test_a_row_in_the_ring_is_not_overwritten_while_it_is_read(op, tokens, vocab, k, dtype):
    """The next row's copies wait for places that this row's gradient is made
    from: with lists the ring has one place more than a row's, or none.  Every
    word of every row is right, in each of several passes."""
    call, oracle = ring_case(op, tokens, vocab, k, dtype)
    outs = [call() for _ in range(8)]
    want = oracle()
    grad, w = (want[3], want[4]) if op == "policy" else (want[2], want[3])
    check("grad", f64(outs[0].grad), grad, 6 * ds(vocab) * np.abs(w)[:, None] + 1e-37,
          6 * ds(vocab) + (2 ** -8 if dtype is BF16 else 4 * U))
    loss_alone = call(need_grad=False)
    assert torch.equal(loss_alone.token_loss, outs[0].token_loss) and torch.equal(loss_alone.loss, outs[0].loss)
    for out in outs[1:]:
        assert torch.equal(out.grad, outs[0].grad) and torch.equal(out.token_loss, outs[0].token_loss)
