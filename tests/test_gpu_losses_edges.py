"""GPU parity of the losses (include/losses.h) at the edges of their formulas
and of their arguments, and what one call may see of another.  The bars are
those of test_gpu_losses.py, which derives them."""
import ctypes
import threading
import types

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


# ---- a student far from its teacher ------------------------------------------------

def check_distill_words(out, x, ids, t, lse, tau, dtype, w=None):
    """Against the oracle, word by word (without `lse` the rest is 0 and the
    entries' own sum stands for it).  With L the largest |ln| of a listed
    word's or of the other words' probability, ln q and ln(others) are good to
    ds + 4u L; a teacher's p to dp = 2^-22 + 4u (|t / T| + |lse|) and the roundings
    of a warp's sum of k entries, and so is its rest, absolutely.  The gradient on the list is T w (q (P + u) - p), off it
    T w (q (P + u) - u share), share a word's part of the unlisted mass: each
    product has its factors' relative errors and share u also the rest's."""
    xn, ids, t, lse = f64(x), ids.cpu().numpy(), f64(t), None if lse is None else f64(lse)
    vocab = xn.shape[1]
    want, token, grad, w = o.distill(xn, ids, t, lse, temperature=tau, weights=None if w is None else f64(w))
    rests = lse is not None
    lse = lse if rests else np.logaddexp.reduce(t / tau, axis=1)
    e_token, bar = np.zeros(len(token)), np.zeros(xn.shape)
    for i in range(len(token)):
        lq = o.log_softmax(xn[i] / tau)
        p = np.exp(t[i] / tau - lse[i])
        off = np.ones(vocab, dtype=bool)
        off[ids[i]] = False
        l_off = np.logaddexp.reduce(lq[off])
        rest = max(0.0, 1 - p.sum()) if rests else 0.0
        far = max(np.abs(lq[ids[i]]).max(), abs(l_off))
        dp = 2.0 ** -22 + 4 * U * (np.abs(t[i] / tau).max() + abs(lse[i])) + (p.size / 32 + 24) * U
        rel = 6 * ds(vocab) + 4 * U * far
        e_token[i] = tau ** 2 * (2 * rel + dp * (far + 20))
        share = np.where(off, np.exp(lq - l_off), 0.0) if rests else 0.0
        bar[i] = np.exp(lq) * (p.sum() + rest + dp) * (rel + dp) + share * (rest * rel + dp)
        bar[i, ids[i]] += p * (rel + dp)
    check("token_loss", f64(out.token_loss), token, e_token, 8 * U)
    check("loss", f64(out.loss), want, np.sum(w * e_token), 8 * U)
    if out.grad is not None:
        check("grad", f64(out.grad), grad, tau * w[:, None] * bar + 1e-36, 2.0 ** -8 if dtype is BF16 else 4 * U)


def far_student(vocab, k, tau, gap, dtype):
    """Listed words `gap` nats above the others; below them; one above and the
    others below; above them, and a teacher whose rest is rounding alone."""
    g = torch.Generator().manual_seed(vocab)
    x = torch.randn(4, vocab, generator=g) * 2 * tau
    ids = torch.stack([torch.randperm(vocab, generator=g)[:k] for _ in range(4)])
    for row, move in ((0, gap), (1, -gap), (2, -gap), (3, gap)):
        x[row, ids[row]] += move * tau
    x[2, ids[2, 0]] += 2 * gap * tau
    t = torch.randn(4, k, generator=g) * 2 * tau
    lse = torch.logsumexp(t / tau, 1) + torch.tensor([0.3, 0.3, 0.3, 0.0])
    return x.to(dtype).cuda(), ids.cuda(), t.cuda(), lse.cuda()


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("vocab,k", [(300, 5), (1000, 20), (8000, 64), (50257, 64), (128256, 400), (600011, 20)])
@pytest.mark.parametrize("tau,gap", [(1.0, 25), (1.0, 120), (0.2, 100), (0.1, 250)])
def test_distill_of_a_student_far_from_its_teacher(tau, gap, vocab, k, dtype):
    """The unlisted words' mass is far below what fp32 holds beside the listed
    words', or the other way about: loss and gradient are finite."""
    x, ids, t, lse = far_student(vocab, k, tau, gap, dtype)
    out = meo.distill_loss(x, ids, t, lse, temperature=tau)
    assert out.loss.isfinite() and out.grad.isfinite().all()
    check_distill_words(out, x, ids, t, lse, tau, dtype)
    check_distill_words(meo.distill_loss(x, ids, t, lse, temperature=tau, need_grad=False), x, ids, t, lse, tau, dtype)


def test_distill_small_rest_at_a_low_temperature():
    x = torch.full((1, 1000), -12.0)
    x[0, 5], x[0, 700] = 9.0, 8.5
    x, ids, t = x.cuda(), torch.tensor([[5, 700]]).cuda(), torch.tensor([[2.0, 1.0]]).cuda()
    lse = torch.logsumexp(t / 0.2, 1) + 0.2
    out = meo.distill_loss(x, ids, t, lse, temperature=0.2)
    check_distill_words(out, x, ids, t, lse, 0.2, FP32)


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("vocab,k", [(1000, 20), (50257, 64)])
def test_distill_far_students_in_many_rows_a_cluster(vocab, k, dtype):
    """Far and near rows in turn through the same places of the ring."""
    rows = [far_student(vocab, k, 0.5, gap, dtype) for gap in (0, 150)]
    x, ids, t, lse = (torch.cat([torch.stack([a, b], 1).flatten(0, 1)] * 200) for a, b in zip(*rows))
    first = meo.distill_loss(x[:8], ids[:8], t[:8], lse[:8], temperature=0.5)
    check_distill_words(first, x[:8], ids[:8], t[:8], lse[:8], 0.5, dtype)
    w = torch.full((1600,), 1 / 8.0, device="cuda")
    out = meo.distill_loss(x, ids, t, lse, temperature=0.5, weights=w)
    some = meo.distill_loss(x[800:1600], ids[800:1600], t[800:1600], lse[800:1600], temperature=0.5, weights=w[800:])
    assert torch.equal(out.grad[:800], out.grad[800:]) and torch.equal(out.grad[:800], some.grad)
    assert torch.equal(out.token_loss[:8].repeat(200), out.token_loss)
    again = out.grad[:8].double() - first.grad.double()
    assert again.abs().max() <= 2.0 ** -7 * first.grad.double().abs().max()


# ---- bad offsets -----------------------------------------------------------------

@pytest.mark.parametrize("average", [False, True])
def test_preference_pairs_with_a_bad_offset_answer_nan_in_every_value(average):
    x, y = make(16, 100, FP32)
    ref = per_token(16, 1)
    # sequences 0 .. 3; of the pairs (0, 2) and (1, 3) the second has a bad end
    for at in ([0, 4, 8, 12, 11], [0, 4, 8, 12, 17]):
        out = meo.preference_loss(x, y, ref, seq_offsets=torch.tensor(at).cuda(), average=average)
        assert out.loss.isnan() and out.pair_loss.isnan().tolist() == [False, True]
        assert out.rewards.isnan().tolist() == [False, True, False, True]
        good = meo.preference_loss(x[[0, 1, 2, 3, 8, 9, 10, 11]], y[[0, 1, 2, 3, 8, 9, 10, 11]],
                                   ref[[0, 1, 2, 3, 8, 9, 10, 11]], seq_offsets=torch.tensor([0, 4, 8]).cuda(), average=average)
        assert torch.equal(out.rewards[::2], good.rewards) and torch.equal(out.pair_loss[:1], good.pair_loss)
        assert torch.equal(out.logp[:4], good.logp[:4]) and out.grad[[0, 1, 2, 3, 8, 9, 10, 11]].isfinite().all()
    # the first sequence's beginning
    out = meo.preference_loss(x, y, ref, seq_offsets=torch.tensor([-1, 4, 8, 12, 16]).cuda(), average=average)
    assert out.rewards.isnan().tolist() == [True, False, True, False]


# ---- rounding that does not average out ---------------------------------------------

@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("vocab", [1000, 8192, 50257])
def test_log_probabilities_do_not_lean_with_the_rounding_of_1_over_t(vocab, dtype):
    """1 / T held as one fp32 number would be off by a relative d that is the
    same in every row: ln q would lean by d (z_y - m), and sums over tokens would
    collect it.  Over 48 temperatures the mean error of 768 tokens (each rounded
    by at most 5e-7, so the mean scatters by 1e-8) is fitted with that and with
    what the rounding of log2(e) / T makes of the exponents.  d scatters by 3e-8
    and z_y - m is 4 to 10: leaning would show as a slope of 1 with an error of
    0.01 to 0.03.  The bar is 0.2."""
    x, y = make(768, vocab, dtype, 11)
    adv = torch.ones(768).cuda()
    xd = x.double()
    fits = {"token_logprobs": [], "policy_loss": []}
    for k in range(48):
        tau = 0.7 + 0.9 * (k * 0.6180339887498949 % 1.0)
        z = xd / tau
        lq = torch.log_softmax(z, 1)
        want = lq.gather(1, y[:, None])[:, 0]
        m = z.amax(1)
        below = (lq.exp() * (m[:, None] - z)).sum(1).mean().item()
        at = (z.gather(1, y[:, None])[:, 0] - m).mean().item()
        c = np.log2(np.e) / tau
        lean = [(np.float64(np.float32(c)) / c - 1) * below, (np.float64(np.float32(1 / tau)) * tau - 1) * at]
        for name, got in (("token_logprobs", meo.token_logprobs(x, y, temperature=tau).logp),
                          ("policy_loss", meo.policy_loss(x, y, adv, temperature=tau, need_grad=False).logp)):
            fits[name].append([(got.double() - want).mean().item()] + lean)
    for name, rows in fits.items():
        rows = np.array(rows)
        a = np.column_stack([np.ones(48), rows[:, 1:]])
        slope = np.linalg.lstsq(a, rows[:, 0], rcond=None)[0][2]
        assert abs(slope) < 0.2, (name, slope)


# ---- what the front end allocates, refuses and tells autograd ---------------------------

def views(dtype, vocab):
    """Logits as callers cut them out of a longer tensor, and whether the
    default gradient may take the gaps' memory too."""
    def buf(*shape):
        g = torch.Generator().manual_seed(vocab)
        return (torch.randn(*shape, vocab, generator=g) * 3).to(dtype).cuda()
    return {"next token": (buf(3, 33)[:, :-1], True), "first half": (buf(3, 32)[:, :16], False),
            "all but nine": (buf(3, 33)[:, :24], False), "one of two": (buf(3, 2)[:, :1], False),
            "transposed": (buf(9, 3).transpose(0, 1), False), "whole": (buf(3, 9), False), "flat": (buf(9), False),
            "repeated": (buf(1, 9).expand(3, 9, vocab), False)}


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("vocab", [64, 1001, 50257])
def test_the_default_gradient_of_any_view(vocab, dtype):
    """Right, and no larger than the logits' rows but for the few rows that a
    next-token view leaves out."""
    for name, (x, gaps) in views(dtype, vocab).items():
        shape = x.shape[:-1]
        tokens = shape.numel()
        g = torch.Generator().manual_seed(2)
        y = torch.randint(0, vocab, shape, generator=g).cuda()
        d = torch.randn(shape, generator=g).cuda()
        xn, yn, dn = f64(x).reshape(tokens, vocab), y.cpu().numpy().reshape(-1), flat(d)
        r = meo.token_logprobs(x, y)
        pol = o.policy(xn, yn, dn)
        for got, ref, lead in ((meo.token_logprobs_backward(x, y, r.stats, d), o.logprobs_grad(xn, yn, dn), dn),
                               (meo.policy_loss(x, y, d).grad, pol[3], pol[4])):
            assert got.shape == x.shape, name
            check_grad(f64(got).reshape(tokens, vocab), ref, lead, vocab, dtype)
            rows = got.untyped_storage().nbytes() / (vocab * got.element_size())
            assert rows <= tokens + (len(shape) * 4 if gaps else 0) + 1, (name, rows)


def test_autograd_sees_that_the_logits_were_written():
    """A model whose last operation keeps its output gets an error, not the
    gradients of other values; one that does not, its gradients."""
    y = torch.tensor([[1, 2], [3, -100]]).cuda()
    a = torch.ones(2, 2).cuda()
    ids = torch.tensor([[[1, 5], [2, 6]], [[3, 7], [4, 8]]]).cuda()
    t = torch.tensor([1.0, 2.0]).cuda().expand(2, 2, 2)
    calls = [lambda x, g: meo.policy_loss(x, y, a, grad=g), lambda x, g: meo.preference_loss(x, y, grad=g),
             lambda x, g: meo.distill_loss(x, ids, t, grad=g),
             lambda x, g: types.SimpleNamespace(grad=meo.token_logprobs_backward(x, y, meo.token_logprobs(x, y).stats, a,
                                                                                 grad=g))]
    weight = torch.randn(11, 6, generator=torch.Generator().manual_seed(1)).cuda()
    hidden = torch.randn(2, 2, 6, generator=torch.Generator().manual_seed(2)).cuda()
    for call in calls:
        for cap in (False, True):
            def logits():
                w = weight.clone().requires_grad_(True)
                x = torch.nn.functional.linear(hidden, w)
                return w, torch.tanh(x) if cap else x
            w, x = logits()
            x.backward(call(x.detach(), None).grad)
            want = w.grad
            w, x = logits()
            out = call(x.detach(), x.detach())
            if cap:
                with pytest.raises(RuntimeError, match="modified by an inplace operation"):
                    x.backward(out.grad)
            else:
                x.backward(out.grad)
                assert torch.equal(w.grad, want)
    with torch.inference_mode():  # tensors without a version
        x = torch.zeros(4, 10, device="cuda")
        assert meo.policy_loss(x, y.view(-1), a.view(-1), grad=x).grad.isfinite().all()


def test_a_stream_of_another_device_is_refused():
    x, y = make(4, 10, BF16)
    a = torch.zeros(4).cuda()
    other = types.SimpleNamespace(device=torch.device("cuda", 1), device_index=1)
    for call in (lambda: meo.token_logprobs(x, y, stream=other), lambda: meo.policy_loss(x, y, a, stream=other),
                 lambda: meo.token_logprobs_backward(x, y, torch.zeros(4, 2).cuda(), a, stream=other),
                 lambda: meo.preference_loss(x[:, None], y[:, None], stream=other),
                 lambda: meo.distill_loss(x, y[:, None], a[:, None], stream=other)):
        with pytest.raises(ValueError, match="stream"):
            call()
    assert meo.policy_loss(x, y, a, stream=torch.cuda.current_stream()).loss.isfinite()


def test_streams_that_come_and_go():
    """A call for few tokens ends by a counter that is its stream's alone: a
    stream destroyed with its call still waiting, new ones that may get its
    handle, and more streams than there are counters."""
    from memory_efficient_optimizer_gb300 import binding as B
    cu = ctypes.CDLL("libcuda.so.1")
    tokens, vocab = 40, 500
    x, y = make(tokens, vocab, FP32, 3)
    adv = per_token(tokens, 4)
    want = meo.policy_loss(x, y, adv, need_grad=False).loss
    n = B.loss_workspace_size(tokens)
    calls = 1200
    loss = torch.full((calls,), float("nan"), device="cuda")
    work = torch.empty(calls, (n + 255) // 256 * 256, dtype=torch.uint8, device="cuda")
    logits = B.loss_logits(x.data_ptr(), B.ADAF_FLOAT32, 1, tokens, vocab, 0, vocab, 1.0)
    targets = B.loss_targets(B.loss_rows(y.data_ptr(), 0, 1), B.LOSS_INT64, -100)
    none = B.loss_rows(None, 0, 0)
    args = B.loss_policy_args(B.loss_rows(adv.data_ptr(), 0, 1), none, none, none, 0.2, 0.2, 0.0)
    torch.cuda.synchronize()
    handles = set()
    for k in range(calls):
        stream = ctypes.c_void_p()
        assert cu.cuStreamCreate(ctypes.byref(stream), 1) == 0
        handles.add(stream.value)
        if k % 50 == 0:
            with torch.cuda.stream(torch.cuda.ExternalStream(stream.value)):
                torch.cuda._sleep(2000000)
        B.loss_policy(logits, targets, args, B.loss_grad(None, 0, 0, 1.0), loss[k].data_ptr(), None, None,
                      work[k].data_ptr(), n, stream.value)
        assert cu.cuStreamDestroy_v2(stream) == 0
    torch.cuda.synchronize()
    assert torch.equal(loss, want.expand(calls)), (len(handles), loss[loss != want][:4])


def test_a_test_of_stalled_copies_stays_in_its_thread():
    from memory_efficient_optimizer_gb300 import binding as B
    x, y = make(3, 40000, BF16, 4)
    adv = per_token(3, 1)
    want = meo.policy_loss(x, y, adv)
    torch.cuda.synchronize()
    got = []
    B.loss_debug_stall_copies(True)
    try:
        other = threading.Thread(target=lambda: got.append(meo.policy_loss(x, y, adv)))
        other.start()
        other.join()
    finally:
        B.loss_debug_stall_copies(False)
    torch.cuda.synchronize()
    assert torch.equal(got[0].loss, want.loss) and torch.equal(got[0].grad, want.grad)


# ---- every word, and every row of many -------------------------------------------------

def check_words(got, ref, x, y, d, dtype, coef=0.0, d_rel=0.0, tau=1.0):
    """The gradient d (1[j = y] - q) word by word: off the target relative to d q,
    which has q's error (6 ds) and d's (`d_rel`, or `coef` of d absolutely); at
    the target, where 1 - q cancels, 3 ds of d more."""
    vocab = ref.shape[1]
    q = np.exp(np.stack([o.log_softmax(row / tau) for row in f64(x)]))
    q[y < 0] = 0.0
    rows = np.flatnonzero(y >= 0)
    part = q.copy()
    part[rows, y[rows]] = 1 - q[rows, y[rows]]
    bar = coef * part + 1e-37
    bar[rows, y[rows]] += 3 * ds(vocab) * np.abs(d[rows])
    check("grad", got, ref, bar, 6 * ds(vocab) + d_rel + (2 ** -8 if dtype is BF16 else 4 * U))


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("vocab", [33, 1000, 4099, 8193, 20011, 50257, 128256, 600011])
def test_gradients_word_by_word(vocab, dtype):
    x, y = make(6, vocab, dtype, vocab + 6, ignore=(2,))
    xn, yn = f64(x), y.cpu().numpy()
    d = per_token(6, 3)
    r = meo.token_logprobs(x, y, temperature=1.3)
    back = meo.token_logprobs_backward(x, y, r.stats, d, temperature=1.3)
    check_words(f64(back), o.logprobs_grad(xn, yn, f64(d), 1.3), x, yn, f64(d) / 1.3, dtype, tau=1.3)
    logp = o.token_logprobs(xn, yn)
    old = torch.tensor(np.float32(logp - np.array([0.1, 0.6, 0, -0.5, -0.05, 0.1]))).cuda()
    ref = torch.tensor(np.float32(logp + np.array([0.3, -0.2, 0, 0.5, -0.4, 0.01]))).cuda()
    out = meo.policy_loss(x, y, d, old, ref, kl_coef=0.05)
    n = o.policy(xn, yn, f64(d), f64(old), f64(ref), kl_coef=0.05)
    # -r A + kl (1 - exp(ref - logp)): each part has the absolute error of logp
    err = ds(vocab) + 4 * U * (2 * 40 + 40)
    part = 1.5 * (2 * np.abs(f64(d)) + 0.05 * 2) * err / 5
    check_words(f64(out.grad), n[3], x, yn, n[4], dtype, coef=part[:, None])
    at = torch.tensor([0, 2, 4, 5, 6]).cuda()
    out = meo.preference_loss(x, y, ref, seq_offsets=at, beta=0.3)
    n = o.preference(xn, yn, [(0, 2), (2, 4), (4, 5), (5, 6)], f64(ref), beta=0.3)
    # the coefficient moves by beta^2 / 4 of h's error, over two pairs
    check_words(f64(out.grad), n[4], x, yn, n[5], dtype, coef=0.3 ** 2 / 4 / 2 * 4 * err)


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("vocab,k", [(33, 8), (1000, 20), (8193, 64), (20011, 319), (50257, 320), (128256, 64), (131073, 1024),
                                     (600011, 20)])
@pytest.mark.parametrize("tau,rest", [(1.0, True), (2.0, True), (0.7, False)])
def test_distill_gradient_word_by_word(vocab, k, tau, rest, dtype):
    x, ids, t, lse = far_student(vocab, k, tau, 0, dtype)
    lse = lse if rest else None
    check_distill_words(meo.distill_loss(x, ids, t, lse, temperature=tau), x, ids, t, lse, tau, dtype)


MANY = [(2500, 1001, 9, BF16), (2500, 4099, 20, FP32), (2000, 20001, 300, FP32), (1500, 50257, 64, BF16), (900, 50257, 400, FP32),
        (700, 128257, 64, BF16)]


@pytest.mark.parametrize("tokens,vocab,k,dtype", MANY)
def test_many_rows_in_place(tokens, vocab, k, dtype):
    """Rows that share 16-byte granules with their neighbours, several to each
    cluster, overwritten while the next ones are being copied."""
    from test_gpu_losses import distill_inputs
    x, y = make(tokens, vocab, dtype, 7, ignore=range(3, tokens, 7))
    d = per_token(tokens, 5)
    ids, t = distill_inputs(tokens, vocab, k, 8)
    lse = torch.logsumexp(t, 1) + 0.2
    for call in (lambda v, g: meo.policy_loss(v, y, d, grad=g),
                 lambda v, g: meo.distill_loss(v, ids, t, lse, mask=y != -100, grad=g)):
        want = call(x, None)
        for _ in range(3):
            z = x.clone()
            got = call(z, z)
            assert torch.equal(z, want.grad) and torch.equal(got.token_loss, want.token_loss)
    r = meo.token_logprobs(x, y)
    want = meo.token_logprobs_backward(x, y, r.stats, d)
    z = x.clone()
    assert torch.equal(meo.token_logprobs_backward(z, y, r.stats, d, grad=z), want)
    at = torch.tensor([0, tokens // 3, tokens]).cuda()
    want = meo.preference_loss(x, y, seq_offsets=at).grad
    z = x.clone()
    assert torch.equal(meo.preference_loss(z, y, seq_offsets=at, grad=z).grad, want)


@pytest.mark.parametrize("tokens,vocab,k,dtype", MANY)
def test_rows_of_a_large_call_are_those_of_smaller_ones(tokens, vocab, k, dtype):
    """With weights a row's results hang on no other row: bit for bit in calls
    that cut rows alike (short rows always, others from a CTA an SM on), and
    within the bars in calls of a single row."""
    from test_gpu_losses import distill_inputs
    x, y = make(tokens, vocab, dtype, 7, ignore=range(3, tokens, 7))
    d, w = per_token(tokens, 5), per_token(tokens, 6).abs()
    ids, t = distill_inputs(tokens, vocab, k, 8)
    lse = torch.logsumexp(t, 1) + 0.2
    def policy(s):
        return meo.policy_loss(x[s], y[s], d[s], weights=w[s])
    def distill(s):
        return meo.distill_loss(x[s], ids[s], t[s], lse[s], weights=w[s])
    half = tokens // 2
    for call in (policy, distill):
        whole = call(slice(0, tokens))
        for s in (slice(0, half), slice(half, tokens)):
            part = call(s)
            assert torch.equal(part.grad, whole.grad[s]) and torch.equal(part.token_loss, whole.token_loss[s])
        for row in (0, 5, half - 1, tokens - 2):
            one = call(slice(row, row + 1))
            if vocab <= 8192 // (2 if dtype is FP32 else 1) - 8:
                assert torch.equal(one.grad[0], whole.grad[row]) and torch.equal(one.token_loss[0], whole.token_loss[row])
    for row in (0, 5, tokens - 2):
        s = slice(row, row + 1)
        one, n = policy(s), o.policy(f64(x[s]), y[s].cpu().numpy(), f64(d[s]), weights=f64(w[s]))
        check_logp(f64(one.logp), n[2], vocab)
        check_words(f64(one.grad), n[3], x[s], y[s].cpu().numpy(), n[4], dtype)
        check_words(f64(policy(slice(0, tokens)).grad[s]), n[3], x[s], y[s].cpu().numpy(), n[4], dtype)
        check_distill_words(distill(s), x[s], ids[s], t[s], lse[s], 1.0, dtype, w=w[s])
