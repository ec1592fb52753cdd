"""GPU parity of the losses (include/losses.h) against their float64 oracle.

Bars, from the arithmetic (u = 2^-24, one fp32 rounding):
  * a term exp((x - m) / T): the exponent (in powers of two) is scaled once in
    fp32, 2u |z| relative, and the exponential itself is good to 2^-22; the
    terms of a row that carry its sum have |z| < 20, so 2^-22 + 40u < 3e-6.
  * the sum s: no thread adds more than max(128, vocab / 128) terms one after
    another, each addition u: below 3e-6 + u max(128, vocab / 128) =: ds.
  * logp: ds + 3u (|logp| + |x_y - m| / T), taken as ds + 4u (2 |logp| + 40).
  * gradient d (1[j = y] - q): relative 2 ds in what multiplies it (a ratio
    exp(logp - old) has the absolute error of logp), one rounding to its type
    (2^-8 for bf16 covers it), and where 1 - q cancels an absolute ds |d|.
    Distillation the same with the token's weight times T for d.
"""
import numpy as np
import pytest
import torch

import memory_efficient_optimizer_gb300 as meo
from oracle import losses as o

pytestmark = pytest.mark.gpu
U = 2.0 ** -24
BF16, FP32 = torch.bfloat16, torch.float32


@pytest.fixture(scope="module", autouse=True)
def _built():
    from memory_efficient_optimizer_gb300 import build
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    build.build()


def ds(vocab):
    return 3e-6 + U * max(128, vocab / 128)


def f64(t):
    return t.detach().double().cpu().numpy()


def flat(t):
    return f64(t).reshape(-1)


def check(name, got, ref, atol, rtol=0.0):
    got, ref = np.asarray(got, dtype=np.float64), np.asarray(ref, dtype=np.float64)
    assert got.shape == ref.shape, name
    odd = ~np.isfinite(ref)
    assert np.array_equal(np.isnan(got), np.isnan(ref)), name
    assert np.array_equal(got[odd & ~np.isnan(ref)], ref[odd & ~np.isnan(ref)]), name
    atol = np.broadcast_to(atol, ref.shape)[~odd]
    got, ref = got[~odd], ref[~odd]
    err, bound = np.abs(got - ref), atol + rtol * np.abs(ref)
    assert np.all(err <= bound), f"{name}: worst {np.max(err / np.maximum(bound, 1e-300)):.3f} of the bar"


def check_logp(got, ref, vocab):
    ok = np.where(np.isfinite(ref), np.abs(ref), 0)
    check("logp", got, ref, ds(vocab) + 4 * U * (2 * ok + 40))


def check_grad(got, ref, d, vocab, dtype):
    """d: what multiplies 1[j = y] - q of each row (already over T)."""
    lead = np.abs(d)[:, None]
    lead = np.where(np.isfinite(lead), lead, 0)
    check("grad", got, ref, 3 * ds(vocab) * lead + 1e-37, 6 * ds(vocab) + (2 ** -8 if dtype is BF16 else 4 * U))


def make(tokens, vocab, dtype, seed=0, ignore=()):
    g = torch.Generator().manual_seed(seed)
    x = torch.randn(tokens, vocab, generator=g) * 3
    y = torch.randint(0, vocab, (tokens,), generator=g)
    x[torch.arange(tokens), y] += 6 * torch.rand(tokens, generator=g)
    for t in ignore:
        y[t] = -100
    return x.to(dtype).cuda(), y.cuda()


def per_token(tokens, seed, scale=1.0):
    return (torch.randn(tokens, generator=torch.Generator().manual_seed(seed)) * scale).cuda()


VOCABS = [1, 2, 7, 8, 9, 33, 255, 256, 1000, 2047, 4099, 8192, 16385, 32000, 50257, 65537, 128256, 131073, 262147,
          600011]
DTYPES = [BF16, FP32]


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("vocab", VOCABS)
def test_token_logprobs_and_backward(vocab, dtype):
    x, y = make(5, vocab, dtype, vocab, ignore=(3,))
    d = per_token(5, 1)
    for tau in (1.0, 1.7):
        r = meo.token_logprobs(x, y, temperature=tau)
        check_logp(f64(r.logp), o.token_logprobs(f64(x), y.cpu().numpy(), tau), vocab)
        g = meo.token_logprobs_backward(x, y, r.stats, d, temperature=tau, grad_scale=0.5)
        ref = o.logprobs_grad(f64(x), y.cpu().numpy(), 0.5 * f64(d), tau)
        check_grad(f64(g), ref, 0.5 * f64(d) / tau, vocab, dtype)


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("vocab", VOCABS)
def test_policy(vocab, dtype):
    x, y = make(6, vocab, dtype, vocab + 1, ignore=(0,))
    xn, yn = f64(x), y.cpu().numpy()
    logp = o.token_logprobs(xn, yn)
    # ratios on both sides of the clip, none at its edges
    old = torch.tensor(np.float32(logp - np.array([0, 0.6, -0.5, 0.1, -0.05, 0.9]))).cuda()
    ref = torch.tensor(np.float32(logp + np.array([0, 0.3, -0.2, 0.01, 0.5, -0.4]))).cuda()
    adv = torch.tensor([1.0, 1.5, -0.7, 0.4, -1.1, -2.0]).cuda()
    out = meo.policy_loss(x, y, adv, old, ref, clip_low=0.2, clip_high=0.28, kl_coef=0.05)
    want, token, lp, grad, d = o.policy(xn, yn, f64(adv), f64(old), f64(ref), 0.2, 0.28, 0.05)
    check_logp(f64(out.logp), lp, vocab)
    err = 6 * ds(vocab) + 8 * U * 40
    check("token_loss", f64(out.token_loss), token, 4 * err, 4 * err)
    check("loss", f64(out.loss), want, 4 * err, 4 * err)
    # the ratio has logp's absolute error
    check("grad", f64(out.grad), grad, 3 * ds(vocab) * np.abs(d)[:, None] + 1e-37,
          2 * err + (2 ** -8 if dtype is BF16 else 0))
    alone = meo.policy_loss(x, y, adv, old, ref, clip_high=0.28, kl_coef=0.05, need_grad=False)
    assert alone.grad is None
    check("token_loss", f64(alone.token_loss), token, 4 * err, 4 * err)
    check("loss", f64(alone.loss), want, 4 * err, 4 * err)


@pytest.mark.parametrize("tau", [0.7, 1.0, 3.0])
def test_policy_weights_temperature_and_first_step(tau):
    x, y = make(7, 5003, BF16, 5, ignore=(6,))
    adv, w = per_token(7, 2), per_token(7, 3).abs()
    out = meo.policy_loss(x, y, adv, weights=w, temperature=tau, grad_scale=4.0)
    want, token, _, grad, d = o.policy(f64(x), y.cpu().numpy(), f64(adv), weights=f64(w), temperature=tau)
    check("loss", f64(out.loss), want, 1e-6 * np.sum(np.abs(f64(w) * token)))
    check("token_loss", f64(out.token_loss), token, 1e-6, 1e-6)
    check_grad(f64(out.grad), 4 * grad, 4 * d / tau, 5003, BF16)


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("vocab", [7, 1000, 50257, 128256, 600011])
@pytest.mark.parametrize("kind,kw", [("sigmoid", {}), ("sigmoid", dict(label_smoothing=0.1, margin=0.5)),
                                     ("hinge", {}), ("squared", dict(average=True))])
def test_preference(vocab, dtype, kind, kw):
    seqs = [(0, 3), (3, 4), (4, 4), (4, 6), (6, 9), (9, 11)]
    x, y = make(11, vocab, dtype, vocab + 2, ignore=(1, 9, 10))
    ref = per_token(11, 7, 0.3) + torch.tensor(np.float32(o.token_logprobs(f64(x), y.cpu().numpy()))).cuda()
    at = torch.tensor([0] + [b for _, b in seqs], dtype=torch.int32).cuda()
    out = meo.preference_loss(x, y, ref, seq_offsets=at, kind=kind, beta=0.3, **kw)
    want, pair, rewards, lp, grad, d = o.preference(f64(x), y.cpu().numpy(), seqs, f64(ref), beta=0.3, kind=kind, **kw)
    e = 3 * (ds(vocab) + 4 * U * 60)   # of a sequence's sum: three tokens at most
    check_logp(f64(out.logp), lp, vocab)
    check("rewards", f64(out.rewards), rewards, 0.3 * e, 4 * U)
    slope = 2 * np.sqrt(np.max(pair)) + 1 if kind == "squared" else 0.3
    check("pair_loss", f64(out.pair_loss), pair, 2 * slope * e, 4 * U)
    check("loss", f64(out.loss), want, 2 * slope * e, 4 * U)
    # the derivative of the loss moves by at most 2 (squared) or beta^2 (sigmoid) times the error of h
    lead = np.abs(d)[:, None] * 3 * ds(vocab) + 2 * 2 * e * (np.abs(d)[:, None] > 0)
    check("grad", f64(out.grad), grad, lead + 1e-37, 6 * ds(vocab) + (2 ** -8 if dtype is BF16 else 4 * U))


def test_preference_batch_layout_equals_packed():
    x, y = make(4 * 9, 1009, BF16, 3, ignore=(0, 1, 9, 20, 35))
    ref = per_token(36, 1)
    a = meo.preference_loss(x.view(4, 9, -1), y.view(4, 9), ref.view(4, 9))
    b = meo.preference_loss(x, y, ref, seq_offsets=torch.arange(0, 37, 9).cuda())
    assert torch.equal(a.loss, b.loss) and torch.equal(a.grad.view(36, -1), b.grad)
    assert torch.equal(a.pair_loss, b.pair_loss) and torch.equal(a.rewards, b.rewards)
    c = meo.preference_loss(x.view(4, 9, -1), y.view(4, 9), ref.view(4, 9), need_grad=False)
    assert c.grad is None and abs(c.loss.item() - a.loss.item()) < 1e-5


def test_preference_with_bad_offsets_answers_nan():
    x, y = make(8, 100, FP32)
    for at in ([0, 4, 3], [0, 4, 9], [-1, 4, 8]):
        out = meo.preference_loss(x, y, seq_offsets=torch.tensor(at).cuda())
        assert out.loss.isnan() and out.pair_loss.isnan().all()
    # tokens after the last sequence have no gradient
    out = meo.preference_loss(x, y, seq_offsets=torch.tensor([0, 2, 5]).cuda())
    assert out.loss.isfinite() and out.grad[:5].abs().sum(1).min() > 0 and not out.grad[5:].any()


def distill_inputs(tokens, vocab, k, seed=0, bf16=False):
    g = torch.Generator().manual_seed(seed)
    ids = torch.stack([torch.randperm(vocab, generator=g)[:k] for _ in range(tokens)])
    t = torch.randn(tokens, k, generator=g) * 2
    return ids.cuda(), (t.bfloat16() if bf16 else t).cuda()


def check_distill(out, want, token, grad, w, x, tau, vocab, dtype):
    # a term p (ln p - ln q) has an absolute error of p (ds + 8u |ln q|); |ln q| here stays below 60
    e = tau * tau * (2 * ds(vocab) + 8 * U * 60)
    check("token_loss", f64(out.token_loss).reshape(-1), token, e, 8 * U)
    check("loss", f64(out.loss), want, e * np.sum(np.abs(w)), 8 * U)
    check("grad", f64(out.grad).reshape(grad.shape), grad, 6 * ds(vocab) * tau * np.abs(w)[:, None] + 1e-37,
          2 * ds(vocab) + (2 ** -8 if dtype is BF16 else 4 * U))


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("vocab,k", [(1, 1), (2, 1), (9, 9), (300, 31), (8193, 64), (32000, 8), (50257, 257),
                                     (128256, 64), (131073, 1024), (600011, 20)])
@pytest.mark.parametrize("rest", [False, True])
def test_distill(vocab, k, dtype, rest):
    tau = 2.0 if vocab % 2 else 1.0
    x, _ = make(5, vocab, dtype, vocab)
    ids, t = distill_inputs(5, vocab, k, vocab)
    if k > 1:
        ids[1, k // 2] = -1
    ids[2] = -1
    lse = torch.logsumexp(t / tau, 1) + torch.tensor([0.01, 0.1, 0.5, 1.0, 3.0]).cuda() if rest else None
    mask = torch.tensor([True, True, True, False, True]).cuda()
    out = meo.distill_loss(x, ids, t, lse, mask=mask, temperature=tau)
    n = o.distill(f64(x), ids.cpu().numpy(), f64(t), None if lse is None else f64(lse), mask.cpu().numpy(),
                  temperature=tau)
    check_distill(out, n[0], n[1], n[2], n[3], x, tau, vocab, dtype)
    assert not out.grad[3].any() and out.token_loss[3] == 0
    alone = meo.distill_loss(x, ids, t, lse, mask=mask, temperature=tau, need_grad=False)
    assert alone.grad is None
    check("loss", f64(alone.loss), n[0], tau * tau * (2 * ds(vocab) + 8 * U * 60), 8 * U)


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("tokens,vocab,k", [(2400, 9001, 319), (2400, 9001, 320), (250, 128256, 1000), (250, 131073, 1024)])
def test_distill_long_lists_over_many_rows(tokens, vocab, k, dtype):
    """Each cluster takes several rows, some of them not counted: lists of 320
    entries and more are made by two warps in turn, those of about 1000 leave
    the ring one row's places."""
    x, _ = make(tokens, vocab, dtype, 7)
    ids, t = distill_inputs(tokens, vocab, k, 8)
    lse = torch.logsumexp(t, 1) + 0.2
    ids[1, 5:300] = -1
    ids[2] = -1
    mask = torch.rand(tokens, generator=torch.Generator().manual_seed(9)) < 0.8
    out = meo.distill_loss(x, ids, t, lse, mask=mask.cuda())
    n = o.distill(f64(x), ids.cpu().numpy(), f64(t), f64(lse), mask.numpy())
    check_distill(out, n[0], n[1], n[2], n[3], x, 1.0, vocab, dtype)
    assert not out.grad[~mask.cuda()].any()
    again = meo.distill_loss(x, ids, t, lse, mask=mask.cuda())
    assert torch.equal(again.loss, out.loss) and torch.equal(again.grad, out.grad)


def test_a_copy_that_never_lands_ends_a_call_with_long_lists():
    from memory_efficient_optimizer_gb300 import binding as B
    x, _ = make(600, 40000, BF16, 4)
    ids, t = distill_inputs(600, 40000, 400, 3)
    want = meo.distill_loss(x, ids, t)
    torch.cuda.synchronize()
    B.loss_debug_stall_copies(True)
    try:
        out = meo.distill_loss(x, ids, t)
    finally:
        B.loss_debug_stall_copies(False)
    torch.cuda.synchronize()
    assert out.loss.isnan()
    again = meo.distill_loss(x, ids, t)
    assert torch.equal(again.loss, want.loss) and torch.equal(again.grad, want.grad)


def test_distill_types_weights_and_strides():
    x, _ = make(6, 777, BF16, 4)
    ids, t = distill_inputs(6, 777, 12, 1, bf16=True)
    w = per_token(6, 5).abs()
    wide_ids, wide_t = torch.full((6, 20), -7).cuda(), torch.zeros(6, 15, dtype=BF16).cuda()
    wide_ids[:, 3:15], wide_t[:, 1:13] = ids, t
    out = meo.distill_loss(x.view(2, 3, -1), wide_ids[:, 3:15].view(2, 3, 12), wide_t[:, 1:13].view(2, 3, 12),
                           weights=w.view(2, 3))
    same = meo.distill_loss(x, ids.int(), t, weights=w)
    assert torch.equal(out.loss, same.loss) and torch.equal(out.grad.view(6, -1), same.grad)
    n = o.distill(f64(x), ids.cpu().numpy(), f64(t), weights=f64(w))
    check_distill(out, n[0], n[1], n[2], n[3], x, 1.0, 777, BF16)


def test_distill_small_rest_keeps_its_precision():
    """The student puts nearly everything on the listed words: the rest is the
    sum of the other words' terms, not 1 minus the listed ones'."""
    x = torch.full((1, 1000), -12.0)
    x[0, 5], x[0, 700] = 9.0, 8.5
    ids, t = torch.tensor([[5, 700]]).cuda(), torch.tensor([[2.0, 1.0]]).cuda()
    lse = torch.logsumexp(t, 1) + 0.2
    out = meo.distill_loss(x.cuda(), ids, t, lse)
    n = o.distill(f64(x), ids.cpu().numpy(), f64(t), f64(lse))
    check_distill(out, n[0], n[1], n[2], n[3], x, 1.0, 1000, FP32)


# ---- layouts -------------------------------------------------------------------

LAYOUTS = ["contiguous", "shifted", "transposed", "padded_rows", "offset_base", "repeated"]


def lay_out(kind, batch, seq, vocab, dtype):
    """A [batch, seq, vocab] view of a larger sentinel-filled buffer."""
    if kind == "contiguous":
        buf = torch.full((batch, seq, vocab), 77.0)
        return buf.to(dtype).cuda(), lambda b: b
    if kind == "shifted":
        buf = torch.full((batch, seq + 1, vocab), 77.0)
        return buf.to(dtype).cuda(), lambda b: b[:, :-1]
    if kind == "transposed":
        buf = torch.full((seq, batch, vocab), 77.0)
        return buf.to(dtype).cuda(), lambda b: b.transpose(0, 1)
    if kind == "padded_rows":
        buf = torch.full((batch, seq, vocab + 5), 77.0)
        return buf.to(dtype).cuda(), lambda b: b[..., 2:vocab + 2]
    if kind == "offset_base":
        buf = torch.full((batch * seq * vocab + 9,), 77.0)
        return buf.to(dtype).cuda(), lambda b: b[3:3 + batch * seq * vocab].view(batch, seq, vocab)
    buf = torch.full((seq, vocab), 77.0)
    return buf.to(dtype).cuda(), lambda b: b[None].expand(batch, seq, vocab)


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("vocab", [5, 64, 1001, 4100, 50257])
@pytest.mark.parametrize("grad_layout", LAYOUTS[:-1])
@pytest.mark.parametrize("layout", LAYOUTS)
def test_any_layout_of_logits_and_gradient(layout, grad_layout, vocab, dtype):
    """Right whatever the strides and alignments are, and nothing written
    outside the gradient's rows."""
    batch, seq = 2, 3
    buf, view = lay_out(layout, batch, seq, vocab, dtype)
    x = view(buf)
    g = torch.Generator().manual_seed(1)
    if layout == "repeated":
        buf.copy_(torch.randn(seq, vocab, generator=g) * 3)
    else:
        x.copy_(torch.randn(batch, seq, vocab, generator=g) * 3)
    y = torch.randint(0, vocab, (batch, seq), generator=g).cuda()
    y[0, 1] = -100
    adv = torch.randn(batch, 1, generator=g).cuda().expand(batch, seq)
    xn, yn, an = f64(x).reshape(-1, vocab), y.cpu().numpy().reshape(-1), f64(adv).reshape(-1)
    n = o.policy(xn, yn, an)
    gbuf, gview = lay_out(grad_layout, batch, seq, vocab, dtype)
    out = meo.policy_loss(x, y, adv, grad=gview(gbuf))
    check_logp(f64(out.logp).reshape(-1), n[2], vocab)
    check_grad(f64(out.grad).reshape(-1, vocab), n[3], n[4], vocab, dtype)
    gview(gbuf).fill_(77.0)
    assert torch.all(gbuf == 77.0)
    # the backward pass of the log-probabilities, and distillation
    r = meo.token_logprobs(x, y)
    check_logp(f64(r.logp).reshape(-1), n[2], vocab)
    back = meo.token_logprobs_backward(x, y, r.stats, adv, grad=gview(gbuf))
    check_grad(f64(back).reshape(-1, vocab), o.logprobs_grad(xn, yn, an), an, vocab, dtype)
    gview(gbuf).fill_(77.0)
    assert torch.all(gbuf == 77.0)
    ids, t = distill_inputs(6, vocab, 4, vocab)
    lse = torch.logsumexp(t, 1) + 0.3
    out = meo.distill_loss(x, ids.view(2, 3, 4), t.view(2, 3, 4), lse.view(2, 3), grad=gview(gbuf))
    n = o.distill(xn, ids.cpu().numpy(), f64(t), f64(lse))
    check_distill(out, n[0], n[1].reshape(-1), n[2], n[3], x, 1.0, vocab, dtype)
    gview(gbuf).fill_(77.0)
    assert torch.all(gbuf == 77.0)


@pytest.mark.parametrize("layout", ["contiguous", "shifted", "padded_rows", "offset_base"])
@pytest.mark.parametrize("vocab", [9, 1001, 50257, 128256, 600011])
@pytest.mark.parametrize("dtype", DTYPES)
def test_gradient_in_place_of_the_logits(vocab, dtype, layout):
    batch, seq = 2, 2
    buf, view = lay_out(layout, batch, seq, vocab, dtype)
    x = view(buf)
    x.copy_(torch.randn(batch, seq, vocab, generator=torch.Generator().manual_seed(vocab)) * 3)
    keep = x.clone()
    y = torch.tensor([[0, vocab - 1], [-100, vocab // 2]]).cuda()
    adv = torch.tensor([[1.0, -1.0], [1.0, 0.5]]).cuda()
    ids = torch.stack([torch.randperm(vocab)[:5] for _ in range(4)]).view(2, 2, 5).cuda()
    t = torch.randn(2, 2, 5).cuda()
    lse = torch.logsumexp(t, -1) + 0.5
    at = view(torch.zeros_like(buf))  # another buffer of the same layout, for the comparison
    for run in (lambda v, g: meo.policy_loss(v, y, adv, grad=g).grad,
                lambda v, g: meo.preference_loss(v, y, adv, grad=g).grad,
                lambda v, g: meo.token_logprobs_backward(v, y, meo.token_logprobs(v, y).stats, adv, grad=g),
                lambda v, g: meo.distill_loss(v, ids, t, lse, grad=g).grad):
        x.copy_(keep)
        want = run(x, at).clone()
        got = run(x, x)
        assert got.data_ptr() == x.data_ptr() and torch.equal(x, want)
    x.fill_(77.0)
    assert torch.all(buf == 77.0)


def test_strided_per_token_arguments():
    b, s, v = 3, 5, 600
    x, y = make(b * s, v, BF16, 9, ignore=(4,))
    x, y = x.view(b, s, v), y.view(b, s)
    ids = torch.full((b, s + 1), -1).cuda()
    ids[:, 1:] = y
    adv = torch.randn(b).cuda()
    old = torch.randn(s, b).cuda() - 6
    ref = torch.randn(b, 2 * s).cuda() - 6
    out = meo.policy_loss(x, ids[:, 1:], adv[:, None].expand(b, s), old.t(), ref[:, ::2], kl_coef=0.1)
    same = meo.policy_loss(x, y.int(), adv[:, None].repeat(1, s), old.t().contiguous(), ref[:, ::2].contiguous(),
                           kl_coef=0.1)
    assert torch.equal(out.loss, same.loss) and torch.equal(out.grad, same.grad)


# ---- values where it can go wrong --------------------------------------------------

def lowest(dtype):
    return torch.finfo(dtype).min


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("vocab", [5, 300, 20011, 128256])
def test_masked_words_and_lowest_values(vocab, dtype):
    x, y = make(6, vocab, dtype, 2)
    y[:] = 0
    x[0, 1:] = -float("inf")                 # one word left
    x[1, 1:] = lowest(dtype)                 # the same with the lowest value
    x[2] = lowest(dtype)                     # every word the same: uniform
    x[3, : vocab // 2] = -float("inf")       # the target itself is masked
    x[4, vocab // 3:] = -float("inf")        # whole stretches of the row
    x[5] = -x[5].abs() - 1e4 * (dtype is FP32)
    adv = torch.ones(6).cuda()
    r = meo.token_logprobs(x, y)
    want = o.token_logprobs(f64(x), y.cpu().numpy())
    assert want[0] == 0 and want[1] == 0 and np.isneginf(want[3]) and abs(want[2] + np.log(vocab)) < 1e-9
    check_logp(f64(r.logp), want, vocab)
    g = meo.token_logprobs_backward(x, y, r.stats, adv)
    check_grad(f64(g), o.logprobs_grad(f64(x), y.cpu().numpy(), f64(adv)), f64(adv), vocab, dtype)
    keep = [0, 1, 2, 4, 5]
    out = meo.policy_loss(x[keep], y[keep], adv[keep])
    n = o.policy(f64(x[keep]), y[keep].cpu().numpy(), f64(adv[keep]))
    check_grad(f64(out.grad), n[3], n[4], vocab, dtype)


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("vocab", [5, 300, 9000, 128256])
@pytest.mark.parametrize("tau", [1e-3, 1e-2, 1e20])
def test_large_logits_and_far_temperatures(vocab, tau, dtype):
    """Logits whose product with 1 / T leaves fp32: a row of equal ones, one
    word far above the others, and two words a little apart."""
    x = torch.full((4, vocab), 2e36, dtype=dtype).cuda()
    x[1, 2:] = -3e38
    x[2, 0] = 3e36
    x[3] = 7.0 if tau < 1 else -1e38
    y = torch.zeros(4, dtype=torch.int64).cuda()
    adv = torch.tensor([1.0, -1.0, 2.0, 0.5]).cuda()
    xn, yn, an = f64(x), y.cpu().numpy(), f64(adv)
    r = meo.token_logprobs(x, y, temperature=tau)
    check_logp(f64(r.logp), o.token_logprobs(xn, yn, tau), vocab)
    g = meo.token_logprobs_backward(x, y, r.stats, adv, temperature=tau)
    check_grad(f64(g), o.logprobs_grad(xn, yn, an, tau), an / tau, vocab, dtype)
    out = meo.policy_loss(x, y, adv, temperature=tau)
    n = o.policy(xn, yn, an, temperature=tau)
    check_logp(f64(out.logp), n[2], vocab)
    check_grad(f64(out.grad), n[3], n[4] / tau, vocab, dtype)


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("vocab", [5, 300, 128256])
def test_rows_without_a_distribution_answer_nan_alone(vocab, dtype):
    x, y = make(6, vocab, dtype, 3)
    x[0, vocab // 2] = float("nan")
    x[1, vocab // 2] = float("inf")
    x[2] = -float("inf")
    y[3] = vocab
    y[4] = -1
    y[1] = 0
    adv = torch.ones(6).cuda()
    r = meo.token_logprobs(x, y)
    assert r.logp[:5].isnan().all() and r.logp[5].isfinite()
    g = meo.token_logprobs_backward(x, y, r.stats, adv)
    assert g[:5].isnan().all() and g[5].isfinite().all()
    out = meo.policy_loss(x, y, adv)
    assert out.loss.isnan() and out.token_loss[:5].isnan().all() and out.token_loss[5].isfinite()
    assert out.grad[:5].isnan().all() and out.grad[5].isfinite().all()
    # the same rows ignored: nothing of them shows
    y[:5] = -100
    for res in (meo.policy_loss(x, y, adv), meo.preference_loss(x, y, seq_offsets=torch.tensor([0, 5, 6]).cuda())):
        assert res.loss.isfinite() and not res.grad[:5].any() and res.grad[5].isfinite().all()
        assert not res.logp[:5].any()


def test_distill_bad_data_answers_nan_alone():
    x, _ = make(6, 500, FP32, 1)
    ids, t = distill_inputs(6, 500, 6, 2)
    ids[0, 3] = 500
    ids[1, 0] = -2
    ids[2, 5] = ids[2, 1]
    t[3, 2] = float("nan")
    t[4, 1] = -float("inf")      # no mass: allowed
    for lse in (None, torch.logsumexp(t.nan_to_num(0), 1) + 0.3):
        out = meo.distill_loss(x, ids, t, lse)
        assert out.token_loss[:4].isnan().all() and out.token_loss[4:].isfinite().all()
        assert out.grad[:4].isnan().all() and out.grad[4:].isfinite().all()
    mask = torch.tensor([False] * 4 + [True] * 2).cuda()
    out = meo.distill_loss(x, ids, t, mask=mask)
    n = o.distill(f64(x[4:]), ids[4:].cpu().numpy(), f64(t[4:]))
    check_distill(meo.distill_loss(x[4:], ids[4:], t[4:]), n[0], n[1], n[2], n[3], x, 1.0, 500, FP32)
    assert out.loss.isfinite() and not out.grad[:4].any()


def test_nothing_counted_is_zero():
    x, y = make(4, 1000, BF16)
    y[:] = -100
    ids, t = distill_inputs(4, 1000, 3)
    none = torch.zeros(4, dtype=torch.bool).cuda()
    for res in (meo.policy_loss(x, y, per_token(4, 1)), meo.distill_loss(x, ids, t, mask=none)):
        assert res.loss == 0 and not res.grad.any() and not res.token_loss.any()
    res = meo.preference_loss(x, y, seq_offsets=torch.tensor([0, 2, 4]).cuda(), average=True)
    assert abs(res.loss.item() - np.log(2)) < 1e-6 and not res.grad.any() and not res.rewards.any()


@pytest.mark.parametrize("shape", [(0, 50), (2, 0, 50), (0, 3, 50)])
def test_no_tokens(shape):
    x = torch.empty(shape, dtype=BF16).cuda()
    y = torch.empty(shape[:-1], dtype=torch.int64).cuda()
    a = torch.empty(shape[:-1]).cuda()
    r = meo.token_logprobs(x, y)
    assert r.logp.shape == y.shape and meo.token_logprobs_backward(x, y, r.stats, a).shape == shape
    out = meo.policy_loss(x, y, a)
    assert out.loss == 0 and out.grad.shape == shape
    ids = torch.empty(*shape[:-1], 4, dtype=torch.int64).cuda()
    out = meo.distill_loss(x, ids, ids.float())
    assert out.loss == 0 and out.grad.shape == shape
    if shape[0] == 2:
        assert abs(meo.preference_loss(x, y).loss.item() - np.log(2)) < 1e-6


def test_offsets_past_32_bits():
    """Rows whose element offsets do not fit in 32 bits, forward and back."""
    vocab, far = 1003, (1 << 32) + 11
    buf = torch.zeros(far + 3 * vocab, dtype=BF16, device="cuda")
    x = buf.as_strided((2, vocab), (far, 1))
    x.copy_(torch.randn(2, vocab) * 3)
    y = torch.tensor([5, 1002]).cuda()
    adv = torch.tensor([1.0, -2.0]).cuda()
    xn = f64(x)
    ids, t = distill_inputs(2, vocab, 7)
    out = meo.distill_loss(x, ids, t)
    n = o.distill(xn, ids.cpu().numpy(), f64(t))
    check_distill(out, n[0], n[1], n[2], n[3], x, 1.0, vocab, BF16)
    out = meo.policy_loss(x, y, adv, grad=x)
    n = o.policy(xn, y.cpu().numpy(), f64(adv))
    check_logp(f64(out.logp), n[2], vocab)
    check_grad(f64(x), n[3], n[4], vocab, BF16)
    assert not buf[vocab:far].any() and not buf[far + vocab:].any()


@pytest.mark.parametrize("tokens", [1, 2, 151, 153, 1025, 5000])
def test_many_tokens_of_a_small_vocabulary(tokens):
    x, y = make(tokens, 97, BF16, tokens)
    adv = per_token(tokens, 1)
    out = meo.policy_loss(x, y, adv)
    n = o.policy(f64(x), y.cpu().numpy(), f64(adv))
    check("loss", f64(out.loss), n[0], 1e-6 * np.mean(np.abs(n[1])))
    check_grad(f64(out.grad), n[3], n[4], 97, BF16)


def test_large_batch_rows_agree_with_single_ones():
    """A row's bits do not depend on which other rows are in the call, for
    calls that split rows alike; and runs agree bit for bit."""
    x, y = make(640, 50257, BF16, 8, ignore=range(0, 640, 3))
    adv = per_token(640, 1)
    a, b = meo.policy_loss(x, y, adv), meo.policy_loss(x, y, adv)
    assert torch.equal(a.loss, b.loss) and torch.equal(a.grad, b.grad) and torch.equal(a.logp, b.logp)
    n = o.token_logprobs(f64(x[:40]), y[:40].cpu().numpy())
    check_logp(f64(a.logp[:40]), n, 50257)
    p, q = (meo.preference_loss(x.view(10, 64, -1), y.view(10, 64)) for _ in range(2))
    assert torch.equal(p.loss, q.loss) and torch.equal(p.grad, q.grad) and torch.equal(p.rewards, q.rewards)


def test_streams_and_graphs():
    x, y = make(64, 32000, BF16, 1, ignore=(5,))
    adv = per_token(64, 1)
    ids, t = distill_inputs(64, 32000, 16)
    ref = per_token(64, 2) - 5
    runs = [lambda s=None: meo.policy_loss(x, y, adv, stream=s),
            lambda s=None: meo.distill_loss(x, ids, t, stream=s),
            lambda s=None: meo.preference_loss(x.view(2, 32, -1), y.view(2, 32), ref.view(2, 32), stream=s)]
    want = [r() for r in runs]
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    for r, w in zip(runs, want):
        got = [r(side) for _ in range(3)]
        torch.cuda.current_stream().wait_stream(side)
        for q in got:
            assert torch.equal(q.loss, w.loss) and torch.equal(q.grad, w.grad)
    for r, w in zip(runs, want):
        r()
        torch.cuda.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            out = r()
        for _ in range(2):
            graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(out.loss, w.loss) and torch.equal(out.grad, w.grad)

def test_calls_for_few_tokens_on_several_streams_and_in_graphs():
    """Calls for few tokens end by a counter that the library keeps for the
    stream; captured ones by their workspace's.  Interleaved, each is right."""
    cases = []
    for tokens in (1, 7, 200, 512, 513):
        x, y = make(tokens, 300, BF16, tokens, ignore=(0,) if tokens > 1 else ())
        adv = per_token(tokens, 1)
        n = o.policy(f64(x), y.cpu().numpy(), f64(adv))
        cases.append((x, y, adv, n))
    streams = [torch.cuda.Stream() for _ in range(3)]
    graphs = []
    for x, y, adv, n in cases[:4]:
        meo.policy_loss(x, y, adv)
        torch.cuda.synchronize()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            out = meo.policy_loss(x, y, adv)
        graphs.append((g, out, n))
    torch.cuda.synchronize()
    got = []
    for k in range(30):
        x, y, adv, n = cases[k % 5]
        got.append((meo.policy_loss(x, y, adv, stream=streams[k % 3]).loss, n))
        if k % 4 == 0:
            g, out, n = graphs[k // 4 % 4]
            with torch.cuda.stream(streams[(k + 1) % 3]):
                g.replay()
    torch.cuda.synchronize()
    for loss, n in got + [(out.loss, n) for _, out, n in graphs]:
        check("loss", f64(loss), n[0], 2e-6 * np.mean(np.abs(n[1])))


def test_a_copy_that_never_lands_ends_the_call():
    """Every wait in the kernel is bounded: with the copies expected but not
    made the call ends, the loss says so, and the next call is right."""
    from memory_efficient_optimizer_gb300 import binding as B
    for tokens, vocab in ((3, 40000), (3, 128256), (600, 40000)):  # short rows take no copies
        x, y = make(tokens, vocab, BF16, 4)
        adv = per_token(tokens, 1)
        ids, t = distill_inputs(tokens, vocab, 8, 3)
        calls = [lambda: meo.policy_loss(x, y, adv), lambda: meo.distill_loss(x, ids, t)]
        want = [c() for c in calls]
        for c, w in zip(calls, want):
            torch.cuda.synchronize()
            B.loss_debug_stall_copies(True)
            try:
                out = c()
            finally:
                B.loss_debug_stall_copies(False)
            torch.cuda.synchronize()
            assert out.loss.isnan()
            again = c()
            assert torch.equal(again.loss, w.loss) and torch.equal(again.grad, w.grad)


def test_front_end_refusals():
    x, y = make(4, 10, BF16)
    a = torch.zeros(4).cuda()
    bad = [lambda: meo.policy_loss(x, y.float(), a), lambda: meo.policy_loss(x, y[:3], a),
           lambda: meo.policy_loss(x, y.cpu(), a), lambda: meo.policy_loss(x, y, a.double()),
           lambda: meo.policy_loss(x, y, a[:2]), lambda: meo.policy_loss(x, y, a, kl_coef=0.1),
           lambda: meo.policy_loss(x, y, a, clip_low=-1.0), lambda: meo.policy_loss(x, y, a, temperature=0.0),
           lambda: meo.policy_loss(x, y, a, grad=torch.empty_like(x, dtype=FP32)),
           lambda: meo.policy_loss(x, y, a, grad=x, need_grad=False), lambda: meo.policy_loss(x, y, a, grad=x[:2]),
           lambda: meo.policy_loss(x, y, a, grad=x[:1].expand(4, 10)),
           lambda: meo.policy_loss(x[:, :8], y.clamp(max=7), a, grad=x[:, 2:]),
           lambda: meo.preference_loss(x, y), lambda: meo.preference_loss(x, y, kind="other", seq_offsets=y[:3]),
           lambda: meo.preference_loss(x, y, seq_offsets=y[:2]), lambda: meo.preference_loss(x, y, seq_offsets=a[:3]),
           lambda: meo.preference_loss(x[:3, None], y[:3, None]),
           lambda: meo.distill_loss(x, y, a), lambda: meo.distill_loss(x, y[:, None].float(), a[:, None]),
           lambda: meo.distill_loss(x, y[:, None], a[:, None].half()),
           lambda: meo.distill_loss(x, y[:, None], a[:, None].expand(4, 2)),
           lambda: meo.distill_loss(x, y[:, None], a[:, None], mask=a),
           lambda: meo.distill_loss(x, y[:, None][:, :0], a[:, None][:, :0]),
           lambda: meo.token_logprobs_backward(x, y, a, a)]
    for call in bad:
        with pytest.raises(ValueError):
            call()


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("vocab", [300, 40000])
def test_parts_of_a_row_on_both_sides_of_the_exponent_forms(vocab, dtype):
    """Logits about 65536 T / log2(e), where warps of one row take either form
    of the exponent; half of the row is some steps lower."""
    at = 65536 / 1.4426950408889634
    x = torch.full((3, vocab), 0.0)
    for k, low in enumerate((0.0, 256.0, 1.0 if dtype is FP32 else 512.0)):
        x[k] = at + 2
        x[k, : vocab // 2] = at + 2 - low
    x[0, ::3] += 512
    x, y = x.to(dtype).cuda(), torch.tensor([0, vocab - 1, 1]).cuda()
    adv = torch.tensor([1.0, -1.0, 2.0]).cuda()
    for tau in (1.0, 256.0):
        z = (x.float() * (tau if tau > 1 else 1)).to(dtype)
        n = o.policy(f64(z), y.cpu().numpy(), f64(adv), temperature=tau)
        out = meo.policy_loss(z, y, adv, temperature=tau)
        check_logp(f64(out.logp), n[2], vocab)
        check_grad(f64(out.grad), n[3], n[4] / tau, vocab, dtype)
        r = meo.token_logprobs(z, y, temperature=tau)
        check_logp(f64(r.logp), n[2], vocab)
        g = meo.token_logprobs_backward(z, y, r.stats, adv, temperature=tau)
        check_grad(f64(g), o.logprobs_grad(f64(z), y.cpu().numpy(), f64(adv), tau), f64(adv) / tau, vocab, dtype)
