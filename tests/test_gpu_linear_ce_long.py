"""The linear output layer's cross entropy at the hidden sizes of real models and with long sums, against float64.

Tolerances.  Logits are summed on the tensor cores in parts of 1024 values, 64 steps of 16.  A step cuts off up to 2^-24
or so of the sum as it is; the average of a part, 0.54 64 2^-25 of it, is made up for by a factor, so a part is off by
at most as much again either way: 0.54 64 2^-25 = 1.03e-6 of the largest that the part's sum has been on the way.  The
parts are added in fp32, 2^-24 of the sum each.  Behind that come an exponential (2^-22) and the fp32 roundings of the
logarithm, of lse and of logp (2^-22 of their sizes).

Gradients: a word's coefficient is rounded to bf16 (2^-8 at most; 2^-9 on the average of its two ends), its exponential
to fp16 (2^-11), and the result to bf16 (2^-8) or not at all.  Independent roundings of the terms add up like a norm:
(2^-8 + 2^-11) sqrt(sum of squares), of which four are allowed, and 2^-8 of the norms over all values.
"""
import numpy as np
import pytest
import torch

import memory_efficient_optimizer_gb300 as meo
from oracle import linear_ce as O

pytestmark = pytest.mark.gpu
BF, FP = torch.bfloat16, torch.float32
PART = 1024


def make(n, dim, vocab, seed, ignore=0.2):
    g = torch.Generator().manual_seed(seed)
    w = (torch.randn(vocab, dim, generator=g) * 1.3 / dim ** 0.5).to(BF)
    y = torch.randint(0, vocab, (n,), generator=g)
    h = (torch.randn(n, dim, generator=g) + 8 * torch.rand(n, 1, generator=g) * w[y].float()).to(BF)
    y[torch.rand(n, generator=g) < ignore] = -100
    return h, w, y


def n64(t):
    return t.double().cpu().numpy()


def reached(h, w):
    """For every token, over its words the most that the parts' running sums come to, summed over the parts."""
    out = np.zeros(len(h))
    for t in range(len(h)):
        terms = w * h[t]
        most = sum(np.abs(np.cumsum(terms[:, k:k + PART], axis=1)).max(axis=1) for k in range(0, terms.shape[1], PART))
        out[t] = most.max()
    return out


def logit_tolerance(h, w):
    return (0.54 * 64 * 2.0 ** -25 + -(-h.shape[1] // PART) * 2.0 ** -24) * reached(h, w)


def gradients_hold(got, want, a, b, dtype):
    got = n64(got).reshape(want.shape)
    rounded = np.sqrt((a ** 2) @ (b ** 2))
    tol = (2.0 ** -8 if dtype == BF else 0.0) * np.abs(want) + (2.0 ** -8 + 2.0 ** -11) * 4 * rounded + 2e-6 * (a @ np.abs(b))
    assert np.all(np.abs(got - want) <= tol + 1e-30), (np.abs(got - want) / (tol + 1e-30)).max()
    assert np.linalg.norm(got - want) <= 2.0 ** -8 * (np.linalg.norm(want) + np.linalg.norm(rounded)) + 1e-30


@pytest.mark.parametrize("n,dim,vocab", [(40, 1024, 300), (33, 1025, 257), (150, 1100, 130), (20, 2048, 1003), (70, 2049, 64),
                                         (9, 4096, 500), (140, 4096, 129), (300, 1536, 200), (3, 8192, 300), (1, 5000, 2000),
                                         (2, 65536, 40)])
@pytest.mark.parametrize("gdt", [BF, FP])
def test_long_hidden_states(n, dim, vocab, gdt):
    h, w, y = make(n, dim, vocab, seed=n + dim)
    out = meo.linear_cross_entropy(h.cuda(), w.cuda(), y.cuda(), grad_hidden=torch.empty(n, dim, device="cuda", dtype=gdt),
                                   grad_weight=torch.empty(vocab, dim, device="cuda", dtype=gdt))
    hn, wn, yn = n64(h), n64(w), y.numpy()
    loss, gh, gw, logp, lse = O.linear_cross_entropy(hn, wn, yn)
    off = 2 * logit_tolerance(hn, wn) + 2.0 ** -21       # (logp has two logits' errors)
    keep = yn != -100
    assert np.all(np.abs(n64(out.logp) - logp)[keep] <= (off + 2.0 ** -22 * np.abs(lse))[keep])
    assert np.all(np.abs(n64(out.lse) - lse)[keep] <= (off + 2.0 ** -22 * np.abs(lse))[keep])
    assert abs(out.loss.item() - loss) <= (off + 2.0 ** -22 * np.abs(lse))[keep].max() + 2.0 ** -23 * abs(loss)
    q = np.exp(hn @ wn.T - lse[:, None])
    q[np.arange(n), np.where(keep, yn, 0)] -= 1
    dx = np.abs(q) * (keep / max(1, keep.sum()))[:, None]
    gradients_hold(out.grad_hidden, gh, dx, wn, gdt)
    gradients_hold(out.grad_weight, gw, dx.T, hn, gdt)
    alone = meo.linear_cross_entropy(h.cuda(), w.cuda(), y.cuda(), need_grad=False)
    assert torch.equal(alone.logp, out.logp) and torch.equal(alone.lse, out.lse) and torch.equal(alone.loss, out.loss)


@pytest.mark.parametrize("dim", [512, 1024, 4096])
def test_long_sums_do_not_lean(dim):
    """What the tensor cores cut off is made up for on the average: measured between 0.42 and 0.56 of 2^-25 a step and
    taken as 0.54, so a logit is 0.12 64 2^-25 = 2.3e-7 off at most on the average.  3e-7 is taken; without the factor
    it is 1.0e-6, without the parts 4e-6 at 4096 values."""
    h, w, y = make(256, dim, 128, seed=dim, ignore=0.0)
    out = meo.linear_cross_entropy(h.cuda(), w.cuda(), y.cuda(), need_grad=False)
    got = n64(out.logp) + n64(out.lse)
    want = (n64(h) * n64(w)[y.numpy()]).sum(1)
    assert abs(((got - want) * want).sum() / (want ** 2).sum()) < 3e-7


# What sums of tensor memory may lose: a step cuts off at most 2^-24 or so of the sum as it is on the average of both
# ends of a binade, and no sum has more than 2^17 values, 8192 steps: 8192 2^-24 = 4.9e-4 of a gradient, in its own direction.
LEAN = 8192 * 2.0 ** -24


@pytest.mark.parametrize("vocab", [1 << 21, (1 << 20) + 77, 1 << 17])
@pytest.mark.parametrize("weights", [False, True])
def test_hidden_gradients_over_a_large_vocabulary(vocab, weights):
    """The target comes first and makes most of the gradient; the other words follow in 131072 steps."""
    n, dim = 70, 64
    g = torch.Generator(device="cuda").manual_seed(5)
    w = (torch.randn(vocab, dim, device="cuda", generator=g) * 1.3 / dim ** 0.5).to(BF)
    h = torch.randn(n, dim, device="cuda", generator=g).to(BF)
    y = torch.arange(n, device="cuda") * 3 + torch.arange(n, device="cuda") % 2 * (vocab // 2)
    share = torch.full((n,), 2.0 ** -6, device="cuda") if weights else None
    out = meo.linear_cross_entropy(h, w, y, weights=share, grad_hidden=torch.empty(n, dim, device="cuda"))
    dx = (h.double() @ w.double().T).softmax(1)
    dx[torch.arange(n), y] -= 1
    want = dx @ w.double() * (2.0 ** -6 if weights else 1 / n)
    lean = ((out.grad_hidden.double() - want) * want).sum(1) / want.square().sum(1)
    assert lean.abs().max() <= LEAN
    assert (out.grad_hidden.double() - want).norm() <= 2.0 ** -8 * want.norm()


@pytest.mark.parametrize("dt", [FP, BF])
def test_weight_gradients_over_many_tokens(dt):
    """2^21 tokens of a small vocabulary, whose hidden states have a mean."""
    n, dim, vocab = (1 << 21) + 5, 16, 24
    g = torch.Generator(device="cuda").manual_seed(6)
    w = (torch.randn(vocab, dim, device="cuda", generator=g) / dim ** 0.5).to(BF)
    h = (torch.randn(n, dim, device="cuda", generator=g) + 1).to(BF)
    y = torch.randint(0, vocab, (n,), device="cuda", generator=g)
    y[torch.rand(n, device="cuda", generator=g) < 0.8] = 0
    out = meo.linear_cross_entropy(h, w, y, grad_weight=torch.empty(vocab, dim, device="cuda", dtype=dt))
    want = torch.zeros(vocab, dim, device="cuda", dtype=torch.float64)
    for a, b in zip(h.split(1 << 18), y.split(1 << 18)):
        dx = (a.double() @ w.double().T).softmax(1)
        dx[torch.arange(len(b)), b] -= 1
        want += dx.T @ a.double() / n
    # (a bf16 result is off by up to 2^-8 of each value, at random over a row)
    off = LEAN + (2.0 ** -8 * 2 / dim ** 0.5 if dt == BF else 0)
    assert abs(((out.grad_weight.double() - want)[0] * want[0]).sum() / want[0].square().sum()) <= off
    assert (out.grad_weight.double() - want).norm() <= 2.0 ** -8 * want.norm()


@pytest.mark.parametrize("vocab", [1 << 19, 128256])
def test_hidden_gradients_in_one_sum_over_the_vocabulary(vocab):
    """So many tiles that nothing is gained by sums in parts: one goes over all words, the target's first."""
    n, dim, some = 2048, 4864, 32
    g = torch.Generator(device="cuda").manual_seed(7)
    w = torch.empty(vocab, dim, device="cuda", dtype=BF)
    for c in w.split(1 << 16):
        c.copy_(torch.randn(c.shape, device="cuda", generator=g) * 1.3 / dim ** 0.5)
    h = torch.randn(n, dim, device="cuda", generator=g).to(BF)
    y = torch.randint(0, 64, (n,), device="cuda", generator=g)
    out = meo.linear_cross_entropy(h, w, y, grad_hidden=torch.empty(n, dim, device="cuda"))
    dx = torch.cat([h[:some].double() @ c.double().T for c in w.split(1 << 16)], 1).softmax(1)
    dx[torch.arange(some), y[:some]] -= 1
    want = sum(d @ c.double() for d, c in zip(dx.split(1 << 16, 1), w.split(1 << 16))) / n
    off = out.grad_hidden[:some].double() - want
    assert (off * want).sum(1).div(want.square().sum(1)).abs().max() <= LEAN
    assert off.norm() <= 2.0 ** -8 * want.norm()
