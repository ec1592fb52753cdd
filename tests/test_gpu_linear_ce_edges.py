"""The linear output layer's cross entropy at the ends of its ranges, against float64."""
import numpy as np
import pytest
import torch

import memory_efficient_optimizer_gb300 as meo
from memory_efficient_optimizer_gb300 import binding as B
from oracle import linear_ce as O
from oracle.losses import log_softmax

pytestmark = pytest.mark.gpu
BF = torch.bfloat16


def n64(t):
    return t.double().cpu().numpy()


@pytest.mark.parametrize("temperature", [1.0, 0.7, 0.5, 0.3, 1.5, 2.0, 1.1, 0.9])
@pytest.mark.parametrize("dim", [16, 72, 512, 1030])
def test_words_of_logit_minus_infinity_have_probability_0(dim, temperature):
    """Tolerances as for finite logits: 2e-6 (1 + |value|) and 2^-23 of the largest logit, and 2^-7 of a gradient's norm."""
    n, vocab = 20, 300
    g = torch.Generator().manual_seed(dim)
    h = (torch.rand(n, dim, generator=g) + 0.1).to(BF)
    w = (torch.randn(vocab, dim, generator=g) / dim ** 0.5).to(BF)
    masked = torch.zeros(vocab, dtype=torch.bool)
    masked[5:9] = masked[128:256] = masked[299] = True       # a span of 128 words among them, and the last word
    w[masked] = -float("inf")
    y = torch.randint(0, 5, (n,), generator=g)
    y[3], y[4], y[5], y[6] = 7, 200, 270, -100               # two whose targets are masked
    out = meo.linear_cross_entropy(h.cuda(), w.cuda(), y.cuda(), temperature=temperature)
    z = n64(h) @ np.where(masked[:, None], 0.0, n64(w.masked_fill(masked[:, None], 0))).T / temperature
    z[:, masked.numpy()] = -np.inf
    logp = np.array([log_softmax(v) for v in z])
    lse = np.array([(v - q)[0] for v, q in zip(z, logp)])
    at = np.where(y.numpy() == -100, 0, y.numpy())
    want = np.where(y.numpy() == -100, 0.0, logp[np.arange(n), at])
    got = n64(out.logp)
    assert np.all(got[[3, 4]] == -np.inf) and out.loss.item() == np.inf
    rest = np.delete(np.arange(n), [3, 4])
    big = np.abs(z[:, ~masked.numpy()]).max()
    assert np.all(np.abs(got - want)[rest] <= 2e-6 * (1 + np.abs(want[rest])) + 2.0 ** -23 * big)
    counts = y.numpy() != -100
    assert np.all(np.abs(n64(out.lse) - lse)[counts] <= (2e-6 * (1 + np.abs(lse)) + 2.0 ** -23 * big)[counts])
    dx = np.exp(logp)
    dx[np.arange(n), at] -= 1
    gw = (dx * counts[:, None] / counts.sum() / temperature).T @ n64(h)
    assert np.linalg.norm(n64(out.grad_weight) - gw) <= 2.0 ** -7 * np.linalg.norm(gw)


def test_nothing_but_minus_infinity_has_no_distribution():
    h, w = torch.ones(3, 16, dtype=BF, device="cuda"), torch.full((200, 16), -float("inf"), dtype=BF, device="cuda")
    y = torch.tensor([0, 150, -100], device="cuda")
    out = meo.linear_cross_entropy(h, w, y)
    assert out.logp[:2].isnan().all() and out.lse[:2].isnan().all() and out.loss.isnan()
    assert out.logp[2] == 0 and out.lse[2] == 0


@pytest.mark.parametrize("vocab", [1, 130, 300])
def test_plus_infinity_and_nan_answer_nan(vocab):
    h = torch.ones(4, 16, dtype=BF, device="cuda")
    for bad in (float("inf"), float("nan")):
        for at in {0, vocab - 1}:
            w = (torch.randn(vocab, 16, generator=torch.Generator().manual_seed(1)) / 4).to(BF).cuda()
            w[at] = bad
            for target in {0, vocab - 1}:
                out = meo.linear_cross_entropy(h, w, torch.full((4,), target, device="cuda"))
                assert out.logp.isnan().all() and out.lse.isnan().all() and out.loss.isnan()
                assert out.grad_hidden.isnan().all() and out.grad_weight.isnan().all()


@pytest.mark.parametrize("temperature", [1.0, 1e-3, 1e-5, 3e-6, 1e-6, 3e-7, 1e-7, 1e-9, 1e-20, 1e-30])
def test_low_temperatures(temperature):
    """Whole numbers, whose logits are exact, many of them alike: the largest share their probability at any temperature.

    The logits' factor is off by 2^-25 and the tensor cores' mean, 2^-24 together, of a logarithm's size; an exponential
    by 2^-22.  Gradients: a rounding to bf16 of the coefficient and of the result, 2^-8 each."""
    n, dim, vocab = 60, 16, 300
    g = torch.Generator().manual_seed(1)
    h = torch.randint(-3, 4, (n, dim), generator=g).float()
    w = torch.randint(-3, 4, (vocab, dim), generator=g).float()
    w[130:260] = w[:130]                            # on both sides of a span of 128 words
    z = h @ w.T
    y = torch.where(torch.arange(n) % 3 > 0, z.argmax(1), torch.randint(0, vocab, (n,), generator=g))
    out = meo.linear_cross_entropy(h.to(BF).cuda(), w.to(BF).cuda(), y.cuda(), temperature=temperature,
                                   grad_hidden=torch.empty(n, dim, device="cuda"), grad_weight=torch.empty(vocab, dim, device="cuda"))
    loss, gh, gw, logp, lse = O.linear_cross_entropy(n64(h), n64(w), y.numpy(), temperature=temperature)
    for got, want in ((out.logp, logp), (out.lse, lse)):
        assert np.all(np.abs(n64(got) - want) <= 2.0 ** -21 * (1 + np.abs(want)))
    assert abs(out.loss.item() - loss) <= 2.0 ** -20 * (1 + abs(loss))
    for got, want in ((out.grad_hidden, gh), (out.grad_weight, gw)):
        assert np.linalg.norm(n64(got) - want) <= 2.0 ** -7 * np.linalg.norm(want)


@pytest.mark.parametrize("mask", [-3.3e38, -1e38, -1e30, -1e9, -1e7, -4e6, -2.9e6, -1e4])
@pytest.mark.parametrize("temperature", [1.0, 0.5, 2.0])
def test_masked_words_of_very_low_logits(mask, temperature):
    """Words held down by a constant of the hidden states: alone in a span of 128 words, or beside others."""
    n, dim, vocab = 30, 32, 400
    g = torch.Generator().manual_seed(2)
    h = torch.randn(n, dim, generator=g).to(BF)
    h[:, 0] = 1
    w = torch.randn(vocab, dim, generator=g).to(BF)
    w[:, 0] = 0
    w[128:256] = 0
    w[128:256, 0] = mask
    w[7, 0] = w[399, 0] = mask
    y = torch.randint(0, 128, (n,), generator=g)
    y[y == 7] = 8
    y[3], y[4] = 140, 399
    out = meo.linear_cross_entropy(h.cuda(), w.cuda(), y.cuda(), temperature=temperature)
    loss, gh, gw, logp, lse = O.linear_cross_entropy(n64(h), n64(w), y.numpy(), temperature=temperature)
    ok = np.abs(logp) < 2e38              # (what fp32 holds, before the logarithm's factor too)
    for got, want in ((out.logp, logp), (out.lse, lse)):
        assert np.all(np.abs(n64(got) - want)[ok] <= 2.0 ** -19 + 2.0 ** -20 * np.abs(want[ok]))
    assert np.all(n64(out.logp)[~ok] < -1e38)
    keep = np.ones(n, dtype=bool)
    keep[3:5] = False
    # (hidden gradients with 0 times the mask: finite, and whole but for the constant)
    assert np.linalg.norm((n64(out.grad_hidden) - gh)[keep][:, 1:]) <= 2.0 ** -7 * np.linalg.norm(gh[keep][:, 1:])
    assert np.linalg.norm(n64(out.grad_weight) - gw) <= 2.0 ** -7 * np.linalg.norm(gw)


def test_rows_with_near_and_far_logits():
    """Logits from thousands to a hundred million in one row, on both sides of where the exponentials change form, with the
    largest in either form.  Whole numbers, so that the logits are exact and alike where they should be."""
    dim, vocab = 16, 512
    g = torch.Generator().manual_seed(3)
    w = torch.zeros(vocab, dim)
    w[:, 0] = torch.randint(-4, 5, (vocab,), generator=g).float()
    w[:128, 1] = 1
    w[128:256, 2] = 1
    w[256:384, 3] = 1
    w[384:, 4] = 1
    steps = torch.tensor([0.0, 1000.0, 2.0 ** 21, 2.0 ** 21 + 2 ** 14, 2.0 ** 22, 2.0 ** 23, 2.0 ** 26, -1000.0, -2.0 ** 22, -2.0 ** 23, -2.0 ** 26])
    rows = [[a, b, c, d] for a in steps for b in steps[::3] for c in steps[1::4] for d in steps[2::5]]
    h = torch.zeros(len(rows), dim)
    h[:, 0] = 1
    h[:, 1:5] = torch.tensor(rows)
    assert torch.equal(h.to(BF).float(), h) and torch.equal(w.to(BF).float(), w)
    z = h.double() @ w.double().T
    for y in (z.argmax(1), torch.randint(0, vocab, (len(rows),), generator=g)):
        for temperature in (1.0, 2.0, 0.25):
            out = meo.linear_cross_entropy(h.to(BF).cuda(), w.to(BF).cuda(), y.cuda(), temperature=temperature)
            loss, gh, gw, logp, lse = O.linear_cross_entropy(n64(h), n64(w), y.numpy(), temperature=temperature)
            # a logit near 2^26 is a whole multiple of 8 in fp32, 2^-24 of it at most off
            far = 2.0 ** -23 * z.abs().amax(1).numpy() / temperature
            assert np.all(np.abs(n64(out.lse) - lse) <= 2e-6 + far + 2.0 ** -22 * np.abs(lse))
            exact = z.abs().amax(1).numpy() < 2 ** 24 - 8
            assert np.all(np.abs(n64(out.logp) - logp)[exact] <= (2e-6 + 2.0 ** -21 * np.abs(logp))[exact])
            assert out.grad_hidden.isfinite().all() and out.grad_weight.isfinite().all()
            # 2^-8 of the result, and of its terms, whose roundings add up like a norm where the terms themselves cancel
            dx = np.exp(z.numpy() / temperature - lse[:, None])
            dx[np.arange(len(y)), y.numpy()] -= 1
            terms = np.sqrt((dx / len(y) / temperature) ** 2 @ n64(w) ** 2)[exact]
            got, want = n64(out.grad_hidden)[exact], gh[exact]
            assert np.linalg.norm(got - want) <= 2.0 ** -8 * (np.linalg.norm(want) + np.linalg.norm(terms))


@pytest.mark.parametrize("n,dim,vocab,dtype", [(70, 96, 500, BF), (70, 97, 501, torch.float32), (1, 64, 3000, BF), (700, 128, 1000, BF),
                                               (0, 16, 40, BF), (600, 8, 1 << 21, BF)])
@pytest.mark.parametrize("weights", [False, True])
def test_one_gradient_alone(n, dim, vocab, dtype, weights):
    """The library's call for the hidden states' gradient or the weight's by itself (a frozen output layer, a frozen
    trunk), in its own workspace, which no call has used: the same bits as both together, and the other left as it is."""
    g = torch.Generator(device="cuda").manual_seed(n)
    h = torch.randn(n, dim, device="cuda", generator=g).to(dtype)
    w = (torch.randn(vocab, dim, device="cuda", generator=g) / dim ** 0.5).to(dtype)
    y = torch.randint(0, vocab, (n,), device="cuda", generator=g)
    y[::5] = -100
    share = torch.rand(n, device="cuda", generator=g) if weights else None
    both = meo.linear_cross_entropy(h, w, y, weights=share)
    code = B.ADAF_BFLOAT16 if dtype == BF else B.ADAF_FLOAT32
    hidden = lambda t: B.linear_ce_hidden(t.data_ptr(), code, 1, n, dim, 0, dim)
    weight = lambda t: B.linear_ce_weight(t.data_ptr(), code, vocab, dim, 0)
    targets = B.loss_targets(B.loss_rows(y.data_ptr(), 0, 1), B.LOSS_INT64, -100)
    args = B.linear_ce_args(B.loss_rows(share.data_ptr() if weights else None, 0, 1), 1.0, 0.0, 1.0)
    for only_hidden in (True, False):
        out = torch.full_like(h if only_hidden else w, 7.0)
        gh, gw = (hidden(out), None) if only_hidden else (None, weight(out))
        loss, logp, lse = torch.empty((), device="cuda"), torch.empty(n, device="cuda"), torch.empty(n, device="cuda")
        size = B.linear_ce_workspace_size(hidden(h), weight(w), gh, gw)
        ws = torch.full((size + 4096,), 255, dtype=torch.uint8, device="cuda")
        B.linear_ce(hidden(h), weight(w), targets, args, gh, gw, loss.data_ptr(), logp.data_ptr(), lse.data_ptr(), ws.data_ptr(), size,
                    torch.cuda.current_stream().cuda_stream)
        assert torch.equal(out, both.grad_hidden if only_hidden else both.grad_weight)
        assert torch.equal(loss, both.loss) and torch.equal(logp, both.logp) and torch.equal(lse, both.lse)
        assert ws[size:].eq(255).all()


@pytest.mark.parametrize("low", [-3.3e38, -1e38, -1e20, -1e9])
def test_nothing_but_masked_words(low):
    """Every word held down, some with -inf: what is left are the words of the lowest finite logits, alike."""
    n, dim, vocab = 5, 16, 500
    h = torch.zeros(n, dim, dtype=BF)
    h[:, 0] = 1
    w = torch.zeros(vocab, dim, dtype=BF)
    w[:, 0] = low
    w[128:256, 0] = -float("inf")
    w[3, 0] = -float("inf")
    left = int((w[:, 0] > -float("inf")).sum())
    y = torch.tensor([0, 127, 499, 300, 4])
    out = meo.linear_cross_entropy(h.cuda(), w.cuda(), y.cuda())
    x = w[0, 0].double().item()
    assert np.all(np.abs(n64(out.logp) + np.log(left)) <= 2.0 ** -19)
    assert np.all(np.abs(n64(out.lse) - (x + np.log(left))) <= 2.0 ** -22 * abs(x))
    q = np.where(n64(w[:, 0]) == -np.inf, 0.0, 1 / left)
    target = np.zeros(vocab)
    target[y.numpy()] = 1
    got = n64(out.grad_weight)[:, 0] * n                     # (the hidden states' first value is 1)
    # the mean of q - 1[y = j], each off by 2^-8, and so is the result
    assert np.all(np.abs(got - (n * q - target)) <= 2.0 ** -7 * (n * q + target) + 1e-7)
