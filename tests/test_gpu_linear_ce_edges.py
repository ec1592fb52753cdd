"""The linear output layer's cross entropy at the ends of its ranges, against float64."""
import numpy as np
import pytest
import torch

import memory_efficient_optimizer_gb300 as meo
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
