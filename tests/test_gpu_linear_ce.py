"""The linear output layer's cross entropy on the GPU against the float64 oracle.

Tolerances.  logp and lse: a logit is an fp32 sum of exact products, off by at
most 2^-23 dim of the sum of their sizes at worst and about 2^-23 sqrt(dim)
of it in truth; with the 2^-22 of an exponential and fp32 roundings of values
about 10, 2e-6 (1 + |value|) + 2^-23 of the largest logit is taken.  Gradients,
2-norm over 2-norm: dx is rounded to bf16 (2^-8 at most), its exponentials to
fp16 (2^-12) and the result to bf16 (2^-8); the norms of the sums of rounded
terms can be larger than the sum's own norm where terms cancel, so each is
compared with the norm that the absolute terms would give.
"""
import numpy as np
import pytest
import torch

import memory_efficient_optimizer_gb300 as meo
from memory_efficient_optimizer_gb300 import binding as B
from oracle import linear_ce as O

pytestmark = pytest.mark.gpu
BF, FP = torch.bfloat16, torch.float32


def make(n, dim, vocab, seed=0, dtype=BF, ignore=0.2, std=1.3):
    g = torch.Generator().manual_seed(seed)
    w = (torch.randn(vocab, dim, generator=g) * std / dim ** 0.5).to(dtype)
    y = torch.randint(0, vocab, (n,), generator=g)
    h = (torch.randn(n, dim, generator=g) + 4 * torch.rand(n, 1, generator=g) * w[y].float()).to(dtype)
    y[torch.rand(n, generator=g) < ignore] = -100
    return h, w, y


def n64(t):
    return t.double().cpu().numpy()


def compare(out, h, w, y, gdt=(BF, BF), **kw):
    """The oracle's values for the bf16 values of h and w."""
    h, w, y = n64(h.to(BF)), n64(w.to(BF)), y.reshape(-1).cpu().numpy()
    h = h.reshape(-1, h.shape[-1])
    if kw.get("weights") is not None:
        kw["weights"] = n64(kw["weights"]).reshape(-1)
    loss, gh, gw, logp, lse = O.linear_cross_entropy(h, w, y, **kw)
    big = np.abs(h @ w.T).max() / kw.get("temperature", 1.0) if len(h) else 0.0
    tol = lambda v: 2e-6 * (1 + np.abs(v)) + 2.0 ** -23 * big
    assert np.all(np.abs(n64(out.logp).reshape(-1) - logp) <= tol(logp)), np.abs(n64(out.logp).reshape(-1) - logp).max()
    assert np.all(np.abs(n64(out.lse).reshape(-1) - lse) <= tol(lse))
    share = kw["weights"] if kw.get("weights") is not None else np.full(len(y), 1 / max(1, (y != -100).sum()))
    parts = np.abs(share) * (kw.get("z_loss", 0.0) * lse ** 2 + np.abs(logp)) * (y != -100)
    assert abs(out.loss.item() - loss) <= 4e-6 * (parts.sum() + np.abs(share[y != -100]).sum() * (1 + big * 0.1)) + 1e-12
    if out.grad_hidden is None:
        return
    # |dx|: what the rounded terms of the gradients' sums amount to
    z = h @ w.T / kw.get("temperature", 1.0)
    z[y == -100] = -1e30                              # (an ignored token has no lse)
    q = np.exp(z - lse[:, None]) * (1 + 2 * kw.get("z_loss", 0.0) * lse[:, None])
    q[np.arange(len(y)), np.where(y == -100, 0, y)] -= 1
    dx = np.abs(q * (share / kw.get("temperature", 1.0) * kw.get("grad_scale", 1.0) * (y != -100))[:, None])
    for got, want, a, b, dt in ((out.grad_hidden, gh, dx, w, gdt[0]), (out.grad_weight, gw, dx.T, h, gdt[1])):
        got = n64(got).reshape(want.shape)
        rounded = np.sqrt((a ** 2) @ (b ** 2))       # of independent roundings of the terms
        tol = (2.0 ** -8 if dt == BF else 0.0) * np.abs(want) + (2.0 ** -8 + 2.0 ** -11) * 4 * rounded + 2e-6 * (a @ np.abs(b))
        assert np.all(np.abs(got - want) <= tol + 1e-30), (np.abs(got - want) / (tol + 1e-30)).max()
        # half a step of bf16 each for the terms and for the result, as norms
        assert np.linalg.norm(got - want) <= 2.0 ** -8 * (np.linalg.norm(want) + np.linalg.norm(rounded)) + 1e-30


@pytest.mark.parametrize("n,dim,vocab", [(1, 8, 1), (1, 1, 2), (1, 64, 100), (2, 7, 33), (5, 72, 333), (64, 64, 128), (65, 100, 129),
                                         (128, 128, 127), (130, 257, 1000), (256, 256, 512), (300, 512, 1003), (257, 40, 4099)])
def test_matches_the_oracle(n, dim, vocab):
    h, w, y = make(n, dim, vocab, seed=n)
    out = meo.linear_cross_entropy(h.cuda(), w.cuda(), y.cuda())
    compare(out, h, w, y)


@pytest.mark.parametrize("kw", [dict(temperature=0.3), dict(temperature=3.0, z_loss=0.01), dict(grad_scale=512.0), dict(z_loss=1.0),
                                dict(weights=True), dict(weights=True, temperature=0.5, z_loss=1e-3)])
def test_options(kw):
    h, w, y = make(70, 96, 500, seed=3)
    if kw.get("weights"):
        kw = dict(kw, weights=torch.randn(70, generator=torch.Generator().manual_seed(1)))
    on = {k: (v.cuda() if torch.is_tensor(v) else v) for k, v in kw.items()}
    compare(meo.linear_cross_entropy(h.cuda(), w.cuda(), y.cuda(), **on), h, w, y, **kw)


@pytest.mark.parametrize("hdt,wdt", [(FP, FP), (BF, FP), (FP, BF)])
def test_types(hdt, wdt):
    h, w, y = make(90, 50, 300, seed=4, dtype=FP)
    h, w = h.to(hdt), w.to(wdt)
    for idt in (torch.int32, torch.int64):
        out = meo.linear_cross_entropy(h.cuda(), w.cuda(), y.to(idt).cuda())
        assert out.grad_hidden.dtype == hdt and out.grad_weight.dtype == wdt
        compare(out, h, w, y, gdt=(hdt, wdt))
    gh, gw = torch.empty(90, 50, device="cuda", dtype=FP), torch.empty(300, 50, device="cuda", dtype=BF)
    out = meo.linear_cross_entropy(h.cuda(), w.cuda(), y.cuda(), grad_hidden=gh, grad_weight=gw)
    assert out.grad_hidden is gh and out.grad_weight is gw
    compare(out, h, w, y, gdt=(FP, BF))


def test_strides_and_views():
    h, w, y = make(4 * 33, 80, 200, seed=5)
    wide = torch.zeros(4, 34, 96, dtype=BF, device="cuda")
    hv = wide[:, :33, 3:83]
    hv.copy_(h.view(4, 33, 80))
    ids = torch.zeros(4, 34, dtype=torch.int64, device="cuda")
    ids[:, 1:] = y.view(4, 33).cuda()
    wv = torch.zeros(200, 85, dtype=BF, device="cuda")[:, 2:82]
    wv.copy_(w)
    gw = torch.full((200, 90), 3.0, dtype=FP, device="cuda")
    gh = torch.full((4, 40, 81), 3.0, dtype=BF, device="cuda")
    out = meo.linear_cross_entropy(hv, wv, ids[:, 1:], grad_hidden=gh[:, :33, :80], grad_weight=gw[:, 5:85])
    compare(out, h, w, y, gdt=(BF, FP))
    assert gh[:, 33:].eq(3).all() and gh[:, :, 80:].eq(3).all() and gw[:, :5].eq(3).all() and gw[:, 85:].eq(3).all()
    # a transposed batch: rows in another order than the tokens'
    ht = h.view(33, 4, 80).transpose(0, 1).cuda()
    out = meo.linear_cross_entropy(ht, w.cuda(), y.view(33, 4).t().cuda())
    compare(out, ht, w, y.view(33, 4).t())
    # one advantage a sequence: weights of stride 0
    share = torch.tensor([0.5, -1.0, 0.0, 2.0], device="cuda")[:, None].expand(4, 33)
    out = meo.linear_cross_entropy(hv, wv, ids[:, 1:], weights=share)
    compare(out, h, w, y, weights=share)


@pytest.mark.parametrize("vocab", [1, 2, 130])
def test_weights_with_aligned_gaps(vocab):
    """Rows 16-byte aligned with gaps between them are read where they are; a single row's stride says nothing."""
    h, w, y = make(70, 40, vocab, seed=16)
    wide = torch.full((vocab, 56), float("nan"), dtype=BF, device="cuda")
    for wv in (wide[:, 8:48], wide.as_strided((vocab, 40), (0 if vocab == 1 else 56, 1), 8)):
        wv.copy_(w)
        compare(meo.linear_cross_entropy(h.cuda(), wv, y.cuda()), h, w, y)


def test_in_place_and_accumulated():
    h, w, y = make(150, 64, 300, seed=6)
    hc = h.cuda()
    out = meo.linear_cross_entropy(hc, w.cuda(), y.cuda(), grad_hidden=hc)
    assert out.grad_hidden is hc
    compare(out, h, w, y)
    for dt in (FP, BF):
        gw = torch.ones(300, 64, device="cuda", dtype=dt)
        once = meo.linear_cross_entropy(h.cuda(), w.cuda(), y.cuda(), grad_weight=torch.empty(300, 64, device="cuda", dtype=FP))
        meo.linear_cross_entropy(h.cuda(), w.cuda(), y.cuda(), grad_weight=gw, accumulate=True)
        want = once.grad_weight + 1
        assert ((gw.float() - want).abs() <= (2 ** -8 if dt == BF else 2 ** -23) * want.abs() + 1e-7).all()
    with pytest.raises(ValueError, match="accumulate"):
        meo.linear_cross_entropy(hc, w.cuda(), y.cuda(), accumulate=True)
    with pytest.raises(ValueError, match="need_grad"):
        meo.linear_cross_entropy(hc, w.cuda(), y.cuda(), grad_hidden=hc, need_grad=False)


def test_loss_alone_is_the_same():
    h, w, y = make(200, 72, 700, seed=7)
    a = meo.linear_cross_entropy(h.cuda(), w.cuda(), y.cuda(), z_loss=0.1)
    b = meo.linear_cross_entropy(h.cuda(), w.cuda(), y.cuda(), z_loss=0.1, need_grad=False)
    assert b.grad_hidden is None and b.grad_weight is None
    assert torch.equal(a.loss, b.loss) and torch.equal(a.logp, b.logp) and torch.equal(a.lse, b.lse)


@pytest.mark.parametrize("n", [0, 1, 70])
def test_nothing_counts(n):
    h, w, y = make(max(n, 1), 24, 40, seed=8)
    h, y = h[:n], torch.full((n,), -100)
    gw = torch.ones(40, 24, device="cuda")
    out = meo.linear_cross_entropy(h.cuda(), w.cuda(), y.cuda())
    assert out.loss.item() == 0 and out.grad_hidden.eq(0).all() and out.grad_weight.eq(0).all() and out.logp.eq(0).all()
    meo.linear_cross_entropy(h.cuda(), w.cuda(), y.cuda(), grad_weight=gw, accumulate=True)
    assert gw.eq(1).all()


def test_other_ignore_index_and_bad_targets():
    h, w, y = make(80, 48, 90, seed=9, ignore=0.0)
    y[::7] = 5
    out = meo.linear_cross_entropy(h.cuda(), w.cuda(), y.cuda(), ignore_index=5)
    compare(out, h, w, y, ignore=5) if not (y == -100).any() else None
    for bad in (90, -1, 2 ** 40):
        y2 = y.clone()
        y2[11] = bad
        out = meo.linear_cross_entropy(h.cuda(), w.cuda(), y2.cuda())
        assert out.loss.isnan() and out.logp[11].isnan() and out.grad_hidden[11].isnan().all() and out.grad_weight.isnan().all()
        rest = torch.arange(80) != 11
        assert out.logp[rest.cuda()].isfinite().all() and out.grad_hidden[rest.cuda()].isfinite().all()


def test_values_that_are_not_finite():
    h, w, y = make(40, 32, 300, seed=10, ignore=0.0)
    for bad in (float("nan"), float("inf")):
        h2 = h.clone()
        h2[7, 3] = bad
        out = meo.linear_cross_entropy(h2.cuda(), w.cuda(), y.cuda())
        assert out.logp[7].isnan() and out.loss.isnan() and out.grad_hidden[7].isnan().all()
        rest = torch.arange(40) != 7
        assert out.logp[rest.cuda()].isfinite().all() and out.grad_hidden[rest.cuda()].isfinite().all()
        # an ignored token may hold anything
        y2 = y.clone()
        y2[7] = -100
        out = meo.linear_cross_entropy(h2.cuda(), w.cuda(), y2.cuda())
        h3 = h.clone()
        compare(out, h3, w, y2)


def test_large_logits():
    """Logits of some thousands, and tokens that are certain: what is left of 1 - q comes out."""
    h, w, y = make(60, 64, 200, seed=11, std=12.0)
    h = (h.float() * 20).to(BF)
    out = meo.linear_cross_entropy(h.cuda(), w.cuda(), y.cuda())
    compare(out, h, w, y)
    h = torch.zeros(3, 64)
    w = torch.zeros(200, 64)
    w[5, 0] = 1.0
    h[:, 0] = torch.tensor([8.0, 16.0, 24.0])
    y = torch.tensor([5, 5, 5])
    out = meo.linear_cross_entropy(h.to(BF).cuda(), w.to(BF).cuda(), y.cuda())
    left = n64(out.grad_hidden)[:, 0] * -3
    want = 199 / (199 + np.exp([8.0, 16.0, 24.0]))
    assert np.all(np.abs(left - want) <= 2 ** -6 * want)


def test_pieces():
    """More tokens than a piece holds: the vocabulary of 2^21 words leaves 512 rows to one."""
    n, dim, vocab = 1100, 8, 1 << 21
    g = torch.Generator(device="cuda").manual_seed(0)
    w = torch.randn(vocab, dim, device="cuda", generator=g).to(BF)
    h = torch.randn(n, dim, device="cuda", generator=g).to(BF)
    y = torch.randint(0, vocab, (n,), device="cuda", generator=g)
    y[::5] = -100
    out = meo.linear_cross_entropy(h, w, y)
    fp = meo.linear_cross_entropy(h, w, y, grad_weight=torch.empty(vocab, dim, device="cuda"))
    wd, gw, count = w.double(), torch.zeros(vocab, dim, device="cuda", dtype=torch.float64), int((y != -100).sum())
    for a in range(0, n, 100):
        z = h[a:a + 100].double() @ wd.T
        lse = z.logsumexp(1)
        keep, at = y[a:a + 100] != -100, y[a:a + 100].clamp_min(0)
        lp = torch.where(keep, z.gather(1, at[:, None])[:, 0] - lse, 0.0)
        assert (out.logp[a:a + 100] - lp).abs().max() < 5e-6 * 25
        dx = (z - lse[:, None]).exp()
        dx[torch.arange(len(at)), at] -= 1
        dx = dx * (keep / count)[:, None]
        gh = dx @ wd
        assert (out.grad_hidden[a:a + 100].double() - gh).norm() <= 2 ** -7 * gh.norm()
        gw += dx.T @ h[a:a + 100].double()
    for got in (out.grad_weight, fp.grad_weight):
        assert (got.double() - gw).norm() <= 2 ** -7 * gw.norm()
    for dt in (BF, torch.float32):   # added to what is there, over the pieces
        more = torch.full((vocab, dim), 0.5, device="cuda", dtype=dt)
        meo.linear_cross_entropy(h, w, y, grad_weight=more, accumulate=True)
        want = fp.grad_weight.double() + 0.5
        assert ((more.double() - want).abs() <= (2 ** -8 if dt == BF else 2 ** -22) * want.abs()).all()
    # pieces without a token that counts: all of the first, all of the last
    for cut in (slice(0, 600), slice(500, None)):
        y2 = y.clone()
        y2[cut] = -100
        a = meo.linear_cross_entropy(h, w, y2)
        keep = (y2 != -100).nonzero()[:, 0]
        b = meo.linear_cross_entropy(h[keep], w, y2[keep])
        assert torch.equal(a.logp[keep], b.logp) and torch.equal(a.grad_hidden[keep], b.grad_hidden)
        assert torch.equal(a.grad_weight, b.grad_weight) and a.grad_hidden[y2 == -100].eq(0).all()


@pytest.mark.parametrize("n", [511, 512, 513, 1100, 9000])
def test_masked_tokens_at_every_count(n):
    """Tokens found by the gathering itself and by a scan of their own; masks that leave few, and none in long runs."""
    h, w, y = make(n, 24, 60, seed=n, ignore=0.0)
    for keep in (torch.arange(n) % 7 == 3, torch.arange(n) == n - 1, torch.arange(n) >= n // 2):
        y2 = torch.where(keep, y, -100)
        compare(meo.linear_cross_entropy(h.cuda(), w.cuda(), y2.cuda()), h, w, y2)


def test_equal_bits_and_other_streams():
    h, w, y = (t.cuda() for t in make(500, 200, 3000, seed=12))
    a = meo.linear_cross_entropy(h, w, y)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    b = meo.linear_cross_entropy(h, w, y, stream=s)
    c = meo.linear_cross_entropy(h, w, y)      # at the same time
    torch.cuda.synchronize()
    for x in (b, c):
        assert all(torch.equal(p, q) for p, q in zip(a, x))


def test_captured_and_replayed():
    h, w, y = (t.cuda() for t in make(100, 64, 500, seed=13))
    first = meo.linear_cross_entropy(h, w, y)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = meo.linear_cross_entropy(h, w, y)
    graph.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(p, q) for p, q in zip(first, out))
    y.copy_(y.roll(1))
    graph.replay()
    again = meo.linear_cross_entropy(h, w, y)
    torch.cuda.synchronize()
    assert all(torch.equal(p, q) for p, q in zip(again, out))


def test_gradients_against_differences():
    """fp32 gradients against differences of the loss, along directions."""
    h, w, y = make(48, 40, 150, seed=14)
    out = meo.linear_cross_entropy(h.cuda(), w.cuda(), y.cuda(), grad_hidden=torch.empty(48, 40, device="cuda"),
                                   grad_weight=torch.empty(150, 40, device="cuda"))
    ref = lambda a, b: O.linear_cross_entropy(a, b, y.numpy())[0]
    hn, wn = n64(h), n64(w)
    g = np.random.default_rng(0)
    for _ in range(4):
        d = g.standard_normal(hn.shape)
        assert abs((ref(hn + 1e-5 * d, wn) - ref(hn - 1e-5 * d, wn)) / 2e-5 - (n64(out.grad_hidden) * d).sum()) < 2 ** -7 * np.linalg.norm(n64(out.grad_hidden))
        d = g.standard_normal(wn.shape)
        assert abs((ref(hn, wn + 1e-5 * d) - ref(hn, wn - 1e-5 * d)) / 2e-5 - (n64(out.grad_weight) * d).sum()) < 2 ** -7 * np.linalg.norm(n64(out.grad_weight))


def test_a_step_of_a_model():
    """The operators together: the loss of a small model from its hidden states, Muon on its matrices,
    Adafactor on the embedding and the output weight."""
    torch.manual_seed(0)
    vocab, dim = 300, 32
    embed, mix, head = torch.nn.Embedding(vocab, dim).cuda(), torch.nn.Linear(dim, dim, bias=False).cuda(), torch.nn.Linear(dim, vocab, bias=False).cuda()
    muon = meo.Muon(mix.parameters(), lr=0.02)
    rest = meo.Adafactor([embed.weight, head.weight])
    tokens = torch.randint(0, vocab, (4, 17), device="cuda")
    for _ in range(3):
        x = embed(tokens[:, :-1])
        hidden = x + torch.tanh(mix(x))
        out = meo.linear_cross_entropy(hidden.detach(), head.weight.detach(), tokens[:, 1:])
        hidden.backward(out.grad_hidden)
        head.weight.grad = out.grad_weight
        # the same gradients by autograd, of the rounded hidden states and weight
        h2, w2 = hidden.detach().to(BF).float().requires_grad_(), head.weight.detach().to(BF).float().requires_grad_()
        ref = torch.nn.functional.cross_entropy((h2 @ w2.T).flatten(0, 1), tokens[:, 1:].flatten())
        ref.backward()
        assert abs(out.loss.item() - ref.item()) < 1e-4
        assert (out.grad_hidden - h2.grad).norm() < 2 ** -7 * h2.grad.norm()
        assert (out.grad_weight - w2.grad).norm() < 2 ** -7 * w2.grad.norm()
        before = mix.weight.detach().clone()
        muon.step()
        rest.step()
        assert mix.weight.isfinite().all() and head.weight.isfinite().all() and not torch.equal(before, mix.weight)
        muon.zero_grad()
        rest.zero_grad()


def test_a_copy_that_never_lands_ends_the_call():
    h, w, y = (t.cuda() for t in make(100, 64, 500, seed=15))
    good = meo.linear_cross_entropy(h, w, y)
    B.linear_ce_debug_stall_copies(True)
    try:
        out = meo.linear_cross_entropy(h, w, y, need_grad=False)
        torch.cuda.synchronize()
    finally:
        B.linear_ce_debug_stall_copies(False)
    assert out.loss.isnan()
    again = meo.linear_cross_entropy(h, w, y)
    assert all(torch.equal(p, q) for p, q in zip(good, again))
