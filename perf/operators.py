"""Cases of the losses over a vocabulary: token log-probabilities and their
backward pass, the clipped policy loss with a KL term, the preference loss and
distillation from a teacher's top logits.

``run`` makes one pass through one operator: its plain form in fp32 torch
operations (``own`` false) or the framework's call (``own`` true).  Every
training operator returns its loss, its per-token or per-pair values and the
whole gradient of the logits.
"""
import math

import torch

own = False

IGNORE = -100
V_LARGE = 128256      # the vocabulary of the repository's Llama-3-8B list
CLIP_LOW, CLIP_HIGH, KL_COEF = 0.2, 0.28, 0.05
BETA = 0.1


def listed():
    return [
        # the log-probability of one sampled token (a verifier or sampler that asks for it step by step)
        dict(name="logprobs_one_token", op="logprobs", batch=1, seq=1, vocab=V_LARGE, dtype="bf16", prompt=0),
        # reference log-probabilities of a training batch before the step, prompts masked
        dict(name="logprobs_batch", op="logprobs", batch=4, seq=2048, vocab=V_LARGE, dtype="bf16", prompt=512),
        # the backward pass under a caller's own loss, fp32 logits, an odd vocabulary, next-token views of a longer tensor
        dict(name="logprobs_backward_odd", op="logprobs_backward", batch=3, seq=333, vocab=50257, dtype="fp32", prompt=0,
             shifted=True),
        # a policy step on a handful of tokens: latency
        dict(name="policy_few_tokens", op="policy", batch=1, seq=8, vocab=32000, dtype="bf16", prompt=0, kl=True),
        # a policy micro-batch: prompts masked, KL to a reference
        dict(name="policy_batch", op="policy", batch=4, seq=1024, vocab=V_LARGE, dtype="bf16", prompt=256, kl=True),
        # the largest: a long policy batch, every token trained on, no KL term
        dict(name="policy_long", op="policy", batch=4, seq=2048, vocab=V_LARGE, dtype="bf16", prompt=0, kl=False),
        # fp32 logits of an odd vocabulary
        dict(name="policy_fp32_odd", op="policy", batch=3, seq=259, vocab=50257, dtype="fp32", prompt=0, kl=True),
        # one short pair
        dict(name="preference_one_pair", op="preference", batch=2, seq=48, vocab=32000, dtype="bf16", prompt=16,
             packed=False),
        # a batch of pairs padded to one length, prompts masked
        dict(name="preference_batch", op="preference", batch=8, seq=512, vocab=V_LARGE, dtype="bf16", prompt=128,
             packed=False),
        # pairs of their own lengths, packed one after another
        dict(name="preference_packed_fp32", op="preference", batch=6, seq=200, vocab=50257, dtype="fp32", prompt=40,
             packed=True),
        # a distillation step on few tokens, probabilities renormalised over the teacher's entries
        dict(name="distill_few_tokens", op="distill", batch=1, seq=16, vocab=32000, dtype="bf16", prompt=0, top=8,
             temperature=1.0, rest=False),
        # a distillation micro-batch: 64 entries a token, temperature, the rest of the teacher's mass as one entry
        dict(name="distill_batch", op="distill", batch=4, seq=1024, vocab=V_LARGE, dtype="bf16", prompt=0, top=64,
             temperature=2.0, rest=True),
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["logprobs", "logprobs_backward", "policy", "preference", "distill"])
    dtype = rng.choice(["bf16", "bf16", "fp32"])
    vocab = _log_int(rng, 500, 160000)
    if rng.random() < 0.4:
        vocab = max(512, vocab // 64 * 64)
    most = 4096 * V_LARGE // (2 if dtype == "fp32" else 1) // vocab   # tokens of half the largest case
    tokens = _log_int(rng, 1, min(16384, most))
    batch = rng.choice([1, 2, 3, 4, 8])
    if op == "preference":
        batch = 2 * rng.choice([1, 2, 3, 4, 8])
    seq = max(1, tokens // batch)
    if op in ("preference",):
        seq = max(8, min(seq, most // batch))
    case = dict(op=op, batch=batch, seq=seq, vocab=vocab, dtype=dtype, prompt=rng.choice([0, 0, seq // 4, seq // 2]))
    if op == "policy":
        case["kl"] = rng.random() < 0.6
    if op == "logprobs_backward":
        case["shifted"] = rng.random() < 0.5
    if op == "preference":
        case["packed"] = rng.random() < 0.5
    if op == "distill":
        case["top"] = _log_int(rng, 1, 256)
        case["temperature"] = rng.choice([1.0, 1.0, 2.0, 4.0])
        case["rest"] = rng.random() < 0.5
    return case


# ---- layouts: which tokens of a case are trained on (fixed by the case alone) ----

def _lengths(case):
    """Length of each sequence: about the full one, each a little shorter."""
    s = case["seq"]
    if case["op"] != "preference":
        return [s] * case["batch"]
    return [max(case["prompt"] + 1, s - (i * 37 + 5) % (s // 3 + 1)) for i in range(case["batch"])]


def _active(case):
    return sum(n - case["prompt"] for n in _lengths(case))


def _rows(case):
    return sum(_lengths(case)) if case.get("packed") else case["batch"] * case["seq"]


def work(case):
    es = 2 if case["dtype"] == "bf16" else 4
    v, act, rows = case["vocab"], _active(case), _rows(case)
    read, write = act * v * es + rows * 8, 0
    if case["op"] == "logprobs":
        write = act * 4
    else:
        write = rows * v * es + rows * 4
        read += act * {"policy": 12, "preference": 4, "distill": 0, "logprobs_backward": 4}[case["op"]]
    if case["op"] == "distill":
        read += act * case["top"] * 12
    # subtract, scale, exp and sum once, and for a gradient subtract, scale, exp and multiply again
    return {"bytes": read + write, "flops": act * v * (4 if case["op"] == "logprobs" else 8)}


# ---- inputs ----------------------------------------------------------------

def _generator(seed):
    return torch.Generator(device="cuda").manual_seed(int(seed) * 7919 + 17)


def _logits(g, rows, vocab, dtype, y, tau=None):
    """Logits of a trained model: a wide bulk, and the token that was sampled among the likely ones
    (its probability from a few hundredths to nearly one).  With a temperature, four dozen likely words
    a row, each a third less likely than the one before, that hold most of the mass at that temperature."""
    out = torch.empty(rows, vocab, device="cuda", dtype=dtype)
    for a in range(0, rows, 1024):
        b = min(rows, a + 1024)
        out[a:b] = torch.randn(b - a, vocab, device="cuda", generator=g) * 2
    top = math.log(vocab) + 2 + torch.randn(rows, device="cuda", generator=g)
    if tau is not None:
        step = torch.randint(1, vocab // 49 + 1, (rows, 1), device="cuda", generator=g)   # distinct words
        far = torch.arange(1, 49, device="cuda")
        words, fall = (y[:, None] + far * step) % vocab, 0.35 * far
        out.scatter_(1, words, (tau * (top[:, None] - fall)).to(dtype))
        top = tau * top
    out[torch.arange(rows, device="cuda"), y] = top.to(dtype)
    return out


def _chunked_logp(logits, y):
    """log-softmax at y, in pieces (only to make the other models' log-probabilities)."""
    out = torch.empty(y.shape, device="cuda")
    for a in range(0, y.numel(), 1024):
        x = logits[a:a + 1024].float()
        out[a:a + 1024] = x.gather(1, y[a:a + 1024, None])[:, 0] - torch.logsumexp(x, 1)
    return out


def _mask(case):
    """True where a token is trained on: [rows] in the case's layout."""
    rows = []
    for n in _lengths(case):
        keep = [t >= case["prompt"] for t in range(n)]
        if not case.get("packed"):
            keep += [False] * (case["seq"] - n)
        rows += keep
    return torch.tensor(rows, device="cuda")


def prepare(case, seed):
    g = _generator(seed)
    b, s, v = case["batch"], case["seq"], case["vocab"]
    dtype = torch.bfloat16 if case["dtype"] == "bf16" else torch.float32
    packed, shifted = case.get("packed", False), case.get("shifted", False)
    full = s + 1 if shifted else s
    rows = _rows(case) if packed else b * full
    y = torch.randint(0, v, (rows,), device="cuda", generator=g)
    logits = _logits(g, rows, v, dtype, y, case.get("temperature"))
    st = dict(case=case)
    if not packed:
        logits, y = logits.view(b, full, v), y.view(b, full)
    if shifted:
        # position t predicts token t + 1: views of the longer tensors
        logits = logits[:, :-1]
        ids = torch.cat([torch.zeros_like(y[:, :1]), y[:, :-1]], 1)
        y = ids[:, 1:]
    st["logits"] = logits
    if not shifted:
        keep = _mask(case).view(y.shape)
        y = torch.where(keep, y, torch.full_like(y, IGNORE))
    elif case["prompt"]:
        ids[:, 1:1 + case["prompt"]] = IGNORE
    st["targets"] = y
    op = case["op"]
    if op in ("policy", "preference"):
        flat = logits.reshape(-1, v)
        logp = _chunked_logp(flat, y.reshape(-1).clamp_min(0)).view(y.shape)
    if op == "logprobs_backward":
        st["grad_logp"] = torch.randn(y.shape, device="cuda", generator=g) / y.numel()
    if op == "policy":
        # the ratios of a policy a few updates on: most within the clip, some far outside.  None within a thousandth
        # of the clip's edges, where the gradient jumps and no two ways of summing need agree
        drift = torch.randn(y.shape, device="cuda", generator=g) * 0.2
        for edge in (math.log(1 - CLIP_LOW), math.log(1 + CLIP_HIGH)):
            drift = torch.where((drift - edge).abs() < 1e-3, torch.full_like(drift, edge + 2e-3), drift)
        st["old_logp"] = logp - drift
        # advantages of both signs, the good answers' larger (their mean is not normalised away)
        sign = torch.where(torch.arange(b, device="cuda") % 2 == 0, 1.0, -0.4)[:, None]
        st["advantages"] = sign * (1 + 0.2 * torch.randn(b, 1, device="cuda", generator=g)) + \
            0.1 * torch.randn(y.shape, device="cuda", generator=g)
        st["ref_logp"] = logp + 0.3 * torch.randn(y.shape, device="cuda", generator=g) if case["kl"] else None
    if op == "preference":
        # a policy that has moved toward the chosen answers
        half = b // 2
        sign = torch.ones(b, device="cuda")
        sign[half:] = -1
        if packed:
            lens = torch.tensor(_lengths(case), device="cuda")
            per = torch.repeat_interleave(sign, lens)
            st["seq_offsets"] = torch.cat([torch.zeros(1, dtype=torch.int64, device="cuda"), lens.cumsum(0)])
        else:
            per = sign[:, None].expand(b, s)
            st["seq_offsets"] = None
        st["ref_logp"] = logp - per * (8.0 / s) + 0.1 * torch.randn(y.shape, device="cuda", generator=g)
    if op == "distill":
        k, tau, flat = min(case["top"], v), case["temperature"], logits.reshape(-1, v)
        ids = torch.empty(rows, k, dtype=torch.int64, device="cuda")
        val, lse = torch.empty(rows, k, device="cuda"), torch.empty(rows, device="cuda")
        for a in range(0, rows, 1024):
            t = flat[a:a + 1024].float()
            t = t + 0.7 * torch.randn(t.shape, device="cuda", generator=g)
            val[a:a + 1024], ids[a:a + 1024] = torch.topk(t, k, dim=1)
            lse[a:a + 1024] = torch.logsumexp(t / tau, 1)
        st["teacher_ids"], st["teacher_logits"] = ids.view(b, s, k), val.view(b, s, k)
        st["teacher_lse"] = lse.view(b, s) if case["rest"] else None
        st["mask"] = y != IGNORE
    return st


# ---- one pass --------------------------------------------------------------

def run(st):
    return _own(st) if own else _plain(st)


def _own(st):
    import memory_efficient_optimizer_gb300 as meo
    case, x, y = st["case"], st["logits"], st["targets"]
    op = case["op"]
    if op == "logprobs":
        return {"logp": meo.token_logprobs(x, y, ignore_index=IGNORE).logp}
    if op == "logprobs_backward":
        r = meo.token_logprobs(x, y, ignore_index=IGNORE)
        return {"logp": r.logp, "grad": meo.token_logprobs_backward(x, y, r.stats, st["grad_logp"],
                                                                     ignore_index=IGNORE)}
    if op == "policy":
        r = meo.policy_loss(x, y, st["advantages"], st["old_logp"], st["ref_logp"], clip_low=CLIP_LOW,
                            clip_high=CLIP_HIGH, kl_coef=KL_COEF if case["kl"] else 0.0, ignore_index=IGNORE)
        return {"loss": r.loss, "grad": r.grad, "logp": r.logp, "token_loss": r.token_loss}
    if op == "preference":
        r = meo.preference_loss(x, y, st["ref_logp"], seq_offsets=st["seq_offsets"], beta=BETA, ignore_index=IGNORE)
        return {"loss": r.loss, "grad": r.grad, "pair_loss": r.pair_loss, "rewards": r.rewards}
    r = meo.distill_loss(x, st["teacher_ids"], st["teacher_logits"], st["teacher_lse"], mask=st["mask"],
                         temperature=case["temperature"])
    return {"loss": r.loss, "grad": r.grad, "token_loss": r.token_loss}


def _softmax_parts(x, tau=1.0):
    z = x.float()
    if tau != 1.0:
        z = z / tau
    z = z - z.amax(-1, keepdim=True)
    e = z.exp()
    return z, e, e.sum(-1, keepdim=True)


def _plain(st):
    case, x, y = st["case"], st["logits"], st["targets"]
    op = case["op"]
    if op == "distill":
        return _plain_distill(st)
    keep = y != IGNORE
    at = torch.where(keep, y, torch.zeros_like(y))[..., None]
    z, e, s = _softmax_parts(x)
    logp = torch.where(keep, (z.gather(-1, at) - s.log())[..., 0], torch.zeros_like(s[..., 0]))
    if op == "logprobs":
        return {"logp": logp}

    def gradient(dlogp):
        """dlogp (1[j = y] - q_j), rounded once."""
        d = torch.where(keep, dlogp, torch.zeros_like(dlogp))[..., None]
        return (e * (-d / s)).scatter_add(-1, at, d).to(x.dtype)

    if op == "logprobs_backward":
        return {"logp": logp, "grad": gradient(st["grad_logp"])}
    if op == "policy":
        n = keep.sum().clamp_min(1)
        ratio = (logp - st["old_logp"]).exp()
        adv = st["advantages"]
        raw, cut = ratio * adv, ratio.clamp(1 - CLIP_LOW, 1 + CLIP_HIGH) * adv
        token, d = -torch.minimum(raw, cut), torch.where(raw <= cut, -raw, torch.zeros_like(raw))
        if case["kl"]:
            far = st["ref_logp"] - logp
            token = token + KL_COEF * (torch.expm1(far) - far)
            d = d - KL_COEF * torch.expm1(far)
        token = torch.where(keep, token, torch.zeros_like(token))
        return {"loss": token.sum() / n, "grad": gradient(d / n), "logp": logp, "token_loss": token}
    # preference: sequence i of the first half was preferred to sequence i of the second
    gain = torch.where(keep, logp - st["ref_logp"], torch.zeros_like(logp))
    pairs = case["batch"] // 2
    if st["seq_offsets"] is None:
        total = gain.sum(1)
    else:
        lens = st["seq_offsets"].diff()
        who = torch.repeat_interleave(torch.arange(case["batch"], device=gain.device), lens, output_size=gain.numel())
        total = torch.where(who == torch.arange(case["batch"], device=gain.device)[:, None], gain, 0.0).sum(1)
    h = BETA * (total[:pairs] - total[pairs:])
    pair = torch.log1p((-h.abs()).exp()) + (-h).clamp_min(0)
    c = -BETA / pairs / (1 + h.exp())
    c = torch.cat([c, -c])
    d = c[:, None].expand(gain.shape) if st["seq_offsets"] is None else c[who]
    return {"loss": pair.mean(), "grad": gradient(d), "pair_loss": pair, "rewards": BETA * total}


def _plain_distill(st):
    case, x, ids, keep = st["case"], st["logits"], st["teacher_ids"], st["mask"]
    tau, n = case["temperature"], st["mask"].sum().clamp_min(1)
    z, e, s = _softmax_parts(x, tau)
    t = st["teacher_logits"] / tau
    if case["rest"]:
        logpk = t - st["teacher_lse"][..., None]
    else:
        t = t - t.amax(-1, keepdim=True)
        logpk = t - t.exp().sum(-1, keepdim=True).log()
    p = logpk.exp()
    kl = (p * (logpk - (z.gather(-1, ids) - s.log()))).sum(-1)
    w = torch.where(keep, tau / n, torch.zeros_like(kl))[..., None]
    q = e / s
    if case["rest"]:
        left = (1 - p.sum(-1)).clamp_min(0)
        off = e.scatter(-1, ids, 0.0)
        rest = off.sum(-1) / s[..., 0]
        some = left > 0
        kl = kl + torch.where(some, left * (left.clamp_min(1e-37).log() - rest.log()), torch.zeros_like(kl))
        share = torch.where(some, left / rest, torch.zeros_like(kl))
        # off the list q_j (1 - left / rest), on it q_j - p_j
        grad = q - off / s * share[..., None]
    else:
        grad = q
    token = torch.where(keep, tau * tau * kl, torch.zeros_like(kl))
    return {"loss": token.sum() / n, "grad": (grad.scatter_add(-1, ids, -p) * w).to(x.dtype), "token_loss": token}


# ---- 64 bits ---------------------------------------------------------------

def _in_pieces(x, rows_fn, out_rows, step=512):
    """rows_fn(leaf, a, b) -> a scalar to differentiate, for rows [a, b) of x in 64 bits; the whole gradient."""
    flat = x.reshape(-1, x.shape[-1])
    grad = torch.zeros(flat.shape, dtype=torch.float64, device=x.device)
    for a in range(0, flat.shape[0], step):
        b = min(flat.shape[0], a + step)
        leaf = flat[a:b].double().requires_grad_(True)
        with torch.enable_grad():
            v = rows_fn(leaf, a, b)
        grad[a:b], = torch.autograd.grad(v, leaf)
    return grad.view(x.shape)


def _logp64(leaf, y):
    return torch.log_softmax(leaf, -1).gather(-1, y[:, None])[:, 0]


def exact(case, seed):
    """The same outputs from the definitions in 64 bits, gradients by differentiation."""
    st = prepare(case, seed)
    x, op = st["logits"], case["op"]
    v = x.shape[-1]
    shape = st["targets"].shape
    y = st["targets"].reshape(-1)
    keep = y != IGNORE
    safe = y.clamp_min(0)
    zero = torch.zeros(y.shape, dtype=torch.float64, device=x.device)
    if op == "distill":
        k, tau = st["teacher_ids"].shape[-1], case["temperature"]
        ids = st["teacher_ids"].reshape(-1, k)
        t = st["teacher_logits"].reshape(-1, k).double() / tau
        lse = st["teacher_lse"].reshape(-1).double() if case["rest"] else torch.logsumexp(t, -1)
        p = (t - lse[:, None]).exp()
        left = (1 - p.sum(-1)).clamp_min(0) if case["rest"] else zero
        token, n = zero.clone(), max(1, int(keep.sum()))

        def rows(leaf, a, b):
            lq = torch.log_softmax(leaf / tau, -1)
            kl = (p[a:b] * (p[a:b].log() - lq.gather(-1, ids[a:b]))).sum(-1)
            if case["rest"]:
                off = torch.ones_like(lq, dtype=torch.bool).scatter(-1, ids[a:b], False)
                rest = torch.logsumexp(lq.masked_fill(~off, -math.inf), -1)
                lf = left[a:b]
                kl = kl + torch.where(lf > 0, lf * (lf.clamp_min(1e-300).log() - rest), zero[a:b])
            kl = torch.where(keep[a:b], tau * tau * kl, zero[a:b])
            token[a:b] = kl.detach()
            return kl.sum() / n

        grad = _in_pieces(x, rows, shape)
        return {"loss": token.sum() / n, "grad": grad, "token_loss": token.view(shape)}

    logp = zero.clone()
    flat = x.reshape(-1, v)
    for a in range(0, y.numel(), 512):
        logp[a:a + 512] = _logp64(flat[a:a + 512].double(), safe[a:a + 512])
    logp = torch.where(keep, logp, zero)
    if op == "logprobs":
        return {"logp": logp.view(shape)}
    leaf = logp.clone().requires_grad_(True)
    with torch.enable_grad():
        if op == "logprobs_backward":
            loss = (leaf * st["grad_logp"].reshape(-1).double()).sum()
        elif op == "policy":
            r, adv = (leaf - st["old_logp"].reshape(-1).double()).exp(), st["advantages"].reshape(-1).double()
            token = -torch.minimum(r * adv, r.clamp(1 - CLIP_LOW, 1 + CLIP_HIGH) * adv)
            if case["kl"]:
                far = st["ref_logp"].reshape(-1).double() - leaf
                token = token + KL_COEF * (far.exp() - far - 1)
            token = torch.where(keep, token, zero)
            loss = token.sum() / keep.sum().clamp_min(1)
        else:
            gain = torch.where(keep, leaf - st["ref_logp"].reshape(-1).double(), zero)
            if st["seq_offsets"] is None:
                total = gain.view(shape).sum(1)
            else:
                at = st["seq_offsets"].tolist()
                total = torch.stack([gain[i:j].sum() for i, j in zip(at, at[1:])])
            pairs = case["batch"] // 2
            pair = -torch.nn.functional.logsigmoid(BETA * (total[:pairs] - total[pairs:]))
            loss = pair.mean()
    dlogp, = torch.autograd.grad(loss, leaf)
    dlogp = torch.where(keep, dlogp, zero)
    grad = _in_pieces(x, lambda lf, a, b: (_logp64(lf, safe[a:b]) * dlogp[a:b]).sum(), shape)
    if op == "logprobs_backward":
        return {"logp": logp.view(shape), "grad": grad}
    if op == "policy":
        return {"loss": loss.detach(), "grad": grad, "logp": logp.view(shape), "token_loss": token.detach().view(shape)}
    return {"loss": loss.detach(), "grad": grad, "pair_loss": pair.detach(), "rewards": BETA * total.detach()}
