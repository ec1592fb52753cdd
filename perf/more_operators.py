"""Cases of the operators on matrices: cross entropy from hidden states and an
output weight, orthogonalised updates and the Muon step.

``run`` makes one pass through one operator: its plain form in fp32 torch
operations (``own`` false) or the framework's call (``own`` true).  A training
operator returns its loss, its per-token values and its whole gradients, an
optimizer step the new parameters and state.
"""
import math

import torch

own = False

IGNORE = -100
V_LARGE = 128256      # the vocabulary of the repository's Llama-3-8B list
COEF = (3.4445, -4.7750, 2.0315)
STEPS = 5
EPS = 1e-7
LAYER_ATTENTION = "4096x4096,1024x4096,1024x4096,4096x4096"
LAYER_REST = "14336x4096,14336x4096,4096x14336"


def listed():
    return [
        # a training step on a handful of tokens: the weight is read, its gradient written
        dict(name="ce_few_tokens", op="ce", batch=1, seq=16, dim=4096, vocab=32000, prompt=0, grad=True, weights=False,
             z=0.0, temperature=1.0),
        # an odd vocabulary and odd lengths, a small model, per-token weights and the term that holds lse down
        dict(name="ce_odd", op="ce", batch=3, seq=333, dim=768, vocab=50257, prompt=0, grad=True, weights=True, z=1e-4,
             temperature=1.0),
        # a fine-tuning micro-batch, prompts masked
        dict(name="ce_batch", op="ce", batch=4, seq=512, dim=4096, vocab=V_LARGE, prompt=128, grad=True, weights=False,
             z=0.0, temperature=1.0),
        # the largest: a pre-training micro-batch
        dict(name="ce_long", op="ce", batch=4, seq=2048, dim=4096, vocab=V_LARGE, prompt=0, grad=True, weights=False,
             z=0.0, temperature=1.0),
        # the log-probability of one sampled token from the last hidden state
        dict(name="ce_logp_one", op="ce", batch=1, seq=1, dim=4096, vocab=V_LARGE, prompt=0, grad=False, weights=False,
             z=0.0, temperature=1.0),
        # reference log-probabilities of a batch at a sampling temperature, prompts masked
        dict(name="ce_logp_batch", op="ce", batch=4, seq=1024, dim=4096, vocab=V_LARGE, prompt=256, grad=False,
             weights=False, z=0.0, temperature=0.7),
        # one small matrix: latency
        dict(name="orth_small", op="orth", batch=1, rows=256, cols=512, dtype="bf16"),
        # odd sizes, more rows than columns, fp32 input
        dict(name="orth_odd", op="orth", batch=1, rows=1403, cols=777, dtype="fp32"),
        # the matrices of a stack of experts
        dict(name="orth_experts", op="orth", batch=8, rows=1024, cols=4096, dtype="bf16"),
        # the matrices of a small model's layer, fp32 gradients
        dict(name="muon_small", op="muon", shapes="256x256,256x256,256x256,256x256,1024x256,256x1024", dtype="fp32",
             nesterov=True, adjust="original", lr=2e-3, decay=0.01),
        # one decoder layer's attention matrices
        dict(name="muon_attention", op="muon", shapes=LAYER_ATTENTION, dtype="bf16", nesterov=True, adjust="match_rms",
             lr=3e-4, decay=0.1),
        # the whole decoder layer
        dict(name="muon_layer", op="muon", shapes=LAYER_ATTENTION + "," + LAYER_REST, dtype="bf16", nesterov=True,
             adjust="match_rms", lr=3e-4, decay=0.1),
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def _side(rng, lo, hi):
    n = _log_int(rng, lo, hi)
    return n if rng.random() < 0.4 else max(lo, n // 64 * 64)


def draw(rng):
    op = rng.choice(["ce", "ce", "orth", "muon"])
    if op == "ce":
        grad = rng.random() < 0.7
        vocab, dim = _side(rng, 500, 131072), _side(rng, 64, 4096)
        most = 4096 * 4096 * V_LARGE // (dim * vocab)      # tokens of half the largest case
        tokens = _log_int(rng, 1, max(1, min(16384, most)))
        batch = rng.choice([1, 2, 3, 4, 8])
        seq = max(1, tokens // batch)
        return dict(op=op, batch=batch, seq=seq, dim=dim, vocab=vocab, prompt=rng.choice([0, 0, seq // 4, seq // 2]),
                    grad=grad, weights=rng.random() < 0.3, z=rng.choice([0.0, 0.0, 1e-4]),
                    temperature=rng.choice([1.0, 1.0, 0.7, 1.5]))
    if op == "orth":
        rows, cols = _side(rng, 16, 6144), _side(rng, 16, 6144)
        batch = min(_log_int(rng, 1, 16), max(1, 2 ** 25 // (rows * cols)))
        return dict(op=op, batch=batch, rows=rows, cols=cols, dtype=rng.choice(["bf16", "fp32"]))
    shapes = []
    for _ in range(rng.choice([1, 2, 3, 4])):
        shapes += ["%dx%d" % (_side(rng, 16, 4096), _side(rng, 16, 6144))] * rng.choice([1, 1, 2, 3])
    adjust = rng.choice(["original", "match_rms"])
    return dict(op=op, shapes=",".join(shapes), dtype=rng.choice(["bf16", "fp32"]), nesterov=rng.random() < 0.7,
                adjust=adjust, lr=rng.choice([1e-3, 2e-3]) if adjust == "original" else rng.choice([2e-4, 3e-4]),
                decay=rng.choice([0.0, 0.01, 0.1]))


def _shapes(case):
    return [tuple(int(n) for n in s.split("x")) for s in case["shapes"].split(",")]


def _orth_flops(rows, cols):
    """Products of the iteration, the symmetric ones by one half."""
    m, n = min(rows, cols), max(rows, cols)
    return STEPS * (3 * m * m * n + m * m * m)


def work(case):
    if case["op"] == "ce":
        t, d, v = case["batch"] * (case["seq"] - case["prompt"]), case["dim"], case["vocab"]
        every = case["batch"] * case["seq"]
        if not case["grad"]:
            return {"bytes": 2 * (t * d + v * d) + 16 * every, "flops": 2 * t * d * v}
        return {"bytes": 2 * (t * d + 2 * v * d + every * d) + 16 * every, "flops": 6 * t * d * v}
    es = 2 if case["dtype"] == "bf16" else 4
    if case["op"] == "orth":
        n = case["batch"] * case["rows"] * case["cols"]
        return {"bytes": n * (es + 2), "flops": case["batch"] * _orth_flops(case["rows"], case["cols"])}
    # the gradient is read, momentum and parameter are read and written
    return {"bytes": sum(h * w * (es + 16) for h, w in _shapes(case)), "flops": sum(_orth_flops(h, w) for h, w in _shapes(case))}


# ---- inputs ----------------------------------------------------------------

def _generator(seed):
    return torch.Generator(device="cuda").manual_seed(int(seed) * 7919 + 29)


def _gradient(g, rows, cols):
    """The momentum of a layer's gradient and one gradient beside it: some dozens of strong directions, each weaker
    than the one before, that last from step to step, over the noise of the batches."""
    r = max(1, min(rows, cols, 48))
    left, right = (torch.randn(n, r, device="cuda", generator=g) for n in (rows, cols))
    strong = (left * torch.arange(1, r + 1, device="cuda") ** -1.0) @ right.T
    noise, before = (torch.randn(rows, cols, device="cuda", generator=g) for _ in range(2))
    return 1e-3 * (15 * strong + 3 * before), 1e-3 * (strong + noise)


def prepare(case, seed):
    g = _generator(seed)
    if case["op"] == "ce":
        b, s, d, v = case["batch"], case["seq"], case["dim"], case["vocab"]
        weight = torch.randn(v, d, device="cuda", generator=g).mul_(1.3 / math.sqrt(d)).bfloat16()
        y = torch.randint(0, v, (b, s), device="cuda", generator=g)
        # hidden states of a trained model: they lean toward the word that follows, some strongly, some not at all
        lean = 8 + 3 * torch.randn(b, s, 1, device="cuda", generator=g)
        hidden = torch.randn(b, s, d, device="cuda", generator=g) + lean / 1.69 * weight[y].float()
        y[:, :case["prompt"]] = IGNORE
        weights = torch.rand(b, s, device="cuda", generator=g) / (b * s) if case["weights"] else None
        return dict(case=case, hidden=hidden.bfloat16(), weight=weight, targets=y, weights=weights)
    dtype = torch.bfloat16 if case["dtype"] == "bf16" else torch.float32
    if case["op"] == "orth":
        x = torch.stack([_gradient(g, case["rows"], case["cols"])[0] for _ in range(case["batch"])]).to(dtype)
        return dict(case=case, x=x if case["batch"] > 1 else x[0])
    params, grads, states = [], [], []
    for rows, cols in _shapes(case):
        m, gr = _gradient(g, rows, cols)
        params.append(torch.randn(rows, cols, device="cuda", generator=g) / math.sqrt(cols))
        grads.append(gr.to(dtype))
        states.append({"momentum": m})
    st = dict(case=case, params=params, grads=grads, states=states)
    if own:
        import memory_efficient_optimizer_gb300 as meo
        st["step"] = meo.MuonStep(params, grads, states, lr=case["lr"], momentum=0.95, nesterov=case["nesterov"],
                                  weight_decay=case["decay"], adjust_lr=case["adjust"])
    return st


# ---- one pass --------------------------------------------------------------

def run(st):
    return _own(st) if own else _plain(st)


def _own(st):
    import memory_efficient_optimizer_gb300 as meo
    case = st["case"]
    if case["op"] == "ce":
        r = meo.linear_cross_entropy(st["hidden"], st["weight"], st["targets"], weights=st["weights"], z_loss=case["z"],
                                     temperature=case["temperature"], ignore_index=IGNORE, need_grad=case["grad"])
        out = {"loss": r.loss, "logp": r.logp, "lse": r.lse}
        if case["grad"]:
            out.update(grad_hidden=r.grad_hidden, grad_weight=r.grad_weight)
        return out
    if case["op"] == "orth":
        return {"out": meo.orthogonalize(st["x"])}
    st["step"]()
    return {"params": st["params"], "momentum": [s["momentum"] for s in st["states"]]}


def _plain(st):
    case = st["case"]
    if case["op"] == "ce":
        return _plain_ce(st)
    if case["op"] == "orth":
        return {"out": _plain_orth(st["x"].float()).bfloat16()}
    for p, g, s in zip(st["params"], st["grads"], st["states"]):
        g, m = g.float(), s["momentum"]
        m.mul_(0.95).add_(g)
        o = _plain_orth(g + 0.95 * m if case["nesterov"] else m)
        h, w = p.shape
        scale = math.sqrt(max(1.0, h / w)) if case["adjust"] == "original" else 0.2 * math.sqrt(max(h, w))
        p.mul_(1 - case["lr"] * case["decay"]).sub_(o, alpha=case["lr"] * scale)
    return {"params": st["params"], "momentum": [s["momentum"] for s in st["states"]]}


def _plain_ce(st):
    case, y, tau = st["case"], st["targets"], st["case"]["temperature"]
    keep = y != IGNORE
    at = torch.where(keep, y, torch.zeros_like(y))[..., None]
    h, w = st["hidden"].float(), st["weight"].float()
    z = h @ w.T / tau
    top = z.amax(-1, keepdim=True)
    z -= top
    zy = z.gather(-1, at)
    e = z.exp_()
    s = e.sum(-1, keepdim=True)
    zero = torch.zeros_like(s[..., 0])
    logp = torch.where(keep, (zy - s.log())[..., 0], zero)
    lse = torch.where(keep, (top + s.log())[..., 0], zero)
    share = torch.where(keep, 1.0 / keep.sum().clamp_min(1) if st["weights"] is None else st["weights"], zero)
    out = {"loss": (share * (case["z"] * lse * lse - logp)).sum(), "logp": logp, "lse": lse}
    if case["grad"]:
        share = (share / tau)[..., None]
        e *= share * (1 + 2 * case["z"] * lse[..., None]) / s
        e.scatter_add_(-1, at, -share)
        out["grad_hidden"] = (e @ w).bfloat16()
        out["grad_weight"] = (e.flatten(0, 1).T @ h.flatten(0, 1)).bfloat16()
    return out


def _plain_orth(x):
    turn = x.shape[-2] > x.shape[-1]
    x = x.mT if turn else x
    x = x / x.square().sum((-2, -1), keepdim=True).sqrt().clamp_min(EPS)
    a, b, c = COEF
    for _ in range(STEPS):
        s = x @ x.mT
        x = a * x + (b * s + c * (s @ s)) @ x
    return x.mT if turn else x


# ---- 64 bits ---------------------------------------------------------------

def exact(case, seed):
    """The same outputs from the definitions in 64 bits, the gradients of the loss by differentiation."""
    w = work(case)["flops"] * (1 if case["op"] == "ce" else 1.5)
    if w > 9e12:
        return None
    st = prepare(case, seed)
    if case["op"] == "ce":
        return _exact_ce(st)
    if case["op"] == "orth":
        return {"out": _exact_orth(st["x"].double())}
    params, momentum = [], []
    for p, g, s in zip(st["params"], st["grads"], st["states"]):
        g = g.double()
        m = s["momentum"].double() * 0.95 + g
        u = g + m * 0.95 if case["nesterov"] else m
        h, w = p.shape
        scale = max(1.0, h / w) ** 0.5 if case["adjust"] == "original" else 0.2 * max(h, w) ** 0.5
        params.append(p.double() - case["lr"] * (case["decay"] * p.double() + scale * _exact_orth(u)))
        momentum.append(m)
    return {"params": params, "momentum": momentum}


def _exact_orth(x):
    """The iteration as an odd polynomial of x, one polynomial a step: x (a + x^T x (b + c x^T x)) or its mirror image."""
    a, b, c = COEF
    x = x / x.flatten(-2).norm(dim=-1)[..., None, None].clamp_min(EPS)
    for _ in range(STEPS):
        if x.shape[-1] < x.shape[-2]:
            s = x.mT @ x
            x = x @ (c * (s @ s) + b * s) + a * x
        else:
            s = x @ x.mT
            x = (c * (s @ s) + b * s) @ x + a * x
    return x


def _exact_ce(st):
    case, y = st["case"], st["targets"].reshape(-1)
    keep = torch.nonzero(y != IGNORE)[:, 0]
    dim, n = case["dim"], y.numel()
    w = st["weight"].double().requires_grad_(case["grad"])
    hidden = st["hidden"].reshape(n, dim)
    share = st["weights"].reshape(-1).double() if case["weights"] else torch.full((n,), 1.0 / max(1, keep.numel()),
                                                                                   dtype=torch.float64, device=y.device)
    logp, lse = (torch.zeros(n, dtype=torch.float64, device=y.device) for _ in range(2))
    loss = torch.zeros((), dtype=torch.float64, device=y.device)
    gh = torch.zeros(n, dim, dtype=torch.float64, device=y.device)
    gw = torch.zeros(w.shape, dtype=torch.float64, device=y.device)
    for at in keep.split(1024):
        h = hidden[at].double().requires_grad_(case["grad"])
        with torch.set_grad_enabled(case["grad"]):
            z = h @ w.T / case["temperature"]
            norm = torch.logsumexp(z, -1)
            lp = z[torch.arange(at.numel(), device=y.device), y[at]] - norm
            part = (share[at] * (case["z"] * norm.square() - lp)).sum()
        logp[at], lse[at] = lp.detach(), norm.detach()
        loss += part.detach()
        if case["grad"]:
            dh, dw = torch.autograd.grad(part, (h, w))
            gh[at] = dh
            gw += dw
    shape = st["targets"].shape
    out = {"loss": loss, "logp": logp.view(shape), "lse": lse.view(shape)}
    if case["grad"]:
        out.update(grad_hidden=gh.view(*shape, dim), grad_weight=gw)
    return out
