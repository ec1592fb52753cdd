"""Float64 CPU reference of the losses over a vocabulary (include/losses.h):
the formulas, one token at a time, with numpy.  Test infrastructure only; the
package never imports it.

Every function takes arrays over tokens, ``x`` [tokens, vocab] in float64, and
returns the loss, the per-token values and the gradient of the logits.
"""
from __future__ import annotations

import numpy as np


def log_softmax(z):
    """ln softmax of one row; NaN where the row has no distribution."""
    m = np.max(z)
    with np.errstate(invalid="ignore", divide="ignore", over="ignore"):
        if np.isnan(m) or np.isinf(m):
            return np.full(z.shape, np.nan)
        d = z - m
        return d - np.log(np.sum(np.exp(d)))


def token_logprobs(x, y, temperature=1.0, ignore=-100):
    out = np.zeros(len(y))
    for t in range(len(y)):
        if y[t] != ignore:
            out[t] = log_softmax(x[t] / temperature)[y[t]] if 0 <= y[t] < x.shape[1] else np.nan
    return out


def logprobs_grad(x, y, d, temperature=1.0, ignore=-100):
    """dx = d (1[j = y] - q) / T."""
    g = np.zeros(x.shape)
    for t in range(len(y)):
        if y[t] == ignore:
            continue
        if not 0 <= y[t] < x.shape[1]:
            g[t] = np.nan
            continue
        q = np.exp(log_softmax(x[t] / temperature))
        with np.errstate(invalid="ignore"):  # (an infinite d times a word of probability 0)
            g[t] = -q * d[t] / temperature
        g[t, y[t]] += d[t] / temperature
    return g


def policy(x, y, adv, old=None, ref=None, clip_low=0.2, clip_high=0.2, kl_coef=0.0, weights=None, temperature=1.0,
           ignore=-100):
    logp = token_logprobs(x, y, temperature, ignore)
    n = int(np.sum(y != ignore))
    token, d = np.zeros(len(y)), np.zeros(len(y))
    for t in range(len(y)):
        if y[t] == ignore:
            continue
        r = np.exp(logp[t] - old[t]) if old is not None else 1.0 if not np.isnan(logp[t]) else np.nan
        raw, cut = r * adv[t], np.clip(r, 1 - clip_low, 1 + clip_high) * adv[t]
        token[t] = -min(raw, cut)
        d[t] = -raw if raw <= cut else 0.0
        if kl_coef:
            far = ref[t] - logp[t]
            token[t] += kl_coef * (np.expm1(far) - far if far != np.inf else np.inf)
            d[t] -= kl_coef * np.expm1(far)
    w = np.full(len(y), 1.0 / max(n, 1)) if weights is None else np.asarray(weights, dtype=np.float64)
    w = np.where(y != ignore, w, 0.0)
    return np.sum(w * token), token, logp, logprobs_grad(x, y, w * d, temperature, ignore), w * d


def preference(x, y, sequences, ref=None, beta=0.1, label_smoothing=0.0, kind="sigmoid", margin=0.0, average=False,
               temperature=1.0, ignore=-100):
    """sequences: list of (from, to) token ranges, the chosen ones first."""
    logp = token_logprobs(x, y, temperature, ignore)
    pairs = len(sequences) // 2
    D, n = [], []
    for a, b in sequences:
        keep = y[a:b] != ignore
        gain = (logp[a:b] - (0.0 if ref is None else ref[a:b]))[keep]
        n.append(int(keep.sum()))
        D.append(gain.sum() / (max(n[-1], 1) if average else 1))
    D = np.array(D)
    pair, d = np.zeros(pairs), np.zeros(len(y))
    for i in range(pairs):
        h = D[i] - D[i + pairs]
        if kind == "sigmoid":
            z, e = beta * h - margin, label_smoothing
            pair[i] = (1 - e) * np.logaddexp(0, -z) + (e * np.logaddexp(0, z) if e else 0.0)
            with np.errstate(over="ignore"):
                dh = beta * (e - 1 + 1 / (1 + np.exp(-z)))
        elif kind == "hinge":
            z = 1 + margin - beta * h
            pair[i], dh = max(0.0, z), -beta if z > 0 else 0.0
        else:
            z = h - 1 / (2 * beta) - margin
            pair[i], dh = z * z, 2 * z
        for q, sign in ((i, 1.0), (i + pairs, -1.0)):
            a, b = sequences[q]
            d[a:b] = sign * dh / pairs / (max(n[q], 1) if average else 1)
    d = np.where(y != ignore, d, 0.0)
    return pair.mean(), pair, beta * D, logp, logprobs_grad(x, y, d, temperature, ignore), d


def distill(x, ids, t, lse=None, mask=None, weights=None, temperature=1.0):
    tokens, vocab = x.shape
    keep = np.ones(tokens, dtype=bool) if mask is None else np.asarray(mask, dtype=bool)
    w = np.full(tokens, 1.0 / max(int(keep.sum()), 1)) if weights is None else np.asarray(weights, dtype=np.float64)
    w = np.where(keep, w, 0.0)
    token, g = np.zeros(tokens), np.zeros(x.shape)
    for i in range(tokens):
        if not keep[i]:
            continue
        on = ids[i] != -1
        k, v = ids[i][on], t[i][on] / temperature
        if np.any((k < 0) | (k >= vocab)) or len(set(k.tolist())) != len(k):
            token[i], g[i] = np.nan, np.nan
            continue
        lq = log_softmax(x[i] / temperature)
        if lse is None:
            p = np.exp(log_softmax(v)) if len(k) else np.zeros(0)
            u = 0.0
        else:
            p = np.exp(v - lse[i])
            u = max(0.0, 1.0 - p.sum()) if len(k) < vocab else 0.0
        with np.errstate(invalid="ignore", divide="ignore"):
            q = np.exp(lq)
            off = np.ones(vocab, dtype=bool)
            off[k] = False
            s = q[off].sum()
            l = sum(a * (np.log(a) - b) for a, b in zip(p, lq[k]) if a != 0)
            grad = q * (p.sum() + u)
            if u > 0:
                l += u * (np.log(u) - np.log(s))
                grad[off] -= u * q[off] / s
                # on the list d ln s / dx = -q: already in the first term
            grad[k] -= p
        token[i] = temperature ** 2 * l
        g[i] = w[i] * temperature * grad
    return np.sum(w * token), token, g, w
