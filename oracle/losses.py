"""Float64 NumPy oracle of token scoring, the policy and preference losses and
their gradients, and of adapter logits.  Written from the definitions, to be
checked by eye; it shares no code with the HIP path.

Rows are float64 arrays; a negative token leaves its row out.
"""
from __future__ import annotations

import numpy as np


def log_softmax(x: np.ndarray, temperature: float) -> np.ndarray:
    z = x / temperature
    top = z.max(axis=-1, keepdims=True)
    return z - top - np.log(np.exp(z - top).sum(axis=-1, keepdims=True))


def bad_rows(x: np.ndarray, tokens: np.ndarray) -> np.ndarray:
    """Row status: 1 for a token past the vocabulary, 2 for a NaN or +inf logit
    or no finite one, 0 otherwise (and for rows that are left out)."""
    bad = np.isnan(x).any(-1) | (x == np.inf).any(-1) | ~np.isfinite(x).any(-1)
    status = np.where(bad, 2, 0)
    status = np.where(tokens >= x.shape[1], 1, status)
    return np.where(tokens < 0, 0, status).astype(np.int32)


def score(x, tokens, temperature=1.0):
    """(log-probabilities, entropies) of the rows; NaN for bad rows."""
    lp, ent = np.zeros(len(x)), np.zeros(len(x))
    status = bad_rows(x, tokens)
    for r in range(len(x)):
        if tokens[r] < 0:
            continue
        if status[r]:
            lp[r] = ent[r] = np.nan
            continue
        row = log_softmax(x[r], temperature)
        lp[r] = row[tokens[r]]
        fin = np.isfinite(row)
        ent[r] = -(np.exp(row[fin]) * row[fin]).sum()
    return lp, ent


def score_gradient(x, tokens, temperature, g, h=None):
    """dL/dx of dL/dlp = g and dL/dH = h; a row with both 0 is 0."""
    h = np.zeros(len(x)) if h is None else h
    out = np.zeros_like(x)
    status = bad_rows(x, tokens)
    for r in range(len(x)):
        if tokens[r] < 0 or (g[r] == 0 and h[r] == 0):
            continue
        if status[r]:
            out[r] = np.nan
            continue
        row = log_softmax(x[r], temperature)
        p = np.exp(row)
        d = -g[r] * p
        d[tokens[r]] = g[r] * -np.expm1(row[tokens[r]])
        fin = np.isfinite(row)
        ent = -(p[fin] * row[fin]).sum()
        d[fin] -= h[r] * p[fin] * (row[fin] + ent)
        out[r] = d / temperature
    return out


def policy(x, tokens, old, adv, ref=None, weights=None, *, clip_low=0.2, clip_high=0.2, kl_coef=0.0,
           temperature=1.0, grad_loss=1.0):
    """dict of loss, logprobs, ratios, kl, grad (of the logits)."""
    n = len(x)
    weights = np.ones(n) if weights is None else weights
    live = np.where(weights == 0, -1, tokens)
    lp, _ = score(x, live, temperature)
    status = bad_rows(x, live)
    ratios, kl, g, loss = np.ones(n), np.zeros(n), np.zeros(n), 0.0
    for r in range(n):
        if live[r] < 0:
            continue
        ratios[r] = np.exp(lp[r] - old[r])
        a = adv[r]
        clipped = min(max(ratios[r], 1 - clip_low), 1 + clip_high)
        s, slope = 0.0, 0.0
        if a != 0:
            s = min(ratios[r] * a, clipped * a)
            slope = a * ratios[r] if ratios[r] * a <= clipped * a else 0.0
        term = -s
        g[r] = -slope
        if ref is not None:
            gap = ref[r] - lp[r]
            kl[r] = np.exp(gap) - gap - 1 if gap < np.inf else gap
            if kl_coef:
                term += kl_coef * kl[r]
                g[r] += kl_coef * (1 - np.exp(gap))
        if status[r]:
            term = g[r] = np.nan
        loss += weights[r] * term
    grad = score_gradient(x, live, temperature, np.where(live < 0, 0.0, g * weights * grad_loss))
    return {"loss": loss, "logprobs": lp, "ratios": ratios, "kl": kl, "grad": grad,
            "status": status}


def preference(x, tokens, offsets, ref=None, pair_weights=None, *, beta=0.1, label_smoothing=0.0,
               margin=0.0, mean=False, temperature=1.0, grad_loss=1.0):
    """dict of loss, pair_losses, rewards, logprobs, grad (of the logits)."""
    pairs = len(offsets) // 2
    ref = np.zeros(len(x)) if ref is None else ref
    pair_weights = np.full(pairs, 1.0 / max(pairs, 1)) if pair_weights is None else pair_weights
    live = np.full(len(x), -1, dtype=np.int64)
    live[offsets[0]:offsets[-1]] = tokens[offsets[0]:offsets[-1]]
    lp, _ = score(x, live, temperature)
    rho, count = np.zeros(2 * pairs), np.ones(2 * pairs)
    for i in range(2 * pairs):
        part = [r for r in range(offsets[i], offsets[i + 1]) if live[r] >= 0]
        rho[i] = sum(lp[r] - ref[r] for r in part)
        if mean and part:
            count[i] = len(part)
    rho = rho / count
    z = beta * (rho[:pairs] - rho[pairs:]) - margin
    ls = lambda v: -np.logaddexp(0.0, -v)  # noqa: E731  ln sigmoid
    # a term of factor 0 is 0, also at an infinite z
    each = sum((-k * ls(v) for k, v in ((1 - label_smoothing, z), (label_smoothing, -z)) if k != 0),
               np.zeros(pairs))
    dz = -(1 - label_smoothing) * np.exp(ls(-z)) + label_smoothing * np.exp(ls(z))
    g = np.zeros(len(x))
    for i in range(2 * pairs):
        side = 1.0 if i < pairs else -1.0
        w = pair_weights[i % pairs]
        g[offsets[i]:offsets[i + 1]] = 0.0 if w == 0 else \
            grad_loss * w * dz[i % pairs] * side * beta / count[i]
    grad = score_gradient(x, live, temperature, np.where(live < 0, 0.0, g))
    loss = float(sum(w * e for w, e in zip(pair_weights, each) if w != 0))
    return {"loss": loss, "pair_losses": each, "rewards": beta * rho, "logprobs": lp,
            "grad": grad, "status": bad_rows(x, live)}


def lora_logits(hidden, lm_head, lora_a, lora_b, ids, scales):
    """hidden W^T + scale (hidden A^T) B^T with each row's own adapter (an id
    of -1: none; an id past the adapters: a row of NaN)."""
    out = hidden @ lm_head.T
    for r in range(len(hidden)):
        i = int(ids[r])
        if i == -1:
            continue
        if i < 0 or i >= len(lora_a):
            out[r] = np.nan
            continue
        out[r] += scales[i] * (lora_b[i] @ (lora_a[i] @ hidden[r]))
    return out
