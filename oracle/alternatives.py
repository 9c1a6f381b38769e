"""Float64 NumPy oracle of scoring with alternatives and of listed tokens with
their gradient.  Written from the definitions, to be checked by eye; it shares no
code with the HIP path.
"""
from __future__ import annotations

import numpy as np

from oracle.losses import log_softmax


def _bad_logits(row: np.ndarray) -> bool:
    return bool(np.isnan(row).any() or (row == np.inf).any() or not np.isfinite(row).any())


def _entropy(logp: np.ndarray) -> float:
    fin = np.isfinite(logp)
    return float(-(np.exp(logp[fin]) * logp[fin]).sum())


def topn(x, tokens, n, temperature=1.0):
    """dict of logprobs, ranks, entropies, ids, top (log-probabilities) and
    status; tokens None: no token is asked for."""
    rows, vocab = x.shape
    out = {"logprobs": np.zeros(rows), "ranks": np.zeros(rows, np.int64),
           "entropies": np.zeros(rows), "ids": np.full((rows, n), -1),
           "top": np.full((rows, n), -np.inf), "status": np.zeros(rows, np.int64)}
    for r in range(rows):
        if tokens is not None and tokens[r] < 0:
            continue
        past = tokens is not None and tokens[r] >= vocab
        if past or _bad_logits(x[r]):
            out["status"][r] = 1 if past else 2
            out["logprobs"][r] = out["entropies"][r] = np.nan
            out["top"][r] = np.nan
            continue
        logp = log_softmax(x[r], temperature)
        order = np.lexsort((np.arange(vocab), -x[r]))  # largest first, lower id among equal ones
        k = min(n, vocab)
        out["ids"][r, :k] = order[:k]
        out["top"][r, :k] = logp[order[:k]]
        out["entropies"][r] = _entropy(logp)
        if tokens is not None:
            out["logprobs"][r] = logp[tokens[r]]
            out["ranks"][r] = 1 + int(np.flatnonzero(order == tokens[r])[0])
    return out


def listed(x, ids, temperature=1.0):
    """(log-probabilities [rows, n], entropies, status)."""
    rows, n = ids.shape
    lp, ent, status = np.zeros((rows, n)), np.zeros(rows), np.zeros(rows, np.int64)
    for r in range(rows):
        used = ids[r] >= 0
        if not used.any():
            continue
        past = (ids[r] >= x.shape[1]).any()
        if past or _bad_logits(x[r]):
            status[r] = 1 if past else 2
            lp[r, used] = ent[r] = np.nan
            continue
        logp = log_softmax(x[r], temperature)
        lp[r, used] = logp[ids[r, used]]
        ent[r] = _entropy(logp)
    return lp, ent, status


def listed_gradient(x, ids, temperature, g, h=None):
    """dL/dx of dL/dlp = g [rows, n] and dL/dH = h [rows]."""
    out = np.zeros_like(x)
    _, _, status = listed(x, ids, temperature)
    for r in range(len(x)):
        used = np.flatnonzero(ids[r] >= 0)
        hr = 0.0 if h is None else h[r]
        if not len(used) or (not g[r, used].any() and hr == 0):
            continue
        if status[r]:
            out[r] = np.nan
            continue
        logp = log_softmax(x[r], temperature)
        p = np.exp(logp)
        for i in used:
            # -g p for every other token, g (1 - p) for the listed one itself
            d = -g[r, i] * p
            d[ids[r, i]] = g[r, i] * -np.expm1(logp[ids[r, i]])
            out[r] += d
        fin = np.isfinite(logp)
        out[r, fin] -= hr * p[fin] * (logp[fin] + _entropy(logp))
        out[r] /= temperature
    return out
