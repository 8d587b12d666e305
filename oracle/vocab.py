"""CPU oracle for the operators over vocabulary-parallel logits.

TEST INFRASTRUCTURE ONLY (same rule as the rest of ``oracle/``). Plain numpy in
64 bits on the whole [rows, vocab] matrix; ``include/tccl.h`` states the
formulas. Rounding to fewer bits happens nowhere here.
"""
from __future__ import annotations

import numpy as np


def log_softmax(x, temperature):
    """(log p, row maximum, log of the sum relative to it), rows all -inf giving
    log p = -inf and (-inf, 0)."""
    x = np.asarray(x, dtype=np.float64)
    m = x.max(axis=1)
    lp = np.full(x.shape, -np.inf)
    log_s = np.zeros(x.shape[0])
    for t in range(x.shape[0]):
        if np.isnan(x[t]).any() or np.isposinf(x[t]).any():
            lp[t], log_s[t] = np.nan, np.nan
        elif np.isfinite(m[t]):
            d = (x[t] - m[t]) / temperature
            log_s[t] = np.log(np.exp(d).sum())
            lp[t] = d - log_s[t]
    return lp, m, log_s


def _plogp(lp):
    return np.where(np.isneginf(lp), 0.0, np.exp(lp) * np.where(np.isneginf(lp), 0.0, lp))


def entropy(lp):
    return -_plogp(lp).sum(axis=1)


def log_probs(x, tokens, temperature, top_k):
    """dict of log_probs, entropy, stats, top_log_probs and top_ids."""
    x = np.asarray(x, dtype=np.float64)
    rows, vocab = x.shape
    lp, m, log_s = log_softmax(x, temperature)
    out = {"log_probs": np.zeros(rows), "entropy": entropy(lp), "stats": np.stack([m, log_s], 1),
           "top_log_probs": np.full((rows, top_k), -np.inf),
           "top_ids": np.full((rows, top_k), -1, dtype=np.int64)}
    for t in range(rows):
        if tokens is not None:
            if not 0 <= tokens[t] < vocab:
                out["entropy"][t] = 0.0
                out["stats"][t] = 0.0
                continue
            out["log_probs"][t] = lp[t, tokens[t]]
        if np.isnan(log_s[t]):
            out["top_log_probs"][t] = np.nan
            continue
        order = np.argsort(-x[t], kind="stable")[:top_k]
        order = order[~np.isneginf(x[t][order])]
        out["top_ids"][t, :len(order)] = order
        out["top_log_probs"][t, :len(order)] = lp[t][order]
    return out


def log_probs_backward(x, tokens, temperature, d_log_probs, d_entropy):
    lp, _, _ = log_softmax(x, temperature)
    rows, vocab = lp.shape
    h = entropy(lp)
    g = np.zeros(lp.shape)
    for t in range(rows):
        a, b = float(d_log_probs[t]), 0.0 if d_entropy is None else float(d_entropy[t])
        if not 0 <= tokens[t] < vocab or (a == 0 and b == 0) or np.isneginf(lp[t]).all():
            continue
        g[t] = -(np.exp(lp[t]) * (a + b * h[t]) + b * _plogp(lp[t]))
        g[t, tokens[t]] += a
    return g / temperature


def teacher(ids, logits, temperature, lse, vocab):
    """(q, log q) of the teacher's entries, empty ones 0 and -inf."""
    z = np.asarray(logits, dtype=np.float64) / temperature
    z = np.where((ids < 0) | (ids >= vocab), -np.inf, z)
    if lse is None:
        top = z.max(axis=1, keepdims=True)
        top = np.where(np.isneginf(top), 0.0, top)
        total = np.exp(z - top).sum(axis=1, keepdims=True)
        log_q = z - top - np.log(np.where(total == 0, 1.0, total))
    else:
        log_q = z - np.asarray(lse, dtype=np.float64)[:, None]
    return np.exp(log_q), log_q


def distill(x, ids, logits, temperature, lse=None, weights=None):
    """(loss, gradient of sum weights * loss or None)."""
    lp, m, _ = log_softmax(x, temperature)
    rows, vocab = lp.shape
    q, log_q = teacher(ids, logits, temperature, lse, vocab)
    loss = np.zeros(rows)
    g = np.zeros(lp.shape)
    for t in range(rows):
        on = q[t] > 0
        loss[t] = (q[t][on] * (log_q[t][on] - lp[t][ids[t][on]])).sum()
        if weights is not None and weights[t] != 0 and on.any() and not np.isneginf(m[t]):
            row = q[t].sum() * np.exp(lp[t])
            np.subtract.at(row, ids[t][on], q[t][on])
            g[t] = row * (float(weights[t]) / temperature)
    return loss, None if weights is None else g
