"""Losses over tokens: the clipped policy loss with a KL term and the
preference loss of paired sequences, with their gradients in the logits.
TEST INFRASTRUCTURE.

Everything is float64 and written from the definitions, a token at a time in
meaning (numpy rows): log softmax of the logits, the loss, and the chain rule
d loss / d x = d loss / d logp * (1[y] - softmax x).  Tokens of weight 0 are
left out before anything of theirs is looked at.
"""
from __future__ import annotations

import numpy as np


def log_softmax(x):
    x = np.asarray(x, np.float64)
    with np.errstate(invalid="ignore", over="ignore"):
        d = x - x.max(axis=1, keepdims=True)
        return d - np.log(np.exp(d).sum(axis=1, keepdims=True))


def policy(logits, ids, old, adv, ref=None, weights=None, clip_low=0.2, clip_high=0.2, kl=0.0,
           norm=None):
    """Returns (stats[4], logps[N], grad[N, V])."""
    n, v = logits.shape
    w = np.ones(n) if weights is None else np.asarray(weights, np.float64)
    total = w.sum() if norm is None else float(norm)
    stats, logps, grad = np.zeros(4), np.zeros(n), np.zeros((n, v))
    for i in range(n):
        if w[i] == 0:
            continue
        lp = log_softmax(logits[i:i + 1])[0]
        y, a = int(ids[i]), float(adv[i])
        u = np.exp(lp[y] - float(old[i]))
        inside = u * a <= min(max(u, 1 - clip_low), 1 + clip_high) * a
        term = -u * a if inside else -min(max(u, 1 - clip_low), 1 + clip_high) * a
        slope = -u * a if inside else 0.0
        k = 0.0
        if kl:
            d = float(ref[i]) - lp[y]
            k = np.expm1(d) - d
            slope -= kl * np.expm1(d)
        s = w[i] / total
        stats += s * np.array([term + kl * k, term, k, 0.0 if inside else 1.0])
        logps[i] = lp[y]
        hot = np.zeros(v)
        hot[y] = 1.0
        grad[i] = slope * s * (hot - np.exp(lp))
    return stats, logps, grad


def preference(logits, ids, lens, ref, beta=0.1, smoothing=0.0, weights=None, norm=None):
    """Returns (stats[3], log_ratios[2P], logps[N], grad[N, V])."""
    n, v = logits.shape
    w = np.ones(n) if weights is None else np.asarray(weights, np.float64)
    pairs = len(lens) // 2
    total = pairs if norm is None else float(norm)
    start = np.concatenate([[0], np.cumsum(lens)]).astype(int)
    logps, ratios, grad = np.zeros(n), np.zeros(2 * pairs), np.zeros((n, v))
    prob = [None] * n
    for i in range(n):
        if w[i] != 0:
            lp = log_softmax(logits[i:i + 1])[0]
            logps[i], prob[i] = lp[int(ids[i])], np.exp(lp)
    for s in range(2 * pairs):
        ratios[s] = sum(w[i] * (logps[i] - float(ref[i]))
                        for i in range(start[s], start[s + 1]) if w[i] != 0)
    h = beta * (ratios[0::2] - ratios[1::2])
    soft = lambda x: np.logaddexp(0.0, x)  # noqa: E731
    loss = (1 - smoothing) * soft(-h) + smoothing * soft(h)
    slope = smoothing / (1 + np.exp(-h)) - (1 - smoothing) / (1 + np.exp(h))
    for s in range(2 * pairs):
        c = beta * slope[s // 2] * (1 if s % 2 == 0 else -1) / total
        for i in range(start[s], start[s + 1]):
            if w[i] != 0:
                hot = np.zeros(v)
                hot[int(ids[i])] = 1.0
                grad[i] = c * w[i] * (hot - prob[i])
    stats = np.array([loss.sum(), h.sum(), (h > 0).sum()]) / total
    return stats, ratios, logps, grad
