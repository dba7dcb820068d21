"""The router of an expert layer in FP64: scores, choice, weights, counts, balance loss and gradients."""

from __future__ import annotations

import numpy as np

TINY = 1e-20


def _scores(x: np.ndarray, score: str):
    """(p, share) of logits x [m, E]."""
    if score == "softmax":
        top = x.max(1, keepdims=True)
        with np.errstate(invalid="ignore"):  # a NaN or +inf makes its whole row NaN
            e = np.exp(x - np.where(top == -np.inf, 0.0, top))
        total = e.sum(1, keepdims=True)
        p = np.divide(e, total, out=np.zeros_like(e), where=total != 0)
        return p, p
    e = np.exp(-np.abs(x))
    p = np.where(x >= 0, 1.0, e) / (1.0 + e)
    return p, p / (p.sum(1, keepdims=True) + TINY)


def ref_router(logits, top_k, score="softmax", bias=None, mask=None, normalize=True, scale=1.0):
    """dict of ids, weights, counts, prob_sum, loss; row by row, slot by slot."""
    x = np.asarray(logits, dtype=np.float64)
    m, e = x.shape
    p, share = _scores(x, score)
    key = x if bias is None else np.where(x == -np.inf, x, p + np.asarray(bias, dtype=np.float64))
    ids = np.full((m, top_k), -1, dtype=np.int64)
    weights = np.zeros((m, top_k))
    on = np.ones(m, dtype=bool) if mask is None else np.asarray(mask, dtype=bool)
    for t in np.nonzero(on)[0]:
        left = [j for j in range(e) if key[t, j] > -np.inf]
        for slot in range(min(top_k, len(left))):
            best = max(left, key=lambda j: (key[t, j], -j))
            left.remove(best)
            ids[t, slot], weights[t, slot] = best, p[t, best]
    if normalize:
        weights = np.where(ids >= 0, weights / (weights.sum(1, keepdims=True) + TINY), 0.0)
    counts = np.bincount(ids[ids >= 0], minlength=e)
    prob_sum = share[on].sum(0)
    den = counts.sum() * prob_sum.sum()
    loss = e * (counts * prob_sum).sum() / den if counts.sum() > 0 and den != 0 else 0.0
    return dict(ids=ids, weights=weights * scale, counts=counts, prob_sum=prob_sum, loss=loss)


def ref_router_backward(logits, ids, dweights, counts=None, prob_sum=None, dloss=0.0, score="softmax", normalize=True,
                        scale=1.0):
    """(dlogits [m, E], sums of magnitudes that bound a kernel's roundings)."""
    x = np.asarray(logits, dtype=np.float64)
    m, e = x.shape
    p, share = _scores(x, score)
    g = np.zeros(e)
    if counts is not None and counts.sum() * prob_sum.sum() > 0:
        g = dloss * e * counts.astype(np.float64) / (counts.sum() * np.asarray(prob_sum, dtype=np.float64).sum())
    dx, mag = np.zeros((m, e)), np.zeros((m, e))
    for t in range(m):
        sel = [(j, i) for j, i in enumerate(ids[t]) if 0 <= i < e]
        if not sel:
            continue
        dp, dm = np.zeros(e), np.zeros(e)
        total = sum(p[t, i] for _, i in sel) + TINY
        dot = sum(dweights[t, j] * p[t, i] for j, i in sel)
        adot = sum(abs(dweights[t, j]) * p[t, i] for j, i in sel)
        for j, i in sel:
            dp[i] += scale * ((dweights[t, j] - dot / total) / total if normalize else dweights[t, j])
            dm[i] += scale * ((abs(dweights[t, j]) + adot / total) / total if normalize else abs(dweights[t, j]))
        if score == "softmax":
            dp, dm = dp + g, dm + np.abs(g)
            dx[t] = p[t] * (dp - (p[t] * dp).sum())
            mag[t] = p[t] * (dm + (p[t] * dm).sum())
        else:
            if counts is not None:
                q = p[t].sum() + TINY
                dp, dm = dp + (g - (g * share[t]).sum()) / q, dm + (np.abs(g) + (np.abs(g) * share[t]).sum()) / q
            slope = p[t] * _scores(-x[t:t + 1], "sigmoid")[0][0]
            dx[t], mag[t] = dp * slope, dm * slope
    return dx, mag
