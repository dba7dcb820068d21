"""RMS norm with the residual's addition, and its gradient.
TEST INFRASTRUCTURE ONLY.

For every row, in FP64 from the operands as stored:

    s = x + residual,   r = 1 / sqrt(mean(s^2) + eps),   v = s * r * weight;

and for a gradient dy of v, with xhat = s * r and g = dy * weight,

    dx = r * (g - xhat * mean(g * xhat)) + dresidual,   dw = sum over rows of dy * xhat.

The cast of v is ``quant.py``'s.
"""

from __future__ import annotations

import numpy as np


def ref_add_rms_norm(x, weight, eps: float, residual=None):
    """(s, r, v) in FP64."""
    s = np.asarray(x, dtype=np.float64)
    if residual is not None:
        s = s + np.asarray(residual, dtype=np.float64)
    r = 1.0 / np.sqrt(np.mean(s * s, axis=1) + eps)
    return s, r, s * r[:, None] * np.asarray(weight, dtype=np.float64)


def ref_rms_norm_backward(dy, s, weight, rstd, dresidual=None):
    """(dx, dw, scale of dx's terms, sum of dw's absolute terms) in FP64, for the given rstd."""
    dy, s, w = (np.asarray(t, dtype=np.float64) for t in (dy, s, weight))
    r = np.asarray(rstd, dtype=np.float64)[:, None]
    xhat = s * r
    g = dy * w
    dx = r * (g - xhat * np.mean(g * xhat, axis=1, keepdims=True))
    terms = r * (np.abs(g) + np.abs(xhat) * np.mean(np.abs(g * xhat), axis=1, keepdims=True))
    if dresidual is not None:
        dx = dx + np.asarray(dresidual, dtype=np.float64)
        terms = terms + np.abs(np.asarray(dresidual, dtype=np.float64))
    return dx, np.sum(dy * xhat, axis=0), terms, np.sum(np.abs(dy * xhat), axis=0)
