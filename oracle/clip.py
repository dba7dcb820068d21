"""Global norm over many tensors and clipping by it.
TEST INFRASTRUCTURE ONLY.
"""

from __future__ import annotations

import math

import numpy as np


def ref_clip(grads, max_norm: float):
    """(norm, clipped FP64 arrays); the squares are summed exactly rounded."""
    norm = math.sqrt(math.fsum(math.fsum(np.square(np.asarray(g, dtype=np.float64)).ravel()) for g in grads))
    c = 1.0 if math.isinf(max_norm) else min(1.0, max_norm / (norm + 1e-6))
    return norm, [np.asarray(g, dtype=np.float64) * c for g in grads]
