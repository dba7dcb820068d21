"""A gated expert layer, written out token by token.
TEST INFRASTRUCTURE ONLY.

For token t and slot j with e = ids[t, j] in [0, E):

    h = x_t @ W13[e]^T,   a = silu(h[:I]) * h[I:],   out_t += weights[t, j] * (a @ W2[e]^T)

in FP64 from the dequantised operands; other ids add nothing.  Beside the
result come the sums of absolute values that bound a kernel's rounding:
``second`` for roundings of a (and of the products of the second GEMM),
``first`` for errors of the first GEMM's FP32 accumulation carried through the
activation (|d silu / dg| <= 1.1).
"""

from __future__ import annotations

import numpy as np

from .gemm import dequant_a, dequant_b
from .ue8m0 import decode_ue8m0_sf


def silu(g):
    return g / (1.0 + np.exp(-g))


def ref_moe(x, sfx, w13, sf13, w2, sf2, ids, weights, ue8m0: bool = False):
    """(out, second, first), each FP64 [M, H]."""
    m, h = x.shape
    e_n, i = w13.shape[0], w13.shape[1] // 2
    if ue8m0:
        sfx = decode_ue8m0_sf(sfx, h // 128, axis=0)
        sf13 = decode_ue8m0_sf(sf13, h // 128, axis=2)
        sf2 = decode_ue8m0_sf(sf2, i // 128, axis=2)
    xd = dequant_a(x, sfx)
    out, second, first = (np.zeros((m, h)) for _ in range(3))
    for e in range(e_n):
        tok, slot = np.nonzero(ids == e)
        if len(tok) == 0:
            continue
        a13, a2 = dequant_b(w13[e], sf13[e]), dequant_b(w2[e], sf2[e])
        hid, mag = xd[tok] @ a13.T, np.abs(xd[tok]) @ np.abs(a13).T
        act = silu(hid[:, :i]) * hid[:, i:]
        slack = 1.1 * np.abs(hid[:, i:]) * mag[:, :i] + np.abs(silu(hid[:, :i])) * mag[:, i:]
        w = np.asarray(weights, dtype=np.float64)[tok, slot][:, None]
        np.add.at(out, tok, w * (act @ a2.T))
        np.add.at(second, tok, np.abs(w) * (np.abs(act) @ np.abs(a2).T))
        np.add.at(first, tok, np.abs(w) * (slack @ np.abs(a2).T))
    return out, second, first
