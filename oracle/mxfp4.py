"""Microscaled 4-bit operands (OCP MXFP4) in FP64: the quantisation, the decode and the products.

E2M1 from its closed form: one sign bit, two exponent bits with bias 1, one mantissa bit.  A block is
32 consecutive K values of a row with one E8M0 scale 2^(e - 127) (255 = NaN).  Two codes a byte, the
even K value in the low four bits; four scale bytes a word along K, words transposed [K/128, ld].
"""

from __future__ import annotations

import numpy as np

E2M1_TABLE = np.array([(-1.0 if c & 8 else 1.0) * ((c & 1) * 0.5 if (c >> 1) & 3 == 0
                                                   else (1 + (c & 1) * 0.5) * 2.0 ** (((c >> 1) & 3) - 1))
                       for c in range(16)])


def scale_byte(amax: float) -> int:
    """Byte of the smallest power of two s >= 2^-127 with amax <= 6 s (127 for an empty block)."""
    if not np.isfinite(amax):
        return 255
    if amax == 0:
        return 127
    e = -127
    while 6.0 * 2.0 ** e < amax:
        e += 1
    return e + 127


def _nearest_code(v: np.ndarray) -> np.ndarray:
    """Codes of the magnitudes nearest to |v| (ties to the even code), with v's sign."""
    mags = E2M1_TABLE[:8]
    dist = np.abs(np.abs(v)[..., None] - mags)
    best = dist.min(-1, keepdims=True)
    tied = dist == best
    # of two neighbours at the same distance exactly one has an even code
    code = np.where(tied & (np.arange(8) % 2 == 0), np.arange(8), -1).max(-1)
    code = np.where(tied.sum(-1) == 1, tied.argmax(-1), code)
    return (code + 8 * np.signbit(v)).astype(np.uint8)


def ref_cast_mxfp4(x: np.ndarray):
    """x [rows, K] (finite or not) -> packed codes [rows, K/2], scale bytes [rows, K/32], values FP64 [rows, K]."""
    rows, k = x.shape
    b = x.astype(np.float64).reshape(rows, k // 32, 32)
    with np.errstate(invalid="ignore"):
        amax = np.abs(b).max(-1)  # NaN wins
    byte = np.array([scale_byte(a) for a in amax.ravel()], dtype=np.uint8).reshape(amax.shape)
    s = 2.0 ** (np.where(byte == 255, 127, byte).astype(np.float64) - 127)
    bad = (byte == 255)[..., None]
    code = np.where(bad, 0, _nearest_code(np.where(bad, 0.0, b) / s[..., None])).astype(np.uint8)
    y = np.where(bad, np.nan, E2M1_TABLE[code] * s[..., None]).reshape(rows, k)
    code = code.reshape(rows, k)
    return code[:, 0::2] | (code[:, 1::2] << 4), byte, y


def pack_scale_words(byte: np.ndarray, ld: int | None = None, fill: int = 0x7F7F7F7F) -> np.ndarray:
    """Scale bytes [rows, K/32] -> int32 words [K/128, ld], `fill` in the columns past the rows."""
    rows, nb = byte.shape
    w = byte.reshape(rows, nb // 4, 4).astype(np.uint32)
    out = np.full((nb // 4, rows if ld is None else ld), fill, dtype=np.uint32)
    out[:, :rows] = (w[..., 0] | w[..., 1] << 8 | w[..., 2] << 16 | w[..., 3] << 24).T
    return out.view(np.int32)


def decode_mxfp4(q: np.ndarray, byte: np.ndarray) -> np.ndarray:
    """Packed codes [rows, K/2] and scale bytes [rows, K/32] -> FP64 [rows, K]."""
    rows = q.shape[0]
    code = np.empty((rows, 2 * q.shape[1]), dtype=np.uint8)
    code[:, 0::2], code[:, 1::2] = q & 15, q >> 4
    s = np.where(byte == 255, np.nan, 2.0 ** (byte.astype(np.float64) - 127))
    return E2M1_TABLE[code] * np.repeat(s, 32, axis=1)


def ref_mxfp4(a, b, c=None):
    """(D, S): D = C + A @ B.T and the sums of magnitudes |C| + |A| @ |B|.T that bound its roundings; a and b are
    (codes, scale bytes) pairs."""
    va, vb = decode_mxfp4(*a), decode_mxfp4(*b)
    d, s = va @ vb.T, np.abs(va) @ np.abs(vb).T
    return (d, s) if c is None else (d + c, s + np.abs(c))
