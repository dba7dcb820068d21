"""The division steps of the FP8 casts and the norm (``csrc/dg_cast.hpp``, ``csrc/dg_norm.hip``) in FP32
arithmetic emulated on the CPU: amax / 448 from a rounded 1/448 and two corrections is the correctly rounded
quotient for every mantissa, and so is x / s from a refined reciprocal, on a sample."""

import numpy as np


def _fma(a, b, c):
    """float32 a * b + c rounded once: the product is exact in FP64, the sum is rounded to odd there (its error is
    known exactly and put into the last bit), and FP64's 53 bits leave room for the final rounding to 24."""
    p = a.astype(np.float64) * np.asarray(b, np.float32).astype(np.float64)
    c = np.asarray(c, np.float32).astype(np.float64)
    s = p + c
    t = s - p
    err = (p - (s - t)) + (c - t)
    bits = s.view(np.int64)
    # truncate towards zero where the rounding went away from it, then set the last bit of inexact sums
    away = (err != 0) & ((err < 0) == (s > 0)) & (s != 0)
    bits = bits - away.astype(np.int64)
    return np.where(err != 0, bits | 1, bits).view(np.float64).astype(np.float32)


def _quotient(x, s, y):
    """The norm's quotient(): x / s with y about 1 / s."""
    q0 = x * y
    q1 = _fma(-_fma(s, q0, -x), y, q0)
    return _fma(-_fma(s, q1, -x), y, q1)


def _div_by(x, s, y):
    """The plain cast's div_by(): the same corrections, the sign put back."""
    q0 = x * y
    q1 = _fma(_fma(-s, q0, x), y, q0)
    return np.copysign(_fma(_fma(-s, q1, x), y, q1), x)


def _all_mantissas(chunk):
    bits = np.arange(chunk << 20, (chunk + 1) << 20, dtype=np.uint32)
    return (bits | np.uint32(0x3F800000)).view(np.float32)


def test_emulated_fma():
    """Against exact integers: products and sums whose bits reach past FP64's."""
    from fractions import Fraction
    rng = np.random.default_rng(1)
    a, b = (rng.standard_normal(4000).astype(np.float32) for _ in range(2))
    c = (-(a.astype(np.float64) * b) * rng.choice([1, 1 + 2.0 ** -20, 2.0 ** -30, 2.0 ** 30], 4000)).astype(np.float32)
    got = _fma(a, b, c)
    for x, y, z, g in zip(a, b, c, got):
        exact = Fraction(float(x)) * Fraction(float(y)) + Fraction(float(z))
        lo, hi = np.nextafter(g, np.float32(-np.inf)), np.nextafter(g, np.float32(np.inf))
        d = abs(exact - Fraction(float(g)))
        assert d <= abs(exact - Fraction(float(lo))) and d <= abs(exact - Fraction(float(hi)))


def test_scale_for_every_mantissa_of_amax():
    """All 2^23 mantissas; other exponents only shift them (the steps' range is checked by the kernels)."""
    s = np.float32(448.0)
    y = np.float32(1.0) / s
    for chunk in range(8):
        a = _all_mantissas(chunk)
        assert np.array_equal(_quotient(a, np.full_like(a, s), y), a / s)


def test_quotients_of_a_blocks_values():
    """x / s for scales of random mantissas and |x| <= 448 s, from the reciprocal the kernels refine: whatever
    estimate within 1 ulp the hardware gives."""
    rng = np.random.default_rng(2)
    n = 400_000
    s = (rng.integers(0, 1 << 23, n).astype(np.uint32) | np.uint32(0x3F800000)).view(np.float32)
    x = (s.astype(np.float64) * rng.uniform(2.0 ** -9, 448, n) * rng.choice([-1, 1], n)).astype(np.float32)
    exact = (np.float32(1) / s).astype(np.float32)
    for off in (-1, 0, 1):
        r = (exact.view(np.int32) + off).astype(np.int32).view(np.float32)
        y = _fma(_fma(-s, r, np.ones_like(s)), r, r)
        assert np.array_equal(_quotient(x, s, y), x / s)
        assert np.array_equal(_div_by(x, s, y), x / s)
