"""CPU pins of the oracle's 4-bit operands and router: closed forms, torch's float64 autograd, planted mistakes."""

import itertools
from fractions import Fraction

import numpy as np
import pytest
import torch

import oracle
from oracle.mxfp4 import scale_byte


def test_e2m1_values():
    assert oracle.E2M1_TABLE[:8].tolist() == [0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0]
    assert (oracle.E2M1_TABLE[8:] == -oracle.E2M1_TABLE[:8]).all()


def test_scale_is_the_smallest_power_of_two_that_fits():
    rng = np.random.default_rng(0)
    for a in list(rng.uniform(1, 2, 40) * 2.0 ** rng.integers(-120, 120, 40)) + [6.0, 6.0 * (1 + 2 ** -23), 3.0, 0.75, 2.0 ** -126]:
        e = scale_byte(float(a)) - 127
        assert Fraction(a) <= 6 * Fraction(2) ** e and (e == -127 or Fraction(a) > 6 * Fraction(2) ** (e - 1))
    assert scale_byte(0.0) == 127 and scale_byte(float("inf")) == 255 and scale_byte(float("nan")) == 255
    assert scale_byte(2.0 ** -149) == 0 and scale_byte(float(np.finfo(np.float32).max)) == 127 + 126


def test_codes_round_to_nearest_even():
    # every midpoint, and both neighbours of each, in a block whose scale is 1
    mags = oracle.E2M1_TABLE[:8]
    for lo, hi in zip(range(7), range(1, 8)):
        mid = (mags[lo] + mags[hi]) / 2
        x = np.zeros((1, 32))
        x[0, :7] = [6.0, mid, np.nextafter(mid, 0), np.nextafter(mid, 9), -mid, -0.0, 1e-9]
        q, byte, y = oracle.ref_cast_mxfp4(x)
        assert byte[0, 0] == 127
        even = mags[lo] if lo % 2 == 0 else mags[hi]
        assert y[0, :7].tolist() == [6.0, even, mags[lo], mags[hi], -even, 0.0, 0.0]
        codes = [c for b in q[0] for c in (b & 15, b >> 4)]
        assert codes[5] == 8  # the sign of a zero stays


def test_error_bound_and_round_trip():
    rng = np.random.default_rng(1)
    x = rng.standard_normal((8, 256)) * np.exp(rng.standard_normal((8, 1)) * 4)
    q, byte, y = oracle.ref_cast_mxfp4(x.astype(np.float32))
    assert (oracle.decode_mxfp4(q, byte) == y).all()
    s = np.repeat(2.0 ** (byte.astype(float) - 127), 32, axis=1)
    assert (np.abs(y - x.astype(np.float32)) <= s).all()  # half of the largest step, 2 s
    q2, byte2, y2 = oracle.ref_cast_mxfp4(y)
    assert (y2 == y).all()  # values on a grid keep themselves


def test_scale_words_are_transposed_little_endian():
    byte = np.arange(24, dtype=np.uint8).reshape(3, 8)
    w = oracle.pack_scale_words(byte, ld=4)
    assert w.shape == (2, 4) and (w[:, 3] == 0x7F7F7F7F).all()
    for r, qq in itertools.product(range(3), range(2)):
        assert w[qq, r:r + 1].view(np.uint8).tolist() == byte[r, 4 * qq:4 * qq + 4].tolist()


def test_products_against_rationals():
    rng = np.random.default_rng(2)
    k = 64
    a = (rng.integers(0, 256, (3, k // 2), dtype=np.uint8), rng.integers(120, 134, (3, k // 32), dtype=np.uint8))
    b = (rng.integers(0, 256, (2, k // 2), dtype=np.uint8), rng.integers(120, 134, (2, k // 32), dtype=np.uint8))
    d, s = oracle.ref_mxfp4(a, b)

    def value(op, r, i):
        code = int(op[0][r, i // 2]) >> (4 * (i % 2)) & 15
        return Fraction(float(oracle.E2M1_TABLE[code])) * Fraction(2) ** (int(op[1][r, i // 32]) - 127)

    for i, j in itertools.product(range(3), range(2)):
        terms = [value(a, i, t) * value(b, j, t) for t in range(k)]
        assert float(sum(terms)) == d[i, j] and float(sum(map(abs, terms))) == s[i, j]
    byte = a[1].copy()
    byte[1, 0] = 255
    d, _ = oracle.ref_mxfp4((a[0], byte), b)
    assert np.isnan(d[1]).all() and np.isfinite(d[[0, 2]]).all()


def _torch_router(x, ids, score, normalize, scale):
    p = torch.softmax(x, 1) if score == "softmax" else torch.sigmoid(x)
    share = p if score == "softmax" else p / (p.sum(1, keepdim=True) + 1e-20)
    w = torch.gather(p, 1, ids)
    if normalize:
        w = w / (w.sum(1, keepdim=True) + 1e-20)
    return w * scale, share.sum(0)


@pytest.mark.parametrize("score,normalize", itertools.product(["softmax", "sigmoid"], [True, False]))
def test_router_and_its_gradient_against_autograd(score, normalize):
    rng = np.random.default_rng(3)
    m, e, k, scale = 17, 9, 3, 1.7
    x = rng.standard_normal((m, e)) * 2
    r = oracle.ref_router(x, k, score, normalize=normalize, scale=scale)
    t = torch.tensor(x, requires_grad=True)
    top, ids = torch.topk(t.detach(), k, dim=1)
    assert (ids.numpy() == r["ids"]).all()
    w, s = _torch_router(t, ids, score, normalize, scale)
    np.testing.assert_allclose(w.detach().numpy(), r["weights"], rtol=1e-12)
    counts = torch.bincount(ids.flatten(), minlength=e).double()
    loss = e * (counts * s).sum() / (counts.sum() * m)
    np.testing.assert_allclose(float(loss), r["loss"], rtol=1e-12)
    dw = torch.tensor(rng.standard_normal((m, k)))
    ((w * dw).sum() + 3.0 * loss).backward()
    dx, mag = oracle.ref_router_backward(x, r["ids"], dw.numpy(), r["counts"], r["prob_sum"], 3.0, score, normalize, scale)
    np.testing.assert_allclose(dx, t.grad.numpy(), rtol=1e-9, atol=1e-12)
    assert (np.abs(dx) <= mag * (1 + 1e-12)).all()


@pytest.mark.parametrize("score,normalize", itertools.product(["softmax", "sigmoid"], [True, False]))
def test_router_gradient_against_differences(score, normalize):
    rng = np.random.default_rng(4)
    m, e, k = 5, 7, 2
    x = rng.standard_normal((m, e))
    r = oracle.ref_router(x, k, score, normalize=normalize)
    dw = rng.standard_normal((m, k))
    dx, _ = oracle.ref_router_backward(x, r["ids"], dw, r["counts"], r["prob_sum"], 2.0, score, normalize)

    def value(z):
        s = oracle.ref_router(z, k, score, normalize=normalize)
        assert (s["ids"] == r["ids"]).all()
        return (s["weights"] * dw).sum() + 2.0 * s["loss"]

    for t, j in itertools.product(range(m), range(e)):
        step = np.zeros_like(x)
        step[t, j] = 1e-6
        np.testing.assert_allclose((value(x + step) - value(x - step)) / 2e-6, dx[t, j], rtol=1e-5, atol=1e-7)


def test_router_ties_masks_and_dead_experts():
    x = np.array([[1.0, 1.0, 0.5, 1.0], [-np.inf, 2.0, -np.inf, -np.inf], [-np.inf] * 4, [0.0, 1.0, 2.0, 3.0]])
    r = oracle.ref_router(x, 2, mask=[True, True, True, False])
    assert r["ids"].tolist() == [[0, 1], [1, -1], [-1, -1], [-1, -1]]
    assert r["counts"].tolist() == [1, 2, 0, 0] and r["weights"][1].tolist() == [1.0, 0.0]
    np.testing.assert_allclose(r["prob_sum"].sum(), 2.0)
    dx, _ = oracle.ref_router_backward(x, r["ids"], np.ones((4, 2)), r["counts"], r["prob_sum"], 1.0)
    assert (dx[2:] == 0).all() and (dx[1] == 0).all()
    # the bias steers the choice and nothing else
    b = oracle.ref_router(x[:1], 2, "sigmoid", bias=[0, 0, 1.0, 0])
    assert b["ids"].tolist() == [[2, 0]] and b["weights"][0, 0] < b["weights"][0, 1]


def test_balanced_choice_has_loss_one():
    x = np.where((np.arange(8)[:, None] % 4) == np.arange(4), 1.0, 0.0)
    assert abs(oracle.ref_router(x, 1)["loss"] - 1.0) < 1e-12
    skew = oracle.ref_router(np.tile([3.0, 0, 0, 0], (8, 1)), 1)["loss"]
    assert skew > 3.0


def test_planted_mistakes_are_seen():
    x = np.array([[1.0, 1.0, 0.5, 2.0]])
    r = oracle.ref_router(x, 3)
    highest_first = [3, 1, 0]  # ties to the higher index
    assert r["ids"][0].tolist() != highest_first
    v = np.zeros((1, 32))
    v[0, :2] = [6.0, 2.5]
    assert oracle.ref_cast_mxfp4(v)[2][0, 1] == 2.0 != 3.0  # away from the even code
    assert scale_byte(7.0) == 128 != 127  # the rule that lets the largest value clip
