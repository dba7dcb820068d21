"""CPU pins of the oracle of the norm, the expert layer and the clipping:
closed forms, central differences, torch's autograd and properties."""

import math

import numpy as np
import pytest
import torch

import oracle
from workloads import gen_moe


def test_norm_of_constant_rows_and_scaling():
    x = np.full((2, 256), 3.0)
    s, r, v = oracle.ref_add_rms_norm(x, np.arange(256.0), 0.0, residual=np.full((2, 256), -1.0))
    assert (s == 2.0).all() and np.allclose(r, 0.5) and np.allclose(v, np.arange(256.0))
    rng = np.random.default_rng(1)
    x = rng.standard_normal((3, 128))
    assert np.allclose(oracle.ref_add_rms_norm(8 * x, np.ones(128), 0.0)[2],
                       oracle.ref_add_rms_norm(x, np.ones(128), 0.0)[2])


def test_norm_gradient_matches_central_differences():
    """Directional central differences of sum(dy * v) in FP64: error O(h^2) ~ 1e-8 at h = 1e-4."""
    rng = np.random.default_rng(2)
    x, w, dy = rng.standard_normal((3, 128)), 1 + 0.1 * rng.standard_normal(128), rng.standard_normal((3, 128))
    eps, h = 1e-5, 1e-4
    _, r, _ = oracle.ref_add_rms_norm(x, w, eps)
    dx, dw, _, _ = oracle.ref_rms_norm_backward(dy, x, w, r)

    def loss(x_, w_):
        return float(np.sum(dy * oracle.ref_add_rms_norm(x_, w_, eps)[2]))

    for k in range(5):
        d = rng.standard_normal(x.shape)
        got = (loss(x + h * d, w) - loss(x - h * d, w)) / (2 * h)
        assert math.isclose(got, float(np.sum(dx * d)), rel_tol=1e-6, abs_tol=1e-6)
        d = rng.standard_normal(w.shape)
        got = (loss(x, w + h * d) - loss(x, w - h * d)) / (2 * h)
        assert math.isclose(got, float(np.sum(dw * d)), rel_tol=1e-6, abs_tol=1e-6)


def test_norm_gradient_matches_autograd_with_skip_path():
    rng = np.random.default_rng(3)
    x, res, dy, dres = (rng.standard_normal((4, 256)) for _ in range(4))
    w = rng.standard_normal(256)
    tx, tr, tw = (torch.tensor(t, requires_grad=True) for t in (x, res, w))
    s = tx + tr
    v = s * torch.rsqrt(s.square().mean(1, keepdim=True) + 1e-6) * tw
    ((v * torch.tensor(dy)).sum() + (s * torch.tensor(dres)).sum()).backward()
    s64, r, _ = oracle.ref_add_rms_norm(x, w, 1e-6, residual=res)
    dx, dw, terms, mag = oracle.ref_rms_norm_backward(dy, s64, w, r, dres)
    assert np.allclose(dx, tx.grad.numpy()) and np.allclose(dx, tr.grad.numpy()) and np.allclose(dw, tw.grad.numpy())
    assert (terms >= np.abs(dx) - 1e-12).all() and (mag >= np.abs(dw) - 1e-12).all()


def test_norm_planted_mistakes_are_caught():
    rng = np.random.default_rng(4)
    x, w, dy = rng.standard_normal((2, 128)), rng.standard_normal(128), rng.standard_normal((2, 128))
    _, r, v = oracle.ref_add_rms_norm(x, w, 1e-6)
    dx = oracle.ref_rms_norm_backward(dy, x, w, r)[0]
    assert not np.allclose(r[:, None] * dy * w, dx, rtol=1e-2)              # projection dropped
    assert not np.allclose(v, (x - x.mean(1, keepdims=True)) * r[:, None] * w, rtol=1e-2)  # mean subtracted


@pytest.mark.parametrize("fmt", ["fp32", "ue8m0"])
def test_moe_matches_the_grouped_products(fmt):
    """The layer as two dense products per (token, slot) with the GEMM's own oracle."""
    x = gen_moe(5, 6, 3, 256, 128, seed=5, scale_fmt=fmt, routed=9)
    out, second, first = oracle.ref_moe(x["x"], x["sfx"], x["w13"], x["sf13"], x["w2"], x["sf2"], x["ids"], x["weights"],
                                        ue8m0=fmt == "ue8m0")
    ref = oracle.ref_dense_ue8m0 if fmt == "ue8m0" else oracle.ref_dense
    want = np.zeros_like(out)
    for t in range(5):
        for j in range(3):
            e = x["ids"][t, j]
            if not 0 <= e < 6:
                continue
            h = ref(x["x"], x["sfx"], x["w13"][e], x["sf13"][e], rows=[t])[0]
            a = h[:128] / (1 + np.exp(-h[:128])) * h[128:]
            w2 = oracle.dequant_b(x["w2"][e], oracle.decode_ue8m0_sf(x["sf2"][e], 1, 1) if fmt == "ue8m0" else x["sf2"][e])
            want[t] += float(x["weights"][t, j]) * (w2 @ a)
    assert np.allclose(out, want, rtol=1e-10, atol=1e-12)
    assert (second >= np.abs(out) - 1e-12).all() and (first >= 0).all()


def test_moe_without_local_experts_is_zero_and_linear_in_the_weights():
    x = gen_moe(4, 3, 2, 128, 128, seed=6, poison=True)
    args = (x["x"], x["sfx"], x["w13"], x["sf13"], x["w2"], x["sf2"])
    none = np.full_like(x["ids"], -1)
    assert (oracle.ref_moe(*args, none, np.full_like(x["weights"], np.nan))[0] == 0).all()
    one = oracle.ref_moe(*args, x["ids"], x["weights"])[0]
    assert np.isfinite(one).all()
    assert np.allclose(oracle.ref_moe(*args, x["ids"], 2 * x["weights"])[0], 2 * one)


def test_moe_planted_mistakes_are_caught():
    x = gen_moe(3, 2, 1, 128, 128, seed=7)
    out = oracle.ref_moe(x["x"], x["sfx"], x["w13"], x["sf13"], x["w2"], x["sf2"], x["ids"], x["weights"])[0]
    i = x["inter"]
    swapped = np.concatenate([x["w13"][:, i:], x["w13"][:, :i]], axis=1)  # up rows taken for gate rows
    sf = np.concatenate([x["sf13"][:, 1:], x["sf13"][:, :1]], axis=1)
    bad = oracle.ref_moe(x["x"], x["sfx"], swapped, sf, x["w2"], x["sf2"], x["ids"], x["weights"])[0]
    assert np.linalg.norm(bad - out) > 0.1 * np.linalg.norm(out)
    other = oracle.ref_moe(x["x"], x["sfx"], x["w13"], x["sf13"], x["w2"], x["sf2"], 1 - x["ids"], x["weights"])[0]
    assert np.linalg.norm(other - out) > 0.1 * np.linalg.norm(out)


def test_clip_closed_forms():
    n, out = oracle.ref_clip([np.array([3.0]), np.array([[4.0, 0.0]]), np.zeros(0)], 1.0)
    assert n == 5.0 and np.allclose(out[0], 0.6) and np.allclose(out[1], [[0.8, 0.0]]) and out[2].size == 0
    n, out = oracle.ref_clip([np.array([3.0])], 10.0)
    assert n == 3.0 and out[0][0] == 3.0
    n, out = oracle.ref_clip([np.array([1e30, 1e30], np.float32)], math.inf)
    assert math.isclose(n, math.sqrt(2) * 1e30, rel_tol=1e-6) and out[0][0] == np.float32(1e30)


def test_clip_matches_torch():
    rng = np.random.default_rng(8)
    ps = [torch.nn.Parameter(torch.zeros(n, dtype=torch.float64)) for n in (5, 1, 700)]
    gs = [rng.standard_normal(p.shape) for p in ps]
    for p, g in zip(ps, gs):
        p.grad = torch.tensor(g)
    n, out = oracle.ref_clip(gs, 0.5)
    assert math.isclose(float(torch.nn.utils.clip_grad_norm_(ps, 0.5)), n, rel_tol=1e-12)
    for p, o in zip(ps, out):
        assert np.allclose(p.grad.numpy(), o)
