"""GPU tests of the router with logits that are not finite and with slots that have no expert, against the FP64 oracle."""

import itertools

import numpy as np
import pytest
import torch

import oracle

pytestmark = pytest.mark.gpu

if torch.cuda.is_available():  # pragma: no cover - GPU only
    from tests._gpu_harness import DEV, as_f64
    from tests.test_gpu_router import STEP, backward, forward, logits, tolerance

# experts and top_k of each number of lanes a row has, with and without room for all experts among the chosen
LAYOUTS = [(12, 12), (60, 4), (200, 15), (256, 20), (400, 6), (1000, 64)]


def bad_logits(e, dtype):
    """Rows with a NaN, with +inf, with both, of NaN alone, of -inf and one NaN, with several +inf; others ordinary."""
    x = logits(40, e, dtype, seed=e)
    x[3, 5 % e], x[7, e - 1], x[11, 0], x[11, e // 2] = float("nan"), float("inf"), float("inf"), float("nan")
    x[15] = float("nan")
    x[19] = -float("inf")
    x[19, 1 % e] = float("nan")
    x[23, : e // 3] = float("inf")
    return x


def check_nan_alike(got, ref, tol, what):
    np.testing.assert_array_equal(np.isnan(got), np.isnan(ref), err_msg=what)
    np.testing.assert_allclose(got, ref, rtol=tol, atol=1e-37, err_msg=what)


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("score,normalize", itertools.product(["softmax", "sigmoid"], [True, False]))
@pytest.mark.parametrize("e,k", LAYOUTS)
def test_nan_and_inf_logits(e, k, score, normalize, dtype):
    x = bad_logits(e, dtype)
    for bias, masked in itertools.product((None, (0.1 * np.random.default_rng(e).standard_normal(e)).astype(np.float32)), (False, True)):
        mask = np.isfinite(as_f64(x)).all(1) if masked else None
        out = forward(x, k, score=score, normalize=normalize, bias=None if bias is None else torch.from_numpy(bias).to(DEV),
                      mask=None if mask is None else torch.from_numpy(mask).to(DEV))
        ref = oracle.ref_router(as_f64(x), k, score, bias=bias, mask=mask, normalize=normalize)
        np.testing.assert_array_equal(out["ids"].cpu().numpy(), ref["ids"])
        np.testing.assert_array_equal(out["counts"].cpu().numpy(), ref["counts"])
        tol = 3 * tolerance(as_f64(x))
        for n in ("weights", "prob_sum", "loss"):  # sums of 40 rows in FP32
            check_nan_alike(as_f64(out[n]), np.broadcast_to(ref[n], out[n].shape), 2 * (tol + 40 * 2.0 ** -24), n)
        assert masked == bool(np.isfinite(as_f64(out["loss"])).all())
        assert not as_f64(out["weights"])[ref["ids"] < 0].any()


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("m", [30, 3000])
def test_no_loss_where_nothing_is_chosen(score, m):
    """A bias of NaN takes every expert out; the rows' shares may still be NaN."""
    x = logits(m, 20, "fp32")
    bias = torch.full((20,), float("nan"), device=DEV)
    for nan in (False, True):
        if nan:
            x[5, 3] = float("nan")
        out = forward(x, 4, score=score, bias=bias)
        assert (out["ids"] == -1).all() and not out["weights"].any() and not out["counts"].any() and float(out["loss"]) == 0.0
        assert bool(torch.isnan(out["prob_sum"]).all()) == nan


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
def test_slots_without_an_expert_weigh_nothing_at_any_scale(score):
    x = logits(50, 16, "fp32", dead=13)
    mask = torch.rand(50, generator=torch.Generator().manual_seed(1)).to(DEV) < 0.5
    for scale in (0.0, 1e-30, 1e20, 3e38):
        out = forward(x, 6, score=score, mask=mask, scale=scale)
        assert bool(((out["ids"] >= 0).sum(1) == torch.where(mask, 3, 0)).all())
        assert not out["weights"][out["ids"] < 0].any()


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("score,normalize", itertools.product(["softmax", "sigmoid"], [True, False]))
@pytest.mark.parametrize("e,k", LAYOUTS)
def test_gradient_of_nan_and_inf_logits(e, k, score, normalize, dtype):
    """NaN where the formula has it.  Without the loss a sigmoid's NaN is its own expert's alone."""
    x = bad_logits(e, dtype)
    ok = torch.from_numpy(np.isfinite(as_f64(x)).all(1)).to(DEV)
    f, sums = forward(x, k, score=score, normalize=normalize), forward(x, k, score=score, normalize=normalize, mask=ok)
    dw = torch.randn(40, k, generator=torch.Generator().manual_seed(2)).to(DEV)
    for stats in ((sums["counts"], sums["prob_sum"], torch.tensor([100.0], device=DEV)), None):
        c, s, dl = (None, None, 0.0) if stats is None else (stats[0].cpu().numpy(), as_f64(stats[1]), float(stats[2]))
        with np.errstate(invalid="ignore"):
            ref, mag = oracle.ref_router_backward(as_f64(x), f["ids"].cpu().numpy(), as_f64(dw), c, s, dl, score=score, normalize=normalize)
        got = as_f64(backward(x, f["ids"], dw, stats, score=score, normalize=normalize))
        np.testing.assert_array_equal(np.isnan(got), np.isnan(ref))
        # four factors of a score and three sums of at most 1 + 22 + top_k roundings, and BF16's own
        tol = (4 * tolerance(as_f64(x)) + 3 * (30 + k) * STEP) * mag + 1e-37
        if dtype == "bf16":
            tol = tol + 2.0 ** -8 * (np.abs(ref) + tol) + 2.0 ** -133
        live = ~np.isnan(ref)
        assert (np.abs(got - ref)[live] <= tol[live]).all()
        if score == "sigmoid" and stats is None:
            assert not np.isnan(got[np.isfinite(as_f64(x))]).any()
