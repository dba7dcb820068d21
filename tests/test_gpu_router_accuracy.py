"""GPU tests of the router's scores and gradients far below the largest score, where an exponential of a rounded argument
would be off by twice its distance.

In steps of 2^-24 relative: the exponential 3 (its instruction's last place is 2, one rounding), 1 + e one, a quotient
or product one each.  Logits are multiples of 1/64, so that their distances are exact.
"""

import numpy as np
import pytest
import torch

pytestmark = pytest.mark.gpu

if torch.cuda.is_available():  # pragma: no cover - GPU only
    from tests._gpu_harness import DEV, as_f64
    from tests.test_gpu_router import STEP, backward, forward

SIZES = [12, 60]  # all experts are chosen: rows of 16 and of 64 lanes


def wide(e, low, high, m=400):
    rng = np.random.default_rng(e)
    return np.round(rng.uniform(64 * low, 64 * high, (m, e))) / 64


def close(got, ref, steps):
    off = np.abs(got - ref) / np.abs(ref) / STEP
    assert off.max() <= steps, off.max()


@pytest.mark.parametrize("e", SIZES)
def test_sigmoids(e):
    x = wide(e, -80, 30)
    t = torch.from_numpy(x.astype(np.float32)).to(DEV)
    out = forward(t, e, score="sigmoid", normalize=False)
    ids = out["ids"].cpu().numpy()
    ref = np.take_along_axis(1 / (1 + np.exp(-x)), ids, 1)
    close(as_f64(out["weights"]), ref, 3 + 1 + 1)


@pytest.mark.parametrize("e", SIZES)
def test_softmax_relative_to_its_largest(e):
    x = wide(e, -80, 0)
    x[:, 3] = 0.25  # the largest, whose exponential is 1
    t = torch.from_numpy(x.astype(np.float32)).to(DEV)
    out = forward(t, e, score="softmax", normalize=False)
    ids, w = out["ids"].cpu().numpy(), as_f64(out["weights"])
    assert (ids[:, 0] == 3).all()
    close(w / w[:, :1], np.take_along_axis(np.exp(x - 0.25), ids, 1), (3 + 1) + 1)


@pytest.mark.parametrize("e", SIZES)
def test_sigmoid_gradient(e):
    """Weights are the sigmoids: the gradient is dw p (1 - p), e r^2 with e = exp(-|x|) and r = 1 / (1 + e)."""
    x = wide(e, -80, 80)
    t = torch.from_numpy(x.astype(np.float32)).to(DEV)
    ids = torch.arange(e, dtype=torch.int32, device=DEV).repeat(len(x), 1)
    dw = torch.randn(len(x), e, generator=torch.Generator().manual_seed(1)).to(DEV)
    dx = as_f64(backward(t, ids, dw, score="sigmoid", normalize=False))
    a = np.exp(-np.abs(x))
    close(dx, as_f64(dw) * a / (1 + a) ** 2, 3 + 2 * 1 + 2 + 1)


@pytest.mark.parametrize("e", SIZES)
def test_softmax_gradient_of_experts_that_are_not_chosen(e):
    """It is -p times what all of a row share."""
    x = wide(e, -80, 0)
    x[:, 3], x[:, 5] = 0.25, 0.0
    t = torch.from_numpy(x.astype(np.float32)).to(DEV)
    ids = torch.full((len(x), 1), 3, dtype=torch.int32, device=DEV)
    dx = as_f64(backward(t, ids, torch.ones(len(x), 1, device=DEV), score="softmax", normalize=False))
    others = [i for i in range(e) if i != 3]
    close(dx[:, others] / dx[:, 5:6], np.exp(x[:, others]), 2 * (3 + 2))
