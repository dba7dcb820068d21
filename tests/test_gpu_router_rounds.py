"""GPU tests of batches whose workgroups take several rounds of rows (16 rows a round with 16 lanes a row, 8 and 4 with 32 and
64, on at most 1280 workgroups), forward and backward: the LDS rows are used again and sums carried on."""

import numpy as np
import pytest
import torch

import oracle

pytestmark = pytest.mark.gpu

if torch.cuda.is_available():  # pragma: no cover - GPU only
    import moe_grouped_gemm_tiles_amd as dg
    from tests._gpu_harness import DEV, as_f64
    from tests.test_gpu_router import DT, STEP, backward, forward, tolerance

# rows, experts, top_k: three rounds and a ragged rest, and lanes of a row
CASES = [(2 * 20480 + 1237, 256, 8), (2 * 20480 + 5, 60, 6), (2 * 10240 + 77, 256, 20), (2 * 10240 + 3, 400, 4),
         (2 * 5120 + 2, 1000, 3)]


def batch(m, e, dtype):
    gen = torch.Generator(device=DEV).manual_seed(m)
    x = (1.5 * torch.randn(m, e, device=DEV, generator=gen)).to(DT[dtype])
    mask = torch.rand(m, device=DEV, generator=gen) < 0.8
    bias = 0.1 * torch.randn(e, device=DEV, generator=gen)
    rows = np.unique(np.concatenate([np.arange(40), np.arange(m - 40, m), np.random.default_rng(m).integers(0, m, 400)]
                                    + [np.arange(r - 20, r + 20) for r in (m // 3, 2 * m // 3)]))
    return x, mask, bias, torch.from_numpy(rows).to(DEV), gen


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("m,e,k", CASES)
def test_forward_of_several_rounds(m, e, k, score, dtype):
    x, mask, bias, rows, _ = batch(m, e, dtype)
    for b in (None, bias):
        out = forward(x, k, score=score, bias=b, mask=mask)
        some = as_f64(x[rows])
        ref = oracle.ref_router(some, k, score, bias=None if b is None else as_f64(b), mask=mask[rows].cpu().numpy())
        np.testing.assert_array_equal(out["ids"][rows].cpu().numpy(), ref["ids"])
        tol = 3 * tolerance(some)
        np.testing.assert_allclose(as_f64(out["weights"][rows]), ref["weights"], rtol=tol, atol=1e-37)
        flat = out["ids"].flatten().long()
        assert bool(((flat < 0).view(m, k).all(1) == ~mask).all())
        counts = torch.bincount(flat[flat >= 0], minlength=e)
        assert torch.equal(out["counts"].long(), counts)
        p = x.double().softmax(1) if score == "softmax" else x.double().sigmoid()
        total = (p / p.sum(1, keepdim=True) * mask[:, None]).sum(0)
        # FP32 sums of three rows a lane and 16 lanes a workgroup at most, FP64 after them: 20 roundings and the share's own
        tol = tolerance(as_f64(x)) + 20 * STEP
        np.testing.assert_allclose(as_f64(out["prob_sum"]), as_f64(total), rtol=tol)
        loss = e * float((counts.double() * total).sum() / (counts.sum() * total.sum()))
        np.testing.assert_allclose(float(out["loss"]), loss, rtol=2 * tol)
        again = forward(x, k, score=score, bias=b, mask=mask)
        assert all(torch.equal(out[n], again[n]) for n in out)


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("m,e,k", CASES)
def test_gradient_of_several_rounds(m, e, k, score, dtype):
    x, mask, _, rows, gen = batch(m, e, dtype)
    f = forward(x, k, score=score, mask=mask)
    dw = torch.randn(m, k, device=DEV, generator=gen)
    stats = (f["counts"], f["prob_sum"], torch.tensor([3.0 * m], device=DEV))
    dx = backward(x, f["ids"], dw, stats, score=score)
    some = as_f64(x[rows])
    ref, mag = oracle.ref_router_backward(some, f["ids"][rows].cpu().numpy(), as_f64(dw[rows]), f["counts"].cpu().numpy(),
                                          as_f64(f["prob_sum"]), 3.0 * m, score=score)
    # four factors of a score and three sums of at most 1 + 22 + top_k roundings
    tol = (4 * tolerance(some) + 3 * (30 + k) * STEP) * mag + 1e-37
    if dtype == "bf16":
        tol = tol + 2.0 ** -8 * (np.abs(ref) + tol) + 2.0 ** -133
    got = as_f64(dx[rows])
    assert (np.abs(got - ref) <= tol).all()
    assert not dx[~mask].any()
    # a row's gradient depends on nothing but the row and the sums: the same bits alone, and over the logits
    alone = backward(x[rows].contiguous(), f["ids"][rows].contiguous(), dw[rows].contiguous(), stats, score=score)
    assert torch.equal(alone, dx[rows])
    inplace = x.clone()
    backward(inplace, f["ids"], dw, stats, out=inplace, score=score)
    assert torch.equal(inplace, dx)


def test_batches_take_several_rounds():
    """The workspace holds one partial row a workgroup: no more than 1280, fewer than a round of these batches needs."""
    lib = dg.load_library()
    for m, e, k in CASES:
        lanes = 16 if e <= 256 and k < 16 else 32 if e <= 512 and k < 32 else 64
        assert m > 2 * 1280 * (256 // lanes) and lib.dg_get_moe_router_workspace_size(m, e) <= 2048 + 1280 * e * 8
