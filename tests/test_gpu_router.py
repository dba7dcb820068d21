"""GPU tests of the router and its gradient against the FP64 oracle.

Choice and counts are whole numbers and equal.  Scores: with |x| <= R the exponential's argument is off by up to
2 R steps of 2^-24 (its rounding and the subtraction of the largest), the instruction by one, a sum of E terms in any
order by E - 1 roundings of non-negative terms at worst (a row's 16 values a lane, then six exchanges: at most 22),
quotients by a few: (2 R + 40) * 2^-24 relative, for each of the two or three factors.
"""

import itertools

import numpy as np
import pytest
import torch

import oracle

pytestmark = pytest.mark.gpu

if torch.cuda.is_available():  # pragma: no cover - GPU only
    import moe_grouped_gemm_tiles_amd as dg
    from tests._gpu_harness import DEV, as_f64

DT = {"bf16": torch.bfloat16, "fp32": torch.float32}
STEP = 2.0 ** -24


def forward(x, k, stats=True, workspace=None, **kw):
    m, e = x.shape
    out = dict(ids=torch.full((m, k), 99, dtype=torch.int32, device=DEV), weights=torch.full((m, k), 9.0, device=DEV))
    if stats:
        out.update(counts=torch.full((e,), 99, dtype=torch.int32, device=DEV), prob_sum=torch.full((e,), 9.0, device=DEV),
                   loss=torch.full((1,), 9.0, device=DEV))
    dg.moe_router(x, out["ids"], out["weights"], out.get("counts"), out.get("prob_sum"), out.get("loss"), workspace=workspace,
                  **kw)
    return out


def tolerance(x):
    r = float(np.abs(x[np.isfinite(x)]).max()) if np.isfinite(x).any() else 0.0
    return (2 * r + 40) * STEP


def check_forward(out, x, k, **kw):
    ref = oracle.ref_router(x, k, **{n: v for n, v in kw.items() if n != "workspace"})
    np.testing.assert_array_equal(out["ids"].cpu().numpy(), ref["ids"])
    tol = 3 * tolerance(x)
    np.testing.assert_allclose(as_f64(out["weights"]), ref["weights"], rtol=tol, atol=1e-37)
    if "counts" in out:
        np.testing.assert_array_equal(out["counts"].cpu().numpy(), ref["counts"])
        # FP32 sums over a workgroup's rows, then FP64: one rounding a row at worst
        np.testing.assert_allclose(as_f64(out["prob_sum"]), ref["prob_sum"], rtol=tol + len(x) * STEP, atol=1e-37)
        np.testing.assert_allclose(as_f64(out["loss"])[0], ref["loss"], rtol=2 * (tol + len(x) * STEP), atol=1e-37)


def logits(m, e, dtype, seed=0, dead=0):
    g = torch.Generator().manual_seed(seed)
    x = torch.randn(m, e, generator=g) * 2
    if dead:
        x[:, torch.randperm(e, generator=g)[:dead]] = -float("inf")
    return x.to(DT[dtype]).to(DEV)


SIZES = [(1, 1, 1), (1, 64, 6), (7, 64, 6), (3, 5, 5), (33, 60, 4), (64, 16, 2), (65, 63, 8), (130, 65, 3), (300, 128, 8),
         (257, 255, 8), (500, 256, 8), (70, 257, 5), (40, 320, 10), (33, 511, 12), (21, 1000, 16), (9, 1024, 64)]


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("m,e,k", SIZES)
def test_router(m, e, k, score, dtype):
    x = logits(m, e, dtype, seed=m + e)
    for normalize, bias, mask in ((True, False, False), (False, True, True), (True, True, False), (True, False, True)):
        rng = np.random.default_rng(m)
        kw = dict(score=score, normalize=normalize, scale=1.0 if normalize else 2.5)
        b = (0.1 * rng.standard_normal(e)).astype(np.float32) if bias else None
        v = rng.random(m) < 0.7 if mask else None
        for stats in (True, False):
            out = forward(x, k, stats, bias=None if b is None else torch.from_numpy(b).to(DEV),
                          mask=None if v is None else torch.from_numpy(v).to(DEV), **kw)
            check_forward(out, as_f64(x), k, bias=b, mask=v, **kw)


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("bias", [False, True])
def test_router_ties_and_near_ties(score, bias):
    """Few distinct values, values one step apart, and biases that nearly undo them: the order of FP64 keys."""
    rng = np.random.default_rng(5)
    e = 160
    x = rng.choice([0.0, 0.5, 1.0], (200, e)).astype(np.float32)
    x[50:100] = np.float32(1.0) + rng.integers(0, 3, (50, e)) * np.float32(2.0 ** -23)
    x[100:150] = rng.integers(-3, 3, (50, 1)).astype(np.float32)
    b = None
    if bias:
        b = np.zeros(e, dtype=np.float32)
        b[::3] = 2.0 ** -24
        b[1::3] = -(2.0 ** -25)
    for dtype in ("fp32", "bf16"):
        t = torch.from_numpy(x).to(DT[dtype]).to(DEV)
        check_forward(forward(t, 8, score=score, bias=None if b is None else torch.from_numpy(b).to(DEV)), as_f64(t), 8,
                      score=score, bias=b)


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
def test_router_random_bias_orders_like_fp64(score):
    """Many rows whose keys cross closely: scores minus their own FP32 value as the bias leaves rounding errors."""
    rng = np.random.default_rng(6)
    e = 96
    row = rng.standard_normal(e).astype(np.float32)
    p = oracle.ref_router(row[None], 1, score)  # noqa: F841
    s = 1 / (1 + np.exp(-row.astype(np.float64))) if score == "sigmoid" else np.exp(row.astype(np.float64)) / np.exp(
        row.astype(np.float64)).sum()
    b = (0.25 - s).astype(np.float32)
    x = np.tile(row, (64, 1))
    t = torch.from_numpy(x).to(DEV)
    check_forward(forward(t, 12, score=score, bias=torch.from_numpy(b).to(DEV)), as_f64(t), 12, score=score, bias=b)


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("e,k,lanes", [(256, 8, 16), (256, 12, 16), (128, 8, 16), (256, 20, 32), (512, 10, 32), (1000, 16, 64)])
def test_router_chosen_experts_of_one_lane(e, k, lanes, score, dtype):
    """The chosen experts lie where one lane holds them all (4 in a row, every 4 * lanes), more than it keeps at hand; in
    every fourth row spread over two lanes, and in others ties among them."""
    rng = np.random.default_rng(9)
    x = rng.standard_normal((120, e))
    for t in range(len(x)):
        lane = int(rng.integers(0, lanes - 1))
        for one in ([lane] if t % 4 else [lane, lane + 1]):
            at = [i for i in range(e) if (i // 4) % lanes == one]
            x[t, at] = 5 + (rng.integers(0, 3, len(at)) if t % 3 == 0 else rng.random(len(at)))
    t = torch.from_numpy(x.astype(np.float32)).to(DT[dtype]).to(DEV)
    for bias in (None, (0.01 * rng.standard_normal(e)).astype(np.float32)):
        check_forward(forward(t, k, score=score, bias=None if bias is None else torch.from_numpy(bias).to(DEV)), as_f64(t), k,
                      score=score, bias=bias)


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
def test_router_dead_experts_and_empty_rows(score, dtype):
    x = logits(50, 40, dtype, dead=30)
    x[7] = -float("inf")
    x[9, :] = -float("inf")
    x[9, 33] = 1.0
    for bias in (None, torch.randn(40, device=DEV)):
        b = None if bias is None else bias.cpu().numpy()
        check_forward(forward(x, 16, score=score, bias=bias), as_f64(x), 16, score=score, bias=b)
    out = forward(x, 16, score=score, mask=torch.zeros(50, dtype=torch.bool, device=DEV))
    assert (out["ids"] == -1).all() and not out["weights"].any() and not out["counts"].any()
    assert not out["prob_sum"].any() and not out["loss"].any()


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("scale", [60.0, 3e4])
def test_router_wide_logits(score, scale):
    """Scores down to zero and up to one.  Few levels, so that equal FP64 scores have equal logits' order too."""
    rng = np.random.default_rng(8)
    x = (rng.permuted(np.tile(np.linspace(-scale, 30.0, 90), (40, 1)), axis=1)).astype(np.float32)
    t = torch.from_numpy(x).to(DEV)
    out = forward(t, 6, score=score, normalize=False)
    ref = oracle.ref_router(as_f64(t), 6, score, normalize=False)
    np.testing.assert_array_equal(out["ids"].cpu().numpy(), ref["ids"])
    np.testing.assert_allclose(as_f64(out["weights"]), ref["weights"], rtol=3 * tolerance(np.minimum(np.abs(x), 100)), atol=2e-38)
    np.testing.assert_array_equal(out["counts"].cpu().numpy(), ref["counts"])


def test_router_ids_stay_in_range_whatever_the_logits():
    x = torch.randn(64, 50, device=DEV)
    x[::3, ::7] = float("nan")
    x[1::3, 4] = float("inf")
    x[2::9] = float("nan")
    for score, bias in itertools.product(["softmax", "sigmoid"], [None, torch.full((50,), float("nan"), device=DEV)]):
        out = forward(x, 5, score=score, bias=bias)
        assert int(out["ids"].min()) >= -1 and int(out["ids"].max()) < 50
        assert int(out["counts"].sum()) == int((out["ids"] >= 0).sum())


def test_router_strided_logits_and_large_batch():
    m, e, k = 20011, 100, 6
    wide = torch.randn(m, 137, device=DEV)
    x = wide[:, 21:121]
    check_forward(forward(x, k, score="sigmoid"), as_f64(x), k, score="sigmoid")
    out, again = forward(x, k), forward(x, k)
    for n in out:
        assert torch.equal(out[n], again[n])  # the same bits every time


def test_router_of_no_rows_writes_zeros():
    x = torch.empty(0, 32, device=DEV)
    out = forward(x, 4)
    assert not out["counts"].any() and not out["prob_sum"].any() and not out["loss"].any()
    dg.moe_router_backward(x, out["ids"], torch.empty(0, 4, device=DEV), torch.empty(0, 32, device=DEV))


def test_router_counts_without_loss():
    x = logits(77, 48, "fp32")
    ids, w = torch.empty(77, 4, dtype=torch.int32, device=DEV), torch.empty(77, 4, device=DEV)
    counts = torch.empty(48, dtype=torch.int32, device=DEV)
    dg.moe_router(x, ids, w, counts)
    assert torch.equal(counts, torch.bincount(ids.flatten().long(), minlength=48).int())


def test_router_in_graphs_that_share_a_workspace():
    m, e, k = 700, 96, 4
    ws = dg.alloc_moe_router_workspace(m, e)
    xs = [logits(m, e, "fp32", seed=s) for s in range(3)]
    want = [forward(x, k, workspace=ws) for x in xs]
    inputs = [x.clone() for x in xs[:2]]
    outs, graphs = [], []
    for x in inputs:
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            outs.append(forward(x, k, workspace=ws))
        graphs.append(g)
    for i, j in ((0, 1), (1, 2), (0, 0), (1, 1)):
        inputs[i].copy_(xs[j])
        graphs[i].replay()
        torch.cuda.synchronize()
        for n in want[j]:
            assert torch.equal(outs[i][n], want[j][n]), n
        again = forward(xs[2], k, workspace=ws)
        assert torch.equal(again["loss"], want[2]["loss"])


def backward(x, ids, dw, stats=None, out=None, **kw):
    dx = torch.full_like(x, 9.0) if out is None else out
    dg.moe_router_backward(x, ids, dw, dx, *(stats or (None, None, None)), **kw)
    return dx


def check_backward(dx, x, ids, dw, stats, dtype, **kw):
    c, s, dl = (None, None, 0.0) if stats is None else (stats[0].cpu().numpy(), as_f64(stats[1]), float(stats[2]))
    ref, mag = oracle.ref_router_backward(as_f64(x), ids.cpu().numpy(), as_f64(dw), c, s, dl, **kw)
    # four factors of a score and three sums of at most 1 + 22 + top_k roundings
    tol = (4 * tolerance(as_f64(x)) + 3 * (30 + ids.shape[1]) * STEP) * mag + 1e-37
    if dtype == "bf16":
        tol = tol + 2.0 ** -8 * (np.abs(ref) + tol) + 2.0 ** -133
    assert (np.abs(as_f64(dx) - ref) <= tol).all(), np.max((np.abs(as_f64(dx) - ref)) / tol)


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("score,normalize", itertools.product(["softmax", "sigmoid"], [True, False]))
@pytest.mark.parametrize("m,e,k", SIZES)
def test_router_gradient(m, e, k, score, normalize, dtype):
    x = logits(m, e, dtype, seed=m + e, dead=e // 5 if e > 2 * k else 0)
    mask = torch.rand(m, generator=torch.Generator().manual_seed(m)).to(DEV) < 0.8
    kw = dict(score=score, normalize=normalize, scale=1.5)
    f = forward(x, k, mask=mask, **kw)
    dw = torch.randn(m, k, generator=torch.Generator().manual_seed(1)).to(DEV)
    stats = (f["counts"], f["prob_sum"], torch.tensor([3.0 * m], device=DEV))
    check_backward(backward(x, f["ids"], dw, stats, **kw), x, f["ids"], dw, stats, dtype, **kw)
    check_backward(backward(x, f["ids"], dw, None, **kw), x, f["ids"], dw, None, dtype, **kw)


def test_router_gradient_against_differences_of_the_forward():
    """Central differences of the library's own forward in FP32: steps of 2^-5, whose second-order error and the FP32
    noise of the values (2^-20 of the loss's magnitude over the step) bound the difference."""
    m, e, k = 6, 12, 3
    for score, normalize in itertools.product(["softmax", "sigmoid"], [True, False]):
        kw = dict(score=score, normalize=normalize)
        x = logits(m, e, "fp32", seed=3)
        top = x.sort(dim=1, descending=True)[0]
        x = torch.where(x >= top[:, k - 1:k], x + 0.5, x)  # the choice does not change within a step
        f = forward(x, k, **kw)
        dw = torch.randn(m, k, generator=torch.Generator().manual_seed(2)).to(DEV)
        dx = as_f64(backward(x, f["ids"], dw, (f["counts"], f["prob_sum"], torch.tensor([2.0], device=DEV)), **kw))

        def value(z):
            r = forward(z, k, **kw)
            order = r["ids"].argsort(1), f["ids"].argsort(1)
            assert torch.equal(r["ids"].sort(1)[0], f["ids"].sort(1)[0])
            return float((r["weights"].gather(1, order[0]).double() * dw.gather(1, order[1]).double()).sum() + 2.0 * r["loss"].double())

        h = 2.0 ** -5
        for t, j in itertools.product(range(m), range(0, e, 3)):
            up, down = x.clone(), x.clone()
            up[t, j] += h
            down[t, j] -= h
            slope = (value(up) - value(down)) / (2 * h)
            # third derivatives of these scores times a weight of up to ~4 are below 8: h^2 / 6 * 8
            assert abs(slope - dx[t, j]) <= h * h * 8 / 6 + 2.0 ** -20 * 20 / h, (score, normalize, t, j)


def test_router_gradient_in_place_strided_and_with_bad_ids():
    m, e, k = 45, 70, 4
    wide = torch.randn(m, 100, device=DEV)
    x = wide[:, 10:80]
    ids = forward(x.contiguous(), k)["ids"]
    ids[3] = -1
    ids[4, 2], ids[5, 0], ids[6] = 70, -9, 2 ** 31 - 1
    dw = torch.randn(m, k, device=DEV)
    want = backward(x.contiguous(), ids, dw)
    check_backward(want, x, ids, dw, None, "fp32")
    assert not want[3].any() and not want[6].any()
    before = wide.clone()
    backward(x, ids, dw, out=x)
    assert torch.equal(x, want)
    assert torch.equal(wide[:, :10], before[:, :10]) and torch.equal(wide[:, 80:], before[:, 80:])


def test_router_gradient_captured_and_replayed():
    m, e, k = 300, 64, 4
    x = logits(m, e, "bf16")
    f = forward(x, k)
    dw, dl = torch.randn(m, k, device=DEV), torch.tensor([5.0], device=DEV)
    stats = (f["counts"], f["prob_sum"], dl)
    want = backward(x, f["ids"], dw, stats)
    dw2 = torch.randn(m, k, device=DEV)
    want2 = backward(x, f["ids"], dw2, stats)
    buf = dw.clone()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        out = backward(x, f["ids"], buf, stats)
    for src, res in ((dw, want), (dw2, want2), (dw, want)):
        buf.copy_(src)
        g.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, res)
        assert torch.equal(backward(x, f["ids"], dw2, stats), want2)


def test_router_gradient_of_the_whole_batch_from_its_parts():
    """Counts and sums added over two halves: each half's gradient is its part of the whole batch's."""
    m, e, k = 90, 24, 3
    x = logits(m, e, "fp32")
    f = forward(x, k)
    dw, dl = torch.randn(m, k, device=DEV), torch.tensor([40.0], device=DEV)
    whole = backward(x, f["ids"], dw, (f["counts"], f["prob_sum"], dl))
    parts = [forward(x[s], k) for s in (slice(0, 37), slice(37, 90))]
    total = (parts[0]["counts"] + parts[1]["counts"], parts[0]["prob_sum"] + parts[1]["prob_sum"], dl)
    assert torch.equal(total[0], f["counts"])
    for s in (slice(0, 37), slice(37, 90)):
        # the two prob_sum differ by roundings, 2^-20 of g
        torch.testing.assert_close(backward(x[s], f["ids"][s].contiguous(), dw[s].contiguous(), total), whole[s], rtol=1e-5, atol=1e-6)
