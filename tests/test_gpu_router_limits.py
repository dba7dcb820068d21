"""GPU tests of the router and its gradient at the ends of their ranges."""

import pytest
import torch

pytestmark = pytest.mark.gpu

if torch.cuda.is_available():  # pragma: no cover - GPU only
    import moe_grouped_gemm_tiles_amd as dg
    from tests._gpu_harness import DEV, as_f64
    from tests.test_gpu_router import DT, backward, check_backward, check_forward, forward


@pytest.mark.parametrize("m", [(1 << 28) + 77, (1 << 31) - 5])
@pytest.mark.parametrize("stats", [True, False])
def test_router_of_as_many_rows_as_an_int_counts(m, stats):
    """One expert: more rows than a grid of one round takes, and row numbers that pass 2^31 with the grid's rows added.  A
    softmax over one expert is 1, so sums are whole numbers; a masked row is known by its id."""
    x = torch.empty(m, 1, dtype=torch.bfloat16, device=DEV).fill_(0.25)
    mask = torch.ones(m, dtype=torch.bool, device=DEV)
    mask[::1000], mask[-1] = False, False
    off = int((~mask[::1000]).sum()) + ((m - 1) % 1000 != 0)
    ids = torch.full((m, 1), 99, dtype=torch.int32, device=DEV)
    w = torch.full((m, 1), 9.0, device=DEV)
    out = [None] * 3
    if stats:
        out = [torch.full((1,), 99, dtype=torch.int32, device=DEV), torch.full((1,), 9.0, device=DEV),
               torch.full((1,), 9.0, device=DEV)]
    dg.moe_router(x, ids, w, *out, mask=mask)
    for at in range(0, m, 1 << 27):
        on = mask[at:at + (1 << 27)]
        assert torch.equal(ids[at:at + (1 << 27), 0] == 0, on) and torch.equal(ids[at:at + (1 << 27), 0] == -1, ~on)
        assert torch.equal(w[at:at + (1 << 27), 0], on.float())
    if stats:
        # each lane and workgroup adds at most 2^24 ones, exactly; the second kernel adds in FP64
        assert int(out[0]) == m - off and float(out[1]) == float(torch.tensor(float(m - off))) and float(out[2]) == 1.0
        return
    # sigmoid, weights as they are: dx = dw * p * (1 - p); zero where there is no expert
    dw = w.fill_(0.5)
    dx = torch.full_like(x, 9.0)
    dg.moe_router_backward(x, ids, dw, dx, score="sigmoid", normalize=False)
    p = torch.sigmoid(torch.tensor(0.25, dtype=torch.float64))
    want = (0.5 * p * (1 - p)).item()  # 2^-8: BF16's rounding, and a little for the FP32 before it
    for at in range(0, m, 1 << 27):
        on, got = mask[at:at + (1 << 27)], dx[at:at + (1 << 27), 0]
        assert not got[~on].any()
        assert bool(((got[on].float() - want).abs() <= (2.0 ** -8 + 2.0 ** -18) * want).all())


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("at,wide", [(1, 71), (1, 72), (2, 76), (3, 137)])
@pytest.mark.parametrize("e", [60, 64])
def test_rows_that_are_aligned_to_their_type_alone(e, at, wide, dtype):
    m, k = 90, 5
    x = torch.randn(m, wide, generator=torch.Generator().manual_seed(at)).to(DT[dtype]).to(DEV)[:, at:at + e]
    for score in ("softmax", "sigmoid"):
        f = forward(x, k, score=score)
        check_forward(f, as_f64(x), k, score=score)
        dw = torch.randn(m, k, generator=torch.Generator().manual_seed(2)).to(DEV)
        stats = (f["counts"], f["prob_sum"], torch.tensor([50.0], device=DEV))
        whole = torch.full((m, wide), 9.0, dtype=DT[dtype], device=DEV)
        check_backward(backward(x, f["ids"], dw, stats, out=whole[:, at:at + e], score=score), x, f["ids"], dw, stats, dtype, score=score)
        assert bool((whole[:, :at] == 9).all()) and bool((whole[:, at + e:] == 9).all())
