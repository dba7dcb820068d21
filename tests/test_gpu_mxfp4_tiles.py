"""The 4-bit products' planner, and their streaming tiles on rings that go round, on the GPU against the FP64 oracle and the
build with a wait and a barrier after each phase of LDS traffic."""

import numpy as np
import pytest
import torch

import moe_grouped_gemm_tiles_amd as dg
import oracle

if torch.cuda.is_available():  # pragma: no cover - GPU only
    from tests._gpu_harness import DEV, as_f64, out_buffer, raw_bits, sentinel_of
    from tests.test_gpu_mxfp4 import check, ld4, operand, stacked
from tests.test_gpu_mxfp4_layer import both_builds, debug  # noqa: F401

# groups, n, k, m_max; the tile where the caller expects every group to be full, and where it says nothing
FULL = [((22, 4224, 7808, 141), (256, 192, False), (128, 128, True)), ((17, 1152, 384, 85), (128, 128, True), (64, 128, True)),
        ((34, 640, 1536, 60), (64, 128, True), (32, 128, True)), ((19, 2560, 768, 83), (256, 224, False), (64, 128, True))]


def test_a_hint_of_full_groups_is_taken_as_it_is():
    for (g, n, k, most), full, unsaid in FULL:
        for rows, want in ((most, full), (0, unsaid), (-1, unsaid)):
            p = dg._mxfp4_plan_for_tests("masked", rows, n, k, groups=g, most_rows=most)
            assert (p["bm"], p["bn"], p["streaming"]) == want, (g, n, k, most, rows, p)


@pytest.mark.gpu
@pytest.mark.parametrize("case", range(1, len(FULL)))
def test_masked_with_a_hint_of_full_groups(case):
    """Full groups as expected, and fewer rows than expected."""
    (g, n, k, most), _, _ = FULL[case]
    rng = np.random.default_rng(case)
    a, b = [operand(rng, most, k) for _ in range(g)], [operand(rng, n, k) for _ in range(g)]
    ta, tb = stacked(a, ld4(most)), stacked(b, ld4(n))
    for counts in ([most] * g, [int(c) for c in rng.integers(0, most + 1, g)]):
        d = out_buffer((g, most), n, "bf16")
        dg.m_grouped_mxfp4_gemm_nt_masked(ta, tb, d, torch.tensor(counts, dtype=torch.int32, device=DEV), 2 * most)
        got, bits = as_f64(d), raw_bits(d)
        for i in range(0, g, 5):
            c = counts[i]
            assert (bits[i, c:] == sentinel_of(d)).all()
            if c:
                ref, mag = oracle.ref_mxfp4((a[i][0][:c], a[i][1][:c]), b[i])
                check(got[i, :c], ref, mag, k, "bf16")


# Rings that go round: a unit has more slabs than its tile has stages (7, 6 and 4 at 32, 64 and 128 rows), and a workgroup more
# than one unit, but for the first and last.  (m, n, k): rows of the tile, K splits.
ROUND_DENSE = [((5, 7168, 16384), 32, 3), ((16, 17152, 15232), 32, 3), ((60, 17152, 15232), 64, 3), ((100, 17152, 15232), 128, 3),
               ((20, 33000, 4224), 32, 1), ((40, 33000, 4224), 64, 1), ((100, 30000, 4224), 128, 1)]
# (groups, n, k, expected rows, most rows): rows of the tile
ROUND_MASKED = [((40, 2048, 4224, 10, 64), 32), ((40, 2048, 4224, 50, 64), 64), ((16, 4096, 4224, 64, 256), 128)]
STAGES = {32: 7, 64: 6, 128: 4}


def test_shapes_whose_rings_go_round():
    for (m, n, k), bm, splits in ROUND_DENSE:
        p = dg._mxfp4_plan_for_tests("dense", m, n, k)
        assert (p["bm"], p["bn"], p["streaming"], p["splits"]) == (bm, 128, True, splits), (m, n, k, p)
        units, slabs = -(-n // 128) * splits, -(-(k // 128 + 1) // 2 // splits)
        assert slabs >= 2 * STAGES[bm] and (units > 256) == (n not in (7168, 30000))
    for (g, n, k, rows, most), bm in ROUND_MASKED:
        p = dg._mxfp4_plan_for_tests("masked", rows, n, k, groups=g, most_rows=most)
        assert (p["bm"], p["bn"], p["streaming"], p["splits"]) == (bm, 128, True, 1), (g, n, k, rows, most, p)
        assert (k // 128 + 1) // 2 >= 2 * STAGES[bm] and (g - 2) * (n // 128) > 256


def near_unit(gen, rows, k):
    """Codes [.., K/2], scale words and FP64 values, on the GPU, with scales of 1/2, 1 and 2."""
    q = torch.randint(0, 256, (rows, k // 2), dtype=torch.uint8, device=DEV, generator=gen)
    byte = torch.randint(126, 129, (rows, k // 32), dtype=torch.uint8, device=DEV, generator=gen)
    table = torch.from_numpy(oracle.E2M1_TABLE).to(DEV)
    values = table[torch.stack((q & 15, q >> 4), -1).flatten(1).int()]
    values *= torch.exp2(byte.double() - 127).repeat_interleave(32, 1)
    words = torch.full((k // 128, ld4(rows)), 0x7F7F7F7F, dtype=torch.int32, device=DEV)
    words[:, :rows] = byte.view(torch.int32).t()
    return q, words, values


def exact_product(a, b):
    """A @ B.T in FP64.  Every term is a multiple of 1/16 and the magnitudes' sums stay below 2^20: any order of additions
    in FP32 gives it too, and BF16 its rounding."""
    assert float((a.abs() @ b.abs().t()).max()) < 2 ** 20
    return a @ b.t()


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("case", range(len(ROUND_DENSE)))
def test_dense_rings_that_go_round(debug, case, dtype):  # noqa: F811
    (m, n, k), _, splits = ROUND_DENSE[case]
    gen = torch.Generator(device=DEV).manual_seed(case)
    (qa, sa, a), (qb, sb, b) = near_unit(gen, m, k), near_unit(gen, n, k)
    ws = dg.alloc_mxfp4_workspace(m, n, k)
    d = both_builds(debug, lambda d: dg.mxfp4_gemm_nt((qa, sa), (qb, sb), d, workspace=ws), lambda: out_buffer((m,), n, dtype))
    assert torch.equal(d, exact_product(a, b).to(d.dtype))
    assert (ws is not None) == (splits > 1) and (ws is None or not ws[:65536].any())


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("case", range(len(ROUND_MASKED)))
def test_masked_rings_that_go_round(debug, case, dtype):  # noqa: F811
    (g, n, k, rows, most), _ = ROUND_MASKED[case]
    rng = np.random.default_rng(case)
    counts = [int(c) for c in rng.integers(1, min(2 * rows, most) + 1, g)]
    counts[1], counts[2], counts[3] = 0, most, -1
    gen = torch.Generator(device=DEV).manual_seed(case)
    qa, sa, a = zip(*[near_unit(gen, most, k) for _ in range(g)])
    qb, sb, b = zip(*[near_unit(gen, n, k) for _ in range(g)])
    ta, tb = (torch.stack(qa), torch.stack(sa)), (torch.stack(qb), torch.stack(sb))
    mm = torch.tensor(counts, dtype=torch.int32, device=DEV)
    d = both_builds(debug, lambda d: dg.m_grouped_mxfp4_gemm_nt_masked(ta, tb, d, mm, rows), lambda: out_buffer((g, most), n, dtype))
    bits = raw_bits(d)
    for i, c in enumerate(counts):
        c = max(c, 0)
        assert (bits[i, c:] == sentinel_of(d)).all()
        if c:
            assert torch.equal(d[i, :c], exact_product(a[i][:c], b[i]).to(d.dtype))
