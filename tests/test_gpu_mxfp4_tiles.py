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
