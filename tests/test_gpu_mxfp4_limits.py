"""GPU tests of the 4-bit cast and products at the ends of their ranges."""

import numpy as np
import pytest
import torch

import oracle

pytestmark = pytest.mark.gpu

if torch.cuda.is_available():  # pragma: no cover - GPU only
    import moe_grouped_gemm_tiles_amd as dg
    from tests._gpu_harness import DEV, as_f64, out_buffer
    from tests.test_gpu_mxfp4 import scale_bytes


@pytest.mark.parametrize("m,n", [(3, 16), (300, 520)])
@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
def test_empty_product_reads_no_operand_whatever_its_strides(m, n, dtype):
    lib = dg.load_library()
    c = torch.randn(m, n, device=DEV).to(torch.bfloat16 if dtype == "bf16" else torch.float32)
    for with_c in (True, False):
        d = out_buffer((m,), n, dtype)
        for ld in (0, 256, (1 << 23) - 16):
            d.fill_(7.0)
            assert lib.dg_mxfp4_gemm_nt(None, ld, None, 0, None, ld, None, 0, c.data_ptr() if with_c else None, n, d.data_ptr(), n,
                                        int(dtype == "fp32"), m, n, 0, None, 0, dg._stream(d)) == 0
            assert torch.equal(d, c if with_c else torch.zeros_like(c))


@pytest.mark.parametrize("m,k,groups", [((1 << 27) + 16 + 5, 128, 0), ((1 << 27) + 37, 128, 1), (130, 1 << 25, 0), (21, 1 << 25, 2)])
def test_cast_of_more_blocks_than_a_grid_holds(m, k, groups):
    """Rows of both launches (K = 128: 16 rows to a workgroup of a grid of 2^23) and the largest K, whose rows' last
    columns are looked at; what is not, is zero and stays so."""
    x = torch.zeros(*([groups] if groups else []), m, k, dtype=torch.bfloat16, device=DEV)
    q = torch.full((*x.shape[:-1], k // 2), 0xA5, dtype=torch.uint8, device=DEV)
    sf = torch.full((*x.shape[:-2], k // 128, m), 7, dtype=torch.int32, device=DEV)
    cols = slice(k - 128, k)
    spots = [slice(0, 20), slice(max(0, m - 60), m)] + ([slice((1 << 27) - 20, (1 << 27) + 20)] if m > 1 << 27 else [])
    xs, qs, ss = (x, q, sf) if not groups else (x[-1], q[-1], sf[-1])
    for s in spots:
        xs[s, cols] = torch.randn(s.stop - s.start, 128, device=DEV).bfloat16()
    dg.cast_to_mxfp4(x, q, sf)
    for s in spots:
        want, byte, _ = oracle.ref_cast_mxfp4(as_f64(xs[s, cols]))
        np.testing.assert_array_equal(qs[s, k // 2 - 64:].cpu().numpy(), want)
        np.testing.assert_array_equal(scale_bytes(ss[-1:, s]), byte)
    for s in spots:
        qs[s, k // 2 - 64:] = 0
        ss[-1, s] = 0x7F7F7F7F
    assert not q.any() and bool((sf == 0x7F7F7F7F).all())
