"""GPU tests of the 4-bit cast and products at the ends of their ranges."""

import pytest
import torch

pytestmark = pytest.mark.gpu

if torch.cuda.is_available():  # pragma: no cover - GPU only
    import moe_grouped_gemm_tiles_amd as dg
    from tests._gpu_harness import DEV, out_buffer


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
