"""CPU tests of the 4-bit and router entry points at the ends of their documented ranges: what is refused before anything
touches a GPU."""

import os

import pytest

import moe_grouped_gemm_tiles_amd as dg
from tests.test_abi_mxfp4_router import INVALID, P, UNSUPPORTED, _cast, _contiguous, _dense, _grad, _masked


@pytest.fixture(scope="module")
def lib():
    if not os.path.exists(dg.library_path()):
        from moe_grouped_gemm_tiles_amd import build
        build.build()
    return dg.load_library()


@pytest.mark.parametrize("k", [0, 512])
def test_dense_strides_are_checked_for_every_k(lib, k):
    """The empty product (k == 0) starts the same kernel, which builds its descriptors from lda and ldb."""
    none = dict(k=k, lda=256, ldb=256) if k else dict(k=0, lda=0, ldb=0, a=None, b=None, sfa=None, sfb=None)
    for bad in (dict(lda=-16), dict(ldb=-16), dict(lda=-(1 << 40)), dict(lda=264), dict(ldb=8 + 256)):
        assert _dense(lib, **{**none, **bad}) == INVALID, bad
    for bad in (dict(lda=1 << 23), dict(ldb=1 << 23), dict(lda=(1 << 24) - 16), dict(lda=1 << 56), dict(ldb=1 << 62)):
        assert _dense(lib, **{**none, **bad}) == UNSUPPORTED, bad


@pytest.mark.parametrize("k", [0, 512])
def test_rows_and_columns_past_their_limit(lib, k):
    most = 1 << 29
    for big in (most, 2 ** 31 - 128):
        assert _dense(lib, m=big, k=k, ld_sfa=big) == UNSUPPORTED
        assert _dense(lib, n=big, k=k, ldd=big, ld_sfb=big) == UNSUPPORTED
        assert _contiguous(lib, m=big, k=k, ld_sfa=big) == UNSUPPORTED
        assert _masked(lib, m=big, k=k, ld_sfa=big) == UNSUPPORTED
        assert lib.dg_get_mxfp4_workspace_size(big, 128, 512) == lib.dg_get_mxfp4_workspace_size(128, big, 512) == 0


def test_scale_arrays_past_their_limit(lib):
    """512 columns are four words a row: 2^31 bytes are 2^27 words between them."""
    for ld in (1 << 27, 1 << 40, 1 << 61, (1 << 62) - 4):
        assert _dense(lib, ld_sfa=ld) == UNSUPPORTED and _dense(lib, ld_sfb=ld) == UNSUPPORTED
        assert _contiguous(lib, ld_sfa=ld) == UNSUPPORTED and _masked(lib, ld_sfb=ld) == UNSUPPORTED


def test_outputs_in_place_need_the_inputs_row_stride(lib):
    assert _cast(lib, y=P, ldx=512, ldy=520) == INVALID
    assert _cast(lib, y=P, ldx=512, ldy=520, m=1, g=2) == INVALID
    assert _grad(lib, x=P, dx=P, ld=64, ld_dx=72) == INVALID


def test_cast_past_its_limits(lib):
    """The limits are on K, on the values of a group and on groups alone."""
    for bad in (dict(k=(1 << 25) + 128, m=1), dict(k=128, m=1 << 29), dict(k=1 << 25, m=1 << 11), dict(k=512, m=1 << 27)):
        k = bad["k"]
        assert _cast(lib, ldx=k, ldq=k // 2, ld_sf=bad["m"], **bad) == UNSUPPORTED, bad


def test_more_tiles_than_an_int_counts_with_the_grid(lib):
    """Without K a masked call's groups are its output alone: one tile each here."""
    for g in ((1 << 30) + 1, 2 ** 31 - 1):
        assert _masked(lib, g=g, m=1, n=8, k=0, ld_sfa=4, ld_sfb=8) == UNSUPPORTED
