"""CPU tests of the refusals of the 4-bit and router entry points: bad arguments are reported before anything touches a
GPU."""

import os

import pytest
import torch

import moe_grouped_gemm_tiles_amd as dg

INVALID, UNSUPPORTED, WORKSPACE = 1, 2, 4
P = 0x10000  # aligned, never dereferenced: validation fails first


@pytest.fixture(scope="module")
def lib():
    if not os.path.exists(dg.library_path()):
        from moe_grouped_gemm_tiles_amd import build
        build.build()
    return dg.load_library()


def _cast(lib, **kw):
    a = dict(x=P, ldx=512, dt=0, q=P, ldq=256, sf=P, ld_sf=64, y=None, ldy=0, masked=None, g=1, m=64, k=512)
    a.update(kw)
    return lib.dg_cast_to_mxfp4(*a.values(), None)


def test_cast_refusals(lib):
    for bad in (dict(k=500), dict(k=64), dict(g=65536), dict(k=1 << 30, ldx=1 << 30, ldq=1 << 30)):
        assert _cast(lib, **bad) == UNSUPPORTED, bad
    for bad in (dict(m=-1), dict(k=-128), dict(g=-1), dict(dt=2), dict(x=None), dict(x=P + 8), dict(ldx=504), dict(ldx=516),
                dict(q=None), dict(q=P + 2), dict(ldq=252), dict(ldq=258), dict(sf=None), dict(sf=P + 2), dict(ld_sf=63),
                dict(y=P, ldy=500), dict(y=P + 8, ldy=512), dict(y=P, ldy=513), dict(masked=P + 2)):
        assert _cast(lib, **bad) == INVALID, bad
    assert _cast(lib, m=0) == 0 and _cast(lib, k=0) == 0 and _cast(lib, g=0) == 0


def _dense(lib, **kw):
    a = dict(a=P, lda=256, sfa=P, ld_sfa=64, b=P, ldb=256, sfb=P, ld_sfb=64, c=None, ldc=0, d=P, ldd=64, dt=0, m=64, n=64,
             k=512, ws=P, wsb=1 << 30)
    a.update(kw)
    return lib.dg_mxfp4_gemm_nt(*a.values(), None)


BAD = (dict(a=None), dict(a=P + 8), dict(sfa=None), dict(sfa=P + 4), dict(b=None), dict(b=P + 1), dict(sfb=None),
       dict(sfb=P + 8), dict(d=None), dict(d=P + 8), dict(dt=2), dict(ld_sfa=60), dict(ld_sfa=66), dict(ld_sfb=60),
       dict(ld_sfb=65))


def test_dense_refusals(lib):
    for bad in BAD + (dict(m=-1), dict(n=-1), dict(k=-128), dict(lda=240), dict(lda=264), dict(ldb=240), dict(ldb=257),
                      dict(ldd=56), dict(ldd=68), dict(c=P + 4, ldc=64), dict(c=P, ldc=60), dict(c=P, ldc=68)):
        assert _dense(lib, **bad) == INVALID, bad
    for bad in (dict(k=500), dict(lda=1 << 23), dict(ldb=1 << 24)):
        assert _dense(lib, **bad) == UNSUPPORTED, bad
    assert _dense(lib, m=0) == 0 and _dense(lib, n=0) == 0
    for m, n, k in ((0, 256, 512), (64, 0, 512), (64, 256, 0), (64, 256, 500), (-1, 256, 512)):
        assert lib.dg_get_mxfp4_workspace_size(m, n, k) == 0


def _contiguous(lib, **kw):
    a = dict(a=P, sfa=P, ld_sfa=128, b=P, sfb=P, ld_sfb=64, d=P, dt=0, idx=P, m=128, n=64, k=512, g=4)
    a.update(kw)
    return lib.dg_m_grouped_mxfp4_gemm_nt_contiguous(*a.values(), None)


def _masked(lib, **kw):
    a = dict(a=P, sfa=P, ld_sfa=64, b=P, sfb=P, ld_sfb=64, d=P, dt=0, mm=P, g=4, m=64, n=64, k=512, em=8)
    a.update(kw)
    return lib.dg_m_grouped_mxfp4_gemm_nt_masked(*a.values(), None)


def test_grouped_refusals(lib):
    for bad in BAD + (dict(g=-1), dict(m=-128), dict(n=-1), dict(n=60, ld_sfb=64), dict(k=-128)):
        bad = {k: (124 if k == "ld_sfa" and v == 60 else 130 if k == "ld_sfa" else v) for k, v in bad.items()}
        assert _contiguous(lib, **bad) == INVALID, bad
    for bad in BAD + (dict(g=-1), dict(m=-1), dict(n=-1), dict(n=60), dict(k=-128), dict(mm=None), dict(mm=P + 1)):
        assert _masked(lib, **bad) == INVALID, bad
    assert _contiguous(lib, idx=None) == INVALID and _contiguous(lib, idx=P + 2) == INVALID
    assert _contiguous(lib, m=130, ld_sfa=132) == UNSUPPORTED
    for f in (_contiguous, _masked):
        assert f(lib, k=500) == UNSUPPORTED and f(lib, k=1 << 24) == UNSUPPORTED
        assert f(lib, m=0) == 0 and f(lib, n=0) == 0 and f(lib, g=0) == 0


def _route(lib, **kw):
    a = dict(x=P, ld=64, dt=0, bias=None, mask=None, score=0, norm=1, scale=1.0, ids=P, w=P, counts=P, ps=P, loss=P, m=64, e=64,
             k=4, ws=P, wsb=1 << 30)
    a.update(kw)
    return lib.dg_moe_router(*a.values(), None)


def test_router_refusals(lib):
    for bad in (dict(e=0), dict(e=1025, ld=2000), dict(k=0), dict(k=65, e=128, ld=128), dict(k=9, e=8)):
        assert _route(lib, **bad) == UNSUPPORTED, bad
    for bad in (dict(m=-1), dict(e=-1), dict(k=-1), dict(dt=2), dict(score=2), dict(score=-1), dict(x=None), dict(x=P + 1),
                dict(dt=1, x=P + 2), dict(ld=63), dict(bias=P + 2), dict(ids=None), dict(ids=P + 2), dict(w=None), dict(w=P + 1),
                dict(counts=None), dict(counts=P + 1), dict(ps=None), dict(loss=None), dict(ps=P + 2), dict(loss=P + 2),
                dict(scale=-1.0), dict(scale=float("nan"))):
        assert _route(lib, **bad) == INVALID, bad
    need = lib.dg_get_moe_router_workspace_size(64, 64)
    assert need > 0
    for bad in (dict(ws=None), dict(ws=P + 128), dict(wsb=need - 1)):
        assert _route(lib, **bad) == WORKSPACE, bad
    assert _route(lib, m=0, counts=None, ps=None, loss=None, ws=None) == 0
    for m, e in ((0, 64), (-1, 64), (64, 0), (64, 1025)):
        assert lib.dg_get_moe_router_workspace_size(m, e) == 0


def _grad(lib, **kw):
    a = dict(x=P, ld=64, dt=0, score=0, norm=1, scale=1.0, ids=P, dw=P, counts=P, ps=P, dl=P, dx=P, ld_dx=64, m=64, e=64, k=4)
    a.update(kw)
    return lib.dg_moe_router_backward(*a.values(), None)


def test_router_gradient_refusals(lib):
    for bad in (dict(e=0), dict(e=1025, ld=2000, ld_dx=2000), dict(k=0), dict(k=65, e=128, ld=128, ld_dx=128), dict(k=9, e=8)):
        assert _grad(lib, **bad) == UNSUPPORTED, bad
    for bad in (dict(m=-1), dict(dt=3), dict(score=5), dict(x=None), dict(x=P + 1), dict(dx=None), dict(dx=P + 1), dict(ids=None),
                dict(ids=P + 1), dict(dw=None), dict(dw=P + 2), dict(ld=60), dict(ld_dx=63), dict(counts=None), dict(ps=None),
                dict(dl=None), dict(counts=P + 2), dict(ps=P + 2), dict(dl=P + 2), dict(scale=-0.5)):
        assert _grad(lib, **bad) == INVALID, bad
    assert _grad(lib, m=0) == 0


def test_bindings_refuse_cpu_tensors_and_wrong_types(lib):
    x = torch.zeros(4, 256)
    q, sf = torch.zeros(4, 128, dtype=torch.uint8), torch.zeros(2, 4, dtype=torch.int32)
    bad = (TypeError, ValueError)
    with pytest.raises(bad):
        dg.cast_to_mxfp4(x, q, sf)
    with pytest.raises(bad):
        dg.mxfp4_gemm_nt((q, sf), (q, sf), torch.zeros(4, 4))
    with pytest.raises(bad):
        dg.m_grouped_mxfp4_gemm_nt_contiguous((q, sf), (q[None], sf[None]), torch.zeros(4, 4), torch.zeros(4, dtype=torch.int32))
    with pytest.raises(bad):
        dg.m_grouped_mxfp4_gemm_nt_masked((q[None], sf[None]), (q[None], sf[None]), torch.zeros(1, 4, 4),
                                          torch.zeros(1, dtype=torch.int32))
    ids, w = torch.zeros(4, 2, dtype=torch.int32), torch.zeros(4, 2)
    with pytest.raises(bad):
        dg.moe_router(x, ids, w)
    with pytest.raises(bad):
        dg.moe_router_backward(x, ids, w, x)
