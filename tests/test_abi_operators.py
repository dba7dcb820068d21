"""CPU tests of the refusals of the norm, expert-layer and clipping entry points:
bad arguments are reported before anything touches a GPU."""

import ctypes
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


def _norm(lib, **kw):
    a = dict(x=P, ldx=512, res=None, ldr=0, ro=None, ldro=0, dt=0, w=P, wdt=0, eps=1e-6, q=P, ldq=512, sf=P, ld_sf=64,
             ue=0, y=None, ldy=0, rstd=None, m=64, k=512)
    a.update(kw)
    return lib.dg_add_rms_norm_cast_to_fp8(*a.values(), None)


def test_norm_refusals(lib):
    for k in (500, 16512):
        assert _norm(lib, k=k, ldx=32768, ldq=32768) == UNSUPPORTED
    for bad in (dict(m=-1), dict(k=-128), dict(dt=2), dict(wdt=5), dict(eps=-1.0), dict(eps=float("nan")), dict(x=None),
                dict(x=P + 8), dict(ldx=504), dict(ldx=516), dict(w=None), dict(w=P + 4), dict(q=None), dict(q=P + 4),
                dict(ldq=504), dict(ldq=516), dict(sf=None), dict(sf=P + 4), dict(ld_sf=60), dict(ld_sf=66),
                dict(res=P, ldr=512), dict(ro=P, ldro=512), dict(res=P, ldr=512, ro=P, ldro=256),
                dict(res=P + 2, ldr=512, ro=P, ldro=512), dict(y=P, ldy=100), dict(y=P + 1, ldy=512), dict(rstd=P + 2)):
        assert _norm(lib, **bad) == INVALID, bad
    assert _norm(lib, m=0) == 0 and _norm(lib, k=0) == 0


def _grad(lib, **kw):
    a = dict(dy=P, lddy=512, s=P, lds=512, dt=0, w=P, wdt=0, rstd=P, dres=None, lddres=0, dx=P, lddx=512, dw=P, acc=0, m=64,
             k=512, ws=P, wsb=1 << 30)
    a.update(kw)
    return lib.dg_rms_norm_backward(*a.values(), None)


def test_norm_gradient_refusals(lib):
    assert _grad(lib, k=500) == UNSUPPORTED and _grad(lib, k=16512) == UNSUPPORTED
    for bad in (dict(m=-1), dict(dt=2), dict(wdt=3), dict(dy=None), dict(s=None), dict(dx=None), dict(dw=None),
                dict(w=None), dict(rstd=None), dict(rstd=P + 1), dict(dw=P + 4), dict(lddy=500), dict(lds=516),
                dict(lddx=100), dict(dres=P, lddres=100), dict(dres=P + 2, lddres=512)):
        assert _grad(lib, **bad) == INVALID, bad
    need = lib.dg_get_rms_norm_backward_workspace_size(64, 512)
    assert 512 * 4 <= need <= 64 * 512 * 4 and need % (512 * 4) == 0  # one row of partial sums per workgroup
    for bad in (dict(ws=None), dict(ws=P + 16), dict(wsb=need - 1)):
        assert _grad(lib, **bad) == WORKSPACE, bad
    assert _grad(lib, k=0) == 0
    for m, k in ((0, 512), (-1, 512), (8, 0), (8, 100), (8, 16512)):
        assert lib.dg_get_rms_norm_backward_workspace_size(m, k) == 0


def _moe(lib, fn=None, **kw):
    a = dict(x=P, ldx=512, sfx=P, ld_sfx=64, w13=P, sf13=P, w2=P, sf2=P, ids=P, tw=P, out=P, ld_out=512, m=64, top_k=4,
             e=8, h=512, i=256, ws=P, wsb=1 << 30)
    a.update(kw)
    return (fn or lib.dg_fp8_moe_few_tokens)(*a.values(), None)


def test_moe_refusals(lib):
    for fn in (lib.dg_fp8_moe_few_tokens, lib.dg_fp8_moe_few_tokens_ue8m0):
        for bad in (dict(h=500), dict(i=100), dict(i=0), dict(top_k=0), dict(top_k=65), dict(e=0), dict(e=1025)):
            assert _moe(lib, fn, **bad) == UNSUPPORTED, bad
        for bad in (dict(m=-1), dict(top_k=-1), dict(e=-1), dict(h=-128), dict(i=-128), dict(x=None), dict(x=P + 8),
                    dict(sfx=None), dict(sfx=P + 4), dict(w13=None), dict(w13=P + 1), dict(sf13=None), dict(w2=None),
                    dict(w2=P + 8), dict(sf2=P + 2), dict(ids=None), dict(ids=P + 2), dict(tw=None), dict(tw=P + 1),
                    dict(out=None), dict(out=P + 8), dict(ldx=504), dict(ldx=520), dict(ld_out=504), dict(ld_out=516),
                    dict(ld_sfx=60), dict(ld_sfx=66)):
            assert _moe(lib, fn, **bad) == INVALID, bad
        need = lib.dg_get_moe_workspace_size(64, 4, 256)
        for bad in (dict(ws=None), dict(ws=P + 16), dict(wsb=need - 1)):
            assert _moe(lib, fn, **bad) == WORKSPACE, bad
        assert _moe(lib, fn, m=0, ld_sfx=0) == 0 and _moe(lib, fn, h=0) == 0
    assert need >= 64 * 4 * 256 * 2
    assert lib.dg_get_moe_workspace_size(0, 4, 256) == 0 and lib.dg_get_moe_workspace_size(1 << 20, 64, 1 << 14) == 1 << 41


def _clip(lib, n=2, numel=16, dtype=1, data=P, out=None, count=None, max_norm=1.0, norm=P, ws=P, wsb=1 << 20):
    table = (dg._Tensor * n)(*[dg._Tensor(data, numel, dtype) for _ in range(n)])
    return lib.dg_clip_grad_norm(table, out, n if count is None else count, max_norm, norm, ws, wsb, None)


def test_clip_refusals(lib):
    for bad in (dict(count=-1), dict(numel=-1), dict(dtype=2), dict(data=None), dict(data=P + 2), dict(dtype=0, data=P + 1),
                dict(max_norm=-1.0), dict(max_norm=float("nan")), dict(norm=None), dict(norm=P + 2)):
        assert _clip(lib, **bad) == INVALID, bad
    other = (dg._Tensor * 2)(dg._Tensor(P, 16, 1), dg._Tensor(P, 17, 1))
    assert _clip(lib, out=other) == INVALID
    other = (dg._Tensor * 2)(dg._Tensor(P, 16, 1), dg._Tensor(P, 16, 0))
    assert _clip(lib, out=other) == INVALID
    assert _clip(lib, numel=1 << 45) == UNSUPPORTED
    assert lib.dg_clip_grad_norm(None, None, 2, 1.0, P, P, 1 << 20, None) == INVALID
    for bad in (dict(ws=None), dict(ws=P + 8), dict(wsb=lib.dg_get_clip_workspace_size() - 1)):
        assert _clip(lib, **bad) == WORKSPACE, bad


def test_descriptor_matches_the_header(lib):
    assert ctypes.sizeof(dg._Tensor) == 24 and dg._Tensor.numel.offset == 8 and dg._Tensor.dtype.offset == 16


def test_bindings_refuse_cpu_tensors_and_wrong_types(lib):
    x = torch.zeros(4, 256)
    q, sf = torch.zeros(4, 256, dtype=torch.uint8), torch.zeros(2, 4)
    with pytest.raises((TypeError, ValueError)):
        dg.add_rms_norm_cast_to_fp8(x, torch.ones(256), 1e-6, q, sf)
    with pytest.raises((TypeError, ValueError)):
        dg.rms_norm_backward(x, x, torch.ones(256), torch.ones(4), x, torch.ones(256))
    w13, w2 = torch.zeros(2, 512, 256, dtype=torch.uint8), torch.zeros(2, 256, 256, dtype=torch.uint8)
    with pytest.raises((TypeError, ValueError)):
        dg.fp8_moe_few_tokens((q, sf), (w13, torch.zeros(2, 4, 2)), (w2, torch.zeros(2, 2, 2)),
                              torch.zeros(4, 1, dtype=torch.int32), torch.ones(4, 1),
                              torch.zeros(4, 256, dtype=torch.bfloat16))
    with pytest.raises((TypeError, ValueError)):
        dg.clip_grad_norm([x], 1.0, torch.zeros(1))
    with pytest.raises((TypeError, ValueError)):
        dg.tensor_list([torch.zeros(3, dtype=torch.float64)])
