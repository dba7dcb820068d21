"""Router, 4-bit cast and products run together, every tile configuration of the products, and the library's build with a
wait and a barrier after each phase of LDS traffic, which has to give the same bits."""

import ctypes
import os

import numpy as np
import pytest
import torch

import moe_grouped_gemm_tiles_amd as dg
import oracle

if torch.cuda.is_available():  # pragma: no cover - GPU only
    from examples import mxfp4_experts
    from tests._gpu_harness import DEV, as_f64, raw_bits, sentinel_of, out_buffer, to_dev
    from tests.test_gpu_mxfp4 import check, ld4, operand, stacked, upload

DEBUG_LIB = os.path.join(os.path.dirname(dg.library_path()), "libdg_debug.so")

# (m, n, k) and the tile, streaming?, split? that 256 CUs give it
DENSE = [((4000, 3600, 384), (256, 256, False, False)), ((4090, 7168, 640), (256, 224, False, False)),
         ((4000, 4104, 384), (256, 192, False, False)), ((2600, 2296, 640), (128, 128, False, False)),
         ((20, 1000, 8320), (32, 128, True, True)), ((60, 7160, 8320), (64, 128, True, True)),
         ((125, 7160, 16256), (128, 128, True, True)), ((40, 20000, 640), (64, 128, True, False))]
CONTIGUOUS = [((8, 4096, 384, 512), (256, 256)), ((16, 3584, 640, 512), (256, 224)), ((10, 2304, 384, 512), (256, 192)),
              ((5, 1008, 1408, 400), (128, 128))]
MASKED = [((16, 4096, 640, 250, 256), (256, 256, False)), ((24, 1792, 640, 200, 256), (256, 192, False)),
          ((16, 3584, 640, 240, 256), (256, 224, False)), ((40, 2048, 640, 10, 64), (32, 128, True)),
          ((40, 2048, 640, 50, 64), (64, 128, True)), ((16, 4096, 640, 64, 256), (128, 128, True))]


def test_shapes_reach_every_configuration():
    for (m, n, k), want in DENSE:
        p = dg._mxfp4_plan_for_tests("dense", m, n, k)
        assert (p["bm"], p["bn"], p["streaming"], p["splits"] > 1) == want, (m, n, k, p)
        assert (p["ws_bytes"] > 0) == want[3]
    for (g, n, k, rows), want in CONTIGUOUS:
        p = dg._mxfp4_plan_for_tests("contiguous", g * -(-rows // 128) * 128, n, k)
        assert (p["bm"], p["bn"]) == want and not p["streaming"] and p["splits"] == 1, (g, n, k, rows, p)
    for (g, n, k, rows, most), want in MASKED:
        p = dg._mxfp4_plan_for_tests("masked", rows, n, k, groups=g, most_rows=most)
        assert (p["bm"], p["bn"], p["streaming"]) == want and p["splits"] == 1, (g, n, k, rows, p)


def test_plans_are_within_their_limits():
    rng = np.random.default_rng(0)
    for _ in range(300):
        m, n = (int(np.exp(rng.uniform(0, np.log(40000)))) for _ in range(2))
        k, cus = 128 * int(rng.integers(1, 140)), int(rng.choice([1, 64, 256]))
        p = dg._mxfp4_plan_for_tests("dense", max(1, m), max(1, n), k, cus)
        slabs = (k // 128 + 1) // 2
        assert 1 <= p["splits"] <= slabs
        part = p["splits"] * -(-max(1, m) // p["bm"]) * -(-max(1, n) // p["bn"]) * p["bm"] * p["bn"] * 4
        assert p["ws_bytes"] == (65536 + part if p["splits"] > 1 else 0) and part * (p["splits"] > 1) <= 32 << 20


@pytest.fixture(scope="module")
def debug():
    lib = ctypes.CDLL(DEBUG_LIB)
    for name in dg._SIGNATURES:
        f = getattr(lib, name)
        f.restype, f.argtypes = dg._SIGNATURES[name]
    return lib


def both_builds(debug, call, fill):
    """call()'s output from the normal library; the other build has to give the same bits in the buffer that fill() makes."""
    d = fill()
    call(d)
    torch.cuda.synchronize()
    normal, dg._lib = dg._lib, debug
    try:
        d2 = fill()
        call(d2)
        torch.cuda.synchronize()
    finally:
        dg._lib = normal
    assert np.array_equal(raw_bits(d), raw_bits(d2))
    return d


def some(rows, tile):
    """Rows around tile edges, the last ones, and a few others."""
    r = {0, 1, rows - 1, rows - 2, rows // 2} | {t + o for t in range(0, rows, tile) for o in (-1, 0)}
    return np.array(sorted(x for x in r if 0 <= x < rows))


@pytest.mark.gpu
@pytest.mark.parametrize("dtype,with_c", [("bf16", False), ("fp32", True)])
@pytest.mark.parametrize("case", range(len(DENSE)))
def test_dense_tiles(debug, case, dtype, with_c):
    (m, n, k), (bm, _, _, _) = DENSE[case]
    rng = np.random.default_rng(case)
    a, b = operand(rng, m, k), operand(rng, n, k)
    ta, tb = upload(a), upload(b)
    ws = dg.alloc_mxfp4_workspace(m, n, k)
    c = torch.randn(m, n, device=DEV).to(torch.bfloat16 if dtype == "bf16" else torch.float32) if with_c else None
    d = both_builds(debug, lambda d: dg.mxfp4_gemm_nt(ta, tb, d, c=c, workspace=ws), lambda: out_buffer((m,), n, dtype))
    r = some(m, 64)
    ref, mag = oracle.ref_mxfp4((a[0][r], a[1][r]), b, None if c is None else as_f64(c[torch.from_numpy(r).to(DEV)]))
    check(as_f64(d[torch.from_numpy(r).to(DEV)]), ref, mag, k + 1, dtype)
    if ws is not None:  # counters are back at zero, and a call without a workspace of its own gives the same bits
        assert not ws[:65536].any()
        d2 = out_buffer((m,), n, dtype)
        dg.mxfp4_gemm_nt(ta, tb, d2, c=c)
        assert torch.equal(d, d2)


@pytest.mark.gpu
@pytest.mark.parametrize("case", range(len(CONTIGUOUS)))
def test_contiguous_tiles(debug, case):
    (g, n, k, rows), _ = CONTIGUOUS[case]
    rng = np.random.default_rng(case)
    per = -(-rows // 128) * 128
    sizes = [int(rng.integers(max(1, per - 300), per + 1)) for _ in range(g)]
    # groups of odd numbers of 128-row blocks meet inside a 256-row tile, which then takes two passes
    index = np.full(g * per, -1, dtype=np.int32)
    at = 0
    for i, s in enumerate(sizes):
        index[at:at + s] = i
        at += -(-s // 128) * 128
    a, b = operand(rng, g * per, k), [operand(rng, n, k) for _ in range(g)]
    ta, tb, ti = upload(a), stacked(b, ld4(n)), to_dev(index)
    d = both_builds(debug, lambda d: dg.m_grouped_mxfp4_gemm_nt_contiguous(ta, tb, d, ti), lambda: out_buffer((g * per,), n, "bf16"))
    got, bits = as_f64(d), raw_bits(d)
    for i in range(g):
        r = np.nonzero(index == i)[0]
        r = r[some(len(r), 64)]
        ref, mag = oracle.ref_mxfp4((a[0][r], a[1][r]), b[i])
        check(got[r], ref, mag, k, "bf16")
    assert (bits[index < 0] == sentinel_of(d)).all()


@pytest.mark.gpu
@pytest.mark.parametrize("case", range(len(MASKED)))
def test_masked_tiles(debug, case):
    (g, n, k, rows, most), _ = MASKED[case]
    rng = np.random.default_rng(case)
    counts = [int(c) for c in rng.integers(0, most + 1, g)]
    counts[1], counts[2] = 0, most
    a, b = [operand(rng, most, k) for _ in range(g)], [operand(rng, n, k) for _ in range(g)]
    ta, tb, mm = stacked(a, ld4(most)), stacked(b, ld4(n)), torch.tensor(counts, dtype=torch.int32, device=DEV)
    d = both_builds(debug, lambda d: dg.m_grouped_mxfp4_gemm_nt_masked(ta, tb, d, mm, rows), lambda: out_buffer((g, most), n, "bf16"))
    got, bits = as_f64(d), raw_bits(d)
    for i, c in enumerate(counts):
        assert (bits[i, c:] == sentinel_of(d)).all()
        if c:
            r = some(c, 64)
            ref, mag = oracle.ref_mxfp4((a[i][0][r], a[i][1][r]), b[i])
            check(got[i, r], ref, mag, k, "bf16")


@pytest.mark.gpu
def test_masked_with_more_groups_than_slots():
    """2500 groups, most of them empty: the numbering takes several groups to a slot."""
    rng = np.random.default_rng(3)
    g, m_max, n, k = 2500, 4, 16, 128
    counts = np.where(rng.random(g) < 0.1, rng.integers(1, m_max + 1, g), 0)
    counts[[0, 1, 2499]] = 0, 4, 3
    a, b = operand(rng, g * m_max, k), operand(rng, g * n, k)
    ta = to_dev(a[0]).view(g, m_max, -1), to_dev(np.stack([oracle.pack_scale_words(a[1][i * m_max:(i + 1) * m_max]) for i in range(g)]))
    tb = to_dev(b[0]).view(g, n, -1), to_dev(np.stack([oracle.pack_scale_words(b[1][i * n:(i + 1) * n]) for i in range(g)]))
    d = out_buffer((g, m_max), n, "fp32")
    dg.m_grouped_mxfp4_gemm_nt_masked(ta, tb, d, torch.from_numpy(counts.astype(np.int32)).to(DEV), 1)
    got, bits = as_f64(d), raw_bits(d)
    for i, c in enumerate(counts):
        assert (bits[i, c:] == sentinel_of(d)).all()
        if c:
            ref, mag = oracle.ref_mxfp4(tuple(t[i * m_max:i * m_max + c] for t in a), tuple(t[i * n:(i + 1) * n] for t in b))
            check(got[i, :c], ref, mag, k, "fp32")


@pytest.mark.gpu
def test_output_offsets_past_32_bits():
    """D of more than 4 GiB: the last rows and the first ones."""
    rng = np.random.default_rng(4)
    m, n, k = 300000, 8192, 128
    a, b = operand(rng, m, k), operand(rng, n, k)
    d = torch.empty(m, n, dtype=torch.bfloat16, device=DEV)
    dg.mxfp4_gemm_nt(upload(a), upload(b), d)
    for r in (slice(0, 70), slice(m - 130, m)):
        ref, mag = oracle.ref_mxfp4((a[0][r], a[1][r]), b)
        check(as_f64(d[r]), ref, mag, k, "bf16")


@pytest.mark.gpu
def test_a_decode_step_replays_like_the_eager_one_and_matches_the_definition():
    replayed, eager, layer = mxfp4_experts.serve(tokens=11, hidden=512, inter=256, experts=12, top_k=3, steps=4)
    for r, e in zip(replayed, eager):
        assert torch.equal(r, e)
    # the last step against FP64, from the layer's own (rounded) stages: codes, routing and BF16 activations
    ids, w = layer.ids.cpu().numpy(), as_f64(layer.weights)
    y = as_f64(layer.y)
    ref = oracle.ref_router(as_f64(layer.y @ layer.router.t()), 3, "sigmoid", bias=layer.bias.cpu().numpy())
    np.testing.assert_array_equal(ids, ref["ids"])
    np.testing.assert_array_equal(layer.counts.cpu().numpy(), ref["counts"])

    def weight(pair, e):
        byte = np.ascontiguousarray(pair[1][e].cpu().numpy()[:, :pair[0].shape[1]].T).view(np.uint8)
        return pair[0][e].cpu().numpy(), byte

    out = np.zeros_like(y)
    for t in range(11):
        for j, e in enumerate(ids[t]):
            q, byte, _ = oracle.ref_cast_mxfp4(y[t:t + 1])
            h, _ = oracle.ref_mxfp4((q, byte), weight(layer.w13, e))
            h = torch.from_numpy(h).bfloat16().double().numpy()[0]
            act = h[:256] / (1 + np.exp(-h[:256])) * h[256:]
            act = torch.from_numpy(act).bfloat16().double().numpy()[None]
            o, _ = oracle.ref_mxfp4(oracle.ref_cast_mxfp4(act)[:2], weight(layer.w2, e))
            out[t] += w[t, j] * o[0]
    # a BF16 rounding of h or act may fall the other way from an FP32 sum than from an FP64 one, and take a 4-bit code (a step of
    # up to a quarter of a value, one in 256 * 2^-15 of them) with it: the norms agree to 2^-6, not each value to a step
    off = np.linalg.norm(as_f64(replayed[-1]) - out) / np.linalg.norm(out)
    assert off < 2.0 ** -6, off


@pytest.mark.gpu
def test_a_training_step_has_the_formulas_gradients():
    s = mxfp4_experts.train(tokens=128, hidden=256, experts=8, top_k=2)
    r = oracle.ref_router(as_f64(s["logits"]), 2)
    np.testing.assert_array_equal(s["ids"].cpu().numpy(), r["ids"])
    dx, mag = oracle.ref_router_backward(as_f64(s["logits"]), r["ids"], as_f64(s["dw"]), r["counts"], r["prob_sum"], s["alpha"])
    assert (np.abs(as_f64(s["dlogits"]) - dx) <= 400 * 2.0 ** -24 * mag + 1e-37).all()
    a = oracle.ref_cast_mxfp4(as_f64(s["dout"]).T)
    b = oracle.ref_cast_mxfp4(as_f64(s["x"]).T)
    ref, m = oracle.ref_mxfp4(a[:2], b[:2])
    check(as_f64(s["dweight"]), ref, m, 129, "fp32")
    ref, m = oracle.ref_mxfp4(oracle.ref_cast_mxfp4(as_f64(s["x"]))[:2], oracle.ref_cast_mxfp4(as_f64(s["values"]))[:2])
    check(as_f64(s["out"]), ref, m, 256, "fp32")
