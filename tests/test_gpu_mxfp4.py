"""GPU tests of the 4-bit cast (bit for bit) and products, against the FP64 oracle.

Products: every A * B term is exact in FP32 (two 2-bit significands and a power of two), so FP32 results differ by
the K additions alone, each off by at most a step of the sum of magnitudes S (the matrix cores may truncate):
K * 2^-23 * S, and K terms of C's addition with it; a BF16 result by half a step more, 2^-8 of itself.  With unit scales every sum is a
multiple of 1/4 below 2^22, so results are exact.
"""

import numpy as np
import pytest
import torch

import oracle

pytestmark = pytest.mark.gpu

if torch.cuda.is_available():  # pragma: no cover - GPU only
    import moe_grouped_gemm_tiles_amd as dg
    from tests._gpu_harness import DEV, as_f64, out_buffer, raw_bits, sentinel_of, to_dev

DT = {"bf16": torch.bfloat16, "fp32": torch.float32}


def ld4(n):
    return -(-n // 4) * 4


# ---------------------------------------------------------------- cast

def scale_bytes(sf):
    """Scale words [.., K/128, M] -> bytes [.., M, K/32]."""
    return np.ascontiguousarray(np.swapaxes(sf.cpu().numpy(), -1, -2)).view(np.uint8)


def run_cast(x, values=True, masked_m=None, pad=0):
    """x: tensor [.., M, K] on the GPU -> (codes, scale bytes, values) as numpy, untouched places still the sentinel."""
    lead, (m, k) = x.shape[:-2], x.shape[-2:]
    q = torch.full((*lead, m, k // 2), 0xA5, dtype=torch.uint8, device=DEV)
    sf = torch.full((*lead, k // 128, m + pad), 0x5A5A5A5A, dtype=torch.int32, device=DEV)
    y = torch.full_like(x, 77.0) if values else None
    dg.cast_to_mxfp4(x, q, sf, y=y, masked_m=masked_m)
    torch.cuda.synchronize()
    assert (sf[..., m:] == 0x5A5A5A5A).all()
    byte = scale_bytes(sf[..., :m])
    return q.cpu().numpy(), byte, None if y is None else as_f64(y)


def check_cast(x, **kw):
    q, byte, y = run_cast(x, **kw)
    rq, rbyte, ry = oracle.ref_cast_mxfp4(as_f64(x).reshape(-1, x.shape[-1]))
    np.testing.assert_array_equal(byte.reshape(rbyte.shape), rbyte)
    np.testing.assert_array_equal(q.reshape(rq.shape), rq)
    if y is not None:  # in x's type, which holds every value but 4 * 2^126 (inputs past 3.5 * 2^126 round to it): Inf there
        with np.errstate(over="ignore"):
            np.testing.assert_array_equal(y.reshape(ry.shape), ry.astype(np.float32))


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("m,k", [(1, 128), (1, 7168), (3, 384), (61, 640), (64, 512), (65, 1408), (130, 4224)])
def test_cast(m, k, dtype):
    g = torch.Generator().manual_seed(m * k)
    x = torch.randn(m, k, generator=g) * torch.exp(4 * torch.randn(m, 1, generator=g))
    x[m // 2, :32] = 0
    check_cast(x.to(DT[dtype]).to(DEV), pad=3)


def test_cast_every_bf16_largest_value():
    """One block for every positive finite BF16 value as its largest, the other values below it."""
    v = torch.arange(1, 0x7F80, dtype=torch.int16).view(torch.bfloat16).double()
    f = torch.linspace(1, 0, 32, dtype=torch.float64) * torch.tensor([1, -1]).repeat(16)
    x = (v[:, None] * f).to(torch.bfloat16)
    x = torch.cat([x, x[-(-len(x) % 4):]]) if len(x) % 4 else x
    check_cast(x.reshape(-1, 128).to(DEV))


def test_cast_every_bf16_value_under_a_scale():
    """Every BF16 value up to 6 s, both signs, for scales in the middle and at both ends of the range."""
    for e in (0, -127, -126, -120, 125):
        v = torch.arange(0, 0x7F80, dtype=torch.int16).view(torch.bfloat16).double()
        top = 6.0 * 2.0 ** e
        v = v[v <= top]
        v = torch.cat([v, -v])
        v = torch.cat([v, torch.zeros(-len(v) % 124)])
        x = torch.cat([torch.full((len(v) // 31, 1), top, dtype=torch.float64), v.view(-1, 31)], 1)
        check_cast(x.view(-1, 128).to(torch.bfloat16).to(DEV))


def test_cast_fp32_next_to_the_midpoints():
    mids = np.array([0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0], dtype=np.float32)
    vals = np.concatenate([mids, np.nextafter(mids, np.float32(0)), np.nextafter(mids, np.float32(9)), [6.0, 0.0, 2.0 ** -149]])
    row = np.zeros(32, dtype=np.float32)
    row[:len(vals)] = vals
    rows = []
    for e in (0, -100, -126, 100, 125):
        for sign in (1, -1):
            rows.append(np.ldexp(row * np.float32(sign), e).astype(np.float32))
    # amax on both sides of 6 * 2^e
    edge = np.zeros((6, 32), dtype=np.float32)
    edge[:, 3] = [6, np.nextafter(np.float32(6), np.float32(9)), np.nextafter(np.float32(6), np.float32(0)), 2.0 ** -149,
                  np.finfo(np.float32).max, 6 * 2.0 ** -127]
    x = np.concatenate([np.stack(rows), edge])
    check_cast(to_dev(x.reshape(-1, 128)))


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
def test_cast_blocks_that_are_not_finite(dtype):
    x = torch.randn(5, 256)
    x[1, 40], x[2, 200], x[3, 0], x[3, 255] = float("nan"), float("inf"), -float("inf"), float("nan")
    check_cast(x.to(DT[dtype]).to(DEV))


def test_cast_strided_and_in_place():
    wide = torch.randn(37, 1024, device=DEV).bfloat16()
    x = wide[:, 128:640]
    want = oracle.ref_cast_mxfp4(as_f64(x))
    q = torch.full((37, 512), 0xA5, dtype=torch.uint8, device=DEV)
    sf = torch.full((4, 50), 7, dtype=torch.int32, device=DEV)
    before = wide.clone()
    dg.cast_to_mxfp4(x, q[:, 16:272], sf[:, :40], y=x)
    np.testing.assert_array_equal(q[:, 16:272].cpu().numpy(), want[0])
    assert (q[:, :16] == 0xA5).all() and (q[:, 272:] == 0xA5).all() and (sf[:, 37:] == 7).all()
    np.testing.assert_array_equal(as_f64(x), want[2])
    assert torch.equal(wide[:, :128], before[:, :128]) and torch.equal(wide[:, 640:], before[:, 640:])


@pytest.mark.parametrize("values", [True, False])
def test_cast_groups_with_fewer_rows(values):
    counts = [0, 70, -3, 1, 200, 64]
    x = torch.randn(6, 70, 384, device=DEV)
    masked = torch.tensor(counts, dtype=torch.int32, device=DEV)
    q, byte, y = run_cast(x, values=values, masked_m=masked, pad=2)
    for g, c in enumerate(counts):
        c = min(max(c, 0), 70)
        rq, rbyte, ry = oracle.ref_cast_mxfp4(as_f64(x[g, :c])) if c else (q[g, :0], byte[g, :0], None)
        np.testing.assert_array_equal(q[g, :c], rq)
        np.testing.assert_array_equal(byte[g, :c], rbyte)
        assert (q[g, c:] == 0xA5).all() and (byte[g, c:] == 0x5A).all()
        if values and c:
            np.testing.assert_array_equal(y[g, :c], ry)
            assert (y[g, c:] == 77.0).all()


def test_cast_row_offsets_past_32_bits():
    """The last rows of an input of more than 4 GiB."""
    m, k = 140000, 16384
    x = torch.zeros(m, k, dtype=torch.bfloat16, device=DEV)
    x[-70:] = torch.randn(70, k, device=DEV).bfloat16()
    q = torch.empty(m, k // 2, dtype=torch.uint8, device=DEV)
    sf = torch.empty(k // 128, m, dtype=torch.int32, device=DEV)
    dg.cast_to_mxfp4(x, q, sf)
    rq, rbyte, _ = oracle.ref_cast_mxfp4(as_f64(x[-70:]))
    np.testing.assert_array_equal(q[-70:].cpu().numpy(), rq)
    np.testing.assert_array_equal(scale_bytes(sf[:, -70:]), rbyte)
    assert not q[:-70].any() and bool((sf[:, :-70] == 0x7F7F7F7F).all())


# ---------------------------------------------------------------- products

def operand(rng, rows, k, unit=False):
    q = rng.integers(0, 256, (rows, k // 2), dtype=np.uint8)
    byte = np.full((rows, k // 32), 127, dtype=np.uint8) if unit else rng.integers(117, 138, (rows, k // 32), dtype=np.uint8)
    return q, byte


def upload(op, ld=None, fill=0x7F7F7F7F):
    q, byte = op
    return to_dev(q), to_dev(oracle.pack_scale_words(byte, ld4(len(q)) if ld is None else ld, fill))


def check(got, ref, mag, k, dtype, exact=False):
    if exact and dtype == "fp32":
        np.testing.assert_array_equal(got, ref)
        return
    tol = 0.0 if exact else k * 2.0 ** -23 * mag
    if dtype == "bf16":
        tol = tol + 2.0 ** -8 * (np.abs(ref) + tol)
    worst = np.max(np.abs(got - ref) - tol, initial=0.0)
    assert worst <= 0, worst


SHAPES = [(1, 16, 128), (1, 1000, 1408), (5, 24, 256), (16, 128, 384), (17, 200, 512), (33, 1000, 2048), (64, 264, 1664),
          (65, 130, 896), (100, 2112, 1024), (128, 512, 4096), (129, 257, 640), (300, 1000, 1408), (513, 700, 384),
          (1030, 1300, 256)]


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("m,n,k", SHAPES)
def test_dense(m, n, k, dtype):
    for unit in (True, False):
        rng = np.random.default_rng(m + n + k)
        a, b = operand(rng, m, k, unit), operand(rng, n, k, unit)
        ref, mag = oracle.ref_mxfp4(a, b)
        ld = -(-n // 8) * 8 + 8
        whole = out_buffer((m,), ld, dtype)
        d = whole[:, :n]
        dg.mxfp4_gemm_nt(upload(a), upload(b), d)
        check(as_f64(d), ref, mag, k, dtype, exact=unit)
        assert (raw_bits(whole)[:, n:] == sentinel_of(d)).all()


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("m,n,k", [(3, 72, 640), (130, 300, 896), (700, 520, 384)])
@pytest.mark.parametrize("in_place", [False, True])
def test_dense_with_c(m, n, k, dtype, in_place):
    rng = np.random.default_rng(7)
    a, b = operand(rng, m, k), operand(rng, n, k)
    ld = -(-n // 8) * 8
    c = torch.randn(m, ld, generator=torch.Generator().manual_seed(1)).to(DT[dtype]).to(DEV)[:, :n]
    ref, mag = oracle.ref_mxfp4(a, b, as_f64(c))
    d = c if in_place else out_buffer((m,), n, dtype, ld)
    dg.mxfp4_gemm_nt(upload(a), upload(b), d, c=c)
    check(as_f64(d), ref, mag, k + 1, dtype)


@pytest.mark.parametrize("m", [7, 90, 300])
def test_dense_strided_operands(m):
    """Rows of A, B and both scales further apart than they are long; what lies between is NaN scales and large codes."""
    rng = np.random.default_rng(8)
    n, k = 200, 640
    a, b = operand(rng, m, k), operand(rng, n, k)
    ref, mag = oracle.ref_mxfp4(a, b)

    def strided(op):
        q, byte = op
        wide = torch.full((len(q), k // 2 + 96), 0x77, dtype=torch.uint8, device=DEV)
        wide[:, 32:32 + k // 2] = to_dev(q)
        words = torch.full((k // 128, ld4(len(q)) + 12), -1, dtype=torch.int32, device=DEV)
        words[:, :len(q)] = to_dev(oracle.pack_scale_words(byte))
        return wide[:, 32:32 + k // 2], words

    d = out_buffer((m,), n, "fp32", n)
    dg.mxfp4_gemm_nt(strided(a), strided(b), d)
    check(as_f64(d), ref, mag, k, "fp32")


@pytest.mark.parametrize("m", [4, 140, 300])
def test_nan_scales_stay_in_their_row_and_column(m):
    rng = np.random.default_rng(9)
    a, b = operand(rng, m, 384), operand(rng, 150, 384)
    a[1][2, 11] = 255
    b[1][149, 0] = 255
    ref, mag = oracle.ref_mxfp4(a, b)
    d = out_buffer((m,), 150, "fp32", 152)
    dg.mxfp4_gemm_nt(upload(a), upload(b), d)
    got = as_f64(d)
    np.testing.assert_array_equal(np.isnan(got), np.isnan(ref))
    live = ~np.isnan(ref)
    check(got[live], ref[live], mag[live], 384, "fp32")


def test_scales_at_both_ends_of_the_range():
    rng = np.random.default_rng(10)
    a, b = operand(rng, 40, 256), operand(rng, 48, 256)
    for ea, eb in ((0, 254), (254, 0), (64, 64), (1, 253), (190, 190)):
        a[1][:], b[1][:] = ea, eb
        ref, mag = oracle.ref_mxfp4(a, b)
        d = out_buffer((40,), 48, "fp32")
        dg.mxfp4_gemm_nt(upload(a), upload(b), d)
        # nothing is asked where the magnitudes' sum is past FP32's range: partial sums may be Inf, and Inf - Inf, there
        held = mag < np.finfo(np.float32).max
        assert held.all() == ((ea, eb) != (190, 190))
        check(as_f64(d)[held], ref[held], mag[held], 256, "fp32")


def test_empty_sizes():
    d = torch.full((3, 16), 5.0, device=DEV)
    c = torch.randn(3, 16, device=DEV)
    a = torch.empty(3, 0, dtype=torch.uint8, device=DEV), torch.empty(0, 4, dtype=torch.int32, device=DEV)
    b = torch.empty(16, 0, dtype=torch.uint8, device=DEV), torch.empty(0, 16, dtype=torch.int32, device=DEV)
    dg.mxfp4_gemm_nt(a, b, d, c=c)
    assert torch.equal(d, c)
    dg.mxfp4_gemm_nt(a, b, d)
    assert not d.any()
    none = torch.empty(0, 64, dtype=torch.uint8, device=DEV), torch.empty(1, 0, dtype=torch.int32, device=DEV)
    dg.mxfp4_gemm_nt(none, (torch.zeros(16, 64, dtype=torch.uint8, device=DEV),
                            torch.zeros(1, 16, dtype=torch.int32, device=DEV)), torch.empty(0, 16, device=DEV))


def stacked(ops, ld):
    q, sf = zip(*[upload(o, ld) for o in ops])
    return torch.stack(q), torch.stack(sf)


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("n,k,sizes", [(128, 256, [128, 5, 0, 300]), (200, 384, [1, 129, 257]), (1008, 1408, [513, 40, 0, 7, 700]),
                                       (16, 128, [3])])
def test_contiguous(n, k, sizes, dtype):
    rng = np.random.default_rng(n + k)
    rows = [-(-s // 128) * 128 for s in sizes]
    index = np.full(sum(rows), -1, dtype=np.int32)
    at = 0
    for g, (s, r) in enumerate(zip(sizes, rows)):
        index[at:at + s] = g
        at += r
    a, b = operand(rng, len(index), k), [operand(rng, n, k) for _ in sizes]
    a[1][index < 0] = 255  # padding rows hold anything
    d = out_buffer((len(index),), n, dtype)
    dg.m_grouped_mxfp4_gemm_nt_contiguous(upload(a), stacked(b, ld4(n) + 4), d, to_dev(index))
    got, bits = as_f64(d), raw_bits(d)
    for g in range(len(sizes)):
        r = index == g
        if r.any():
            ref, mag = oracle.ref_mxfp4((a[0][r], a[1][r]), b[g])
            check(got[r], ref, mag, k, dtype)
    assert (bits[index < 0] == sentinel_of(d)).all()


def test_contiguous_groups_out_of_range_are_not_written():
    rng = np.random.default_rng(11)
    index = np.repeat(np.array([1, 7, -5, 0], dtype=np.int32), 128)
    index[130] = 0  # a row that does not belong to its block's group
    index[5] = 0
    a, b = operand(rng, 512, 128), [operand(rng, 64, 128) for _ in range(2)]
    d = out_buffer((512,), 64, "fp32")
    dg.m_grouped_mxfp4_gemm_nt_contiguous(upload(a), stacked(b, 64), d, to_dev(index))
    bits = raw_bits(d)
    written = ~(bits == sentinel_of(d)).all(1)
    want = np.zeros(512, dtype=bool)
    want[:128], want[384:] = True, True
    want[5] = False
    np.testing.assert_array_equal(written, want)


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("n,k,m_max,counts", [(128, 256, 64, [64, 0, 1, 33]), (200, 384, 130, [130, 129, 7]),
                                              (1008, 1408, 300, [300, -2, 999, 12, 128, 1]), (16, 128, 1, [1, 0]),
                                              (2112, 640, 20, [3] * 9)])
def test_masked(n, k, m_max, counts, dtype):
    rng = np.random.default_rng(n + k)
    a, b = [operand(rng, m_max, k) for _ in counts], [operand(rng, n, k) for _ in counts]
    for g, c in enumerate(counts):
        a[g][1][max(0, c):] = 255  # rows that are not there hold anything
    for expected in (0, 1, m_max):
        d = out_buffer((len(counts), m_max), n, dtype)
        dg.m_grouped_mxfp4_gemm_nt_masked(stacked(a, ld4(m_max)), stacked(b, ld4(n)), d,
                                          torch.tensor(counts, dtype=torch.int32, device=DEV), expected)
        got, bits = as_f64(d), raw_bits(d)
        for g, c in enumerate(counts):
            c = min(max(c, 0), m_max)
            ref, mag = oracle.ref_mxfp4((a[g][0][:c], a[g][1][:c]), b[g])
            if c:
                check(got[g, :c], ref, mag, k, dtype)
            assert (bits[g, c:] == sentinel_of(d)).all()


@pytest.mark.parametrize("m", [1, 8, 48, 128, 260])
def test_product_on_another_stream_and_in_a_graph(m):
    """Eager on a side stream and replayed several times with other inputs: always the eager bits."""
    rng = np.random.default_rng(12)
    n, k = 1040, 2944
    b = upload(operand(rng, n, k))
    ops = [upload(operand(rng, m, k)) for _ in range(3)]
    a = tuple(t.clone() for t in ops[0])
    ws = dg.alloc_mxfp4_workspace(m, n, k)
    want = []
    for o in ops:
        d = torch.empty(m, n, device=DEV)
        dg.mxfp4_gemm_nt(o, b, d, workspace=ws)
        want.append(d)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        d = torch.empty(m, n, device=DEV)
        dg.mxfp4_gemm_nt(ops[1], b, d, workspace=ws)
    torch.cuda.current_stream().wait_stream(side)
    assert torch.equal(d, want[1])
    graph = torch.cuda.CUDAGraph()
    out = torch.empty(m, n, device=DEV)
    with torch.cuda.graph(graph):
        dg.mxfp4_gemm_nt(a, b, out, workspace=ws)
    for i in (0, 1, 2, 0):
        for t, o in zip(a, ops[i]):
            t.copy_(o)
        out.zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, want[i])
        dg.mxfp4_gemm_nt(ops[2], b, d, workspace=ws)  # eager work between the replays
        assert torch.equal(d, want[2])


def test_packed_dtype_is_taken_too():
    rng = np.random.default_rng(13)
    a, b = upload(operand(rng, 20, 256)), upload(operand(rng, 32, 256))
    d, d2 = torch.empty(20, 32, device=DEV), torch.empty(20, 32, device=DEV)
    dg.mxfp4_gemm_nt(a, b, d)
    dg.mxfp4_gemm_nt((a[0].view(torch.float4_e2m1fn_x2), a[1]), (b[0].view(torch.float4_e2m1fn_x2), b[1]), d2)
    assert torch.equal(d, d2)
