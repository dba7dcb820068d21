"""GPU parity of the fused residual addition + RMS norm + FP8 cast and of its
gradient against the FP64 oracle (``oracle/norm.py``, ``oracle/quant.py``).

Bounds, derived from the arithmetic (u = 2^-24, one FP32 rounding):

* s is one FP32 addition of exact inputs, then one rounding to dtype: bits.
* rstd: a thread adds at most 32 squares, then come 6 lane and 8 wave steps and
  the mean, eps, square root and reciprocal: < 64 roundings, halved by the root;
  2^-18 relative leaves room for them all (64 u = 2^-18).
* v: two more products: 2^-17; stored as BF16 half an ulp (at most 2^-8 of the
  value) more.
* codes and scales: with FP32 inputs v itself comes back as y, so they have to be
  the oracle's cast of y, bit for bit; with BF16 the pair has to stand for v within
  the cast's own half step, 2^-4 |v| + 2^-10 sf, and 2^-17 amax of v's error.
* dx: a mean of at most 16384 products summed as above (2^-18 of the sum of
  magnitudes) and a handful of products: 2^-16 of the terms' magnitudes, plus half
  an ulp, 2^-8 |dx|, of what is rounded to BF16.
* dw: at most m / grid + grid / 32 + 32 additions in a row (< 256): 2^-16 of the sum of
  magnitudes.
"""

import numpy as np
import pytest
import torch

import oracle
from workloads import gen_quant_input

pytestmark = pytest.mark.gpu

if torch.cuda.is_available():  # pragma: no cover - GPU only
    import moe_grouped_gemm_tiles_amd as dg
    from tests._gpu_harness import SENT_BF16, SENT_F32, note, to_dev

DT = {"bf16": torch.bfloat16, "fp32": torch.float32}


def _filled(rows, cols, dtype, ld=None):
    """[rows, cols] view of a sentinel-filled buffer with row stride ld."""
    shape = (rows, cols if ld is None else ld)
    t = torch.full(shape, SENT_BF16, dtype=torch.int16, device="cuda:0").view(torch.bfloat16) if dtype == "bf16" \
        else torch.full(shape, SENT_F32, dtype=torch.int32, device="cuda:0").view(torch.float32)
    return t[:, :cols]


def _pad_kept(t, cols):
    """The columns past `cols` of t's buffer still hold the sentinel."""
    full = t.as_strided((t.shape[0], t.stride(0)), (t.stride(0), 1))[:, cols:]
    want = SENT_BF16 if t.dtype == torch.bfloat16 else SENT_F32
    return bool((full.contiguous().view(torch.int16 if t.dtype == torch.bfloat16 else torch.int32) == want).all())


def _f64(t):
    return t.double().cpu().numpy()


def _run(x, w, dtype, ue=False, res=None, wdtype=None, pad=0, eps=1e-6, want_y=True):
    m, k = x.shape
    ld = k + pad
    xd = _filled(m, k, dtype, ld)
    xd.copy_(to_dev(x.astype(np.float32)))
    wd = to_dev(w.astype(np.float32)).to(DT[wdtype or dtype])
    rd = ro = None
    if res is not None:
        rd = _filled(m, k, dtype, ld)
        rd.copy_(to_dev(res.astype(np.float32)))
        ro = _filled(m, k, dtype, ld)
    kr = (k // 128 + 3) // 4 if ue else k // 128
    lds = (m + 3) // 4 * 4 + 4
    sf = torch.full((kr, lds), -7, dtype=torch.int32, device="cuda:0")
    sf = sf if ue else sf.view(torch.float32)
    q = torch.full((m, ld), 0xAA, dtype=torch.uint8, device="cuda:0")
    y = _filled(m, k, dtype, ld) if want_y else None
    rstd = torch.full((m,), -1.0, device="cuda:0")
    dg.add_rms_norm_cast_to_fp8(xd, wd, eps, q[:, :k], sf, residual=rd, residual_out=ro, y=y, rstd=rstd)
    torch.cuda.synchronize()
    assert (q[:, k:] == 0xAA).all() and (sf[:, m:].view(torch.int32) == -7).all()
    for t in (ro, y):
        assert t is None or _pad_kept(t, k)
    return dict(x=xd, w=wd, res=rd, res_out=ro, q=q[:, :k], sf=sf[:, :m], y=y, rstd=rstd)


def _check(o, dtype, ue, eps=1e-6, what=""):
    s, r, v = oracle.ref_add_rms_norm(_f64(o["x"]), _f64(o["w"]), eps, _f64(o["res"]) if o["res"] is not None else None)
    m, k = s.shape
    if o["res_out"] is not None:
        want = (o["x"].float() + o["res"].float()).to(DT[dtype])
        assert torch.equal(want, o["res_out"]), f"{what}: stored sum"
    rstd = o["rstd"].double().cpu().numpy()
    assert (np.abs(rstd - r) <= 2.0 ** -18 * r).all(), f"{what}: rstd"
    if o["y"] is not None:
        tol = 2.0 ** -17 if dtype == "fp32" else 2.0 ** -8 + 2.0 ** -16
        assert (np.abs(_f64(o["y"]) - v) <= tol * np.abs(v) + 1e-37).all(), f"{what}: y"
    q = o["q"].contiguous().cpu().numpy()
    sf = o["sf"].contiguous().cpu().numpy()
    if dtype == "fp32" and o["y"] is not None:
        wq, wsf = oracle.quant_per_token(o["y"].contiguous().cpu().numpy(), ue8m0=ue)
        assert np.array_equal(q, wq), f"{what}: {int((q != wq).sum())} codes are not the cast of y"
        assert np.array_equal(sf.view(np.int32), wsf[:, :m].view(np.int32)), f"{what}: scales"
    sd = oracle.decode_ue8m0_sf(sf, k // 128, 0) if ue else sf.astype(np.float64)
    amax = np.abs(v).reshape(m, -1, 128).max(2)
    if ue:
        lo = np.where(amax == 0, 1.0, amax / 448)
        assert (sd.T >= lo * (1 - 2.0 ** -16)).all() and (sd.T <= 2 * lo * (1 + 2.0 ** -16)).all(), f"{what}: UE8M0"
    else:
        assert (np.abs(sd.T - np.where(amax == 0, 1.0, amax / 448)) <= 2.0 ** -16 * sd.T).all(), f"{what}: sf"
    got = oracle.decode_e4m3(q).reshape(m, -1, 128) * sd.T[:, :, None]
    vb = v.reshape(m, -1, 128)
    bound = 2.0 ** -4 * np.abs(vb) + (2.0 ** -10 * sd.T + 2.0 ** -16 * amax)[:, :, None]
    assert (np.abs(got - vb) <= bound).all(), f"{what}: what the pair stands for"


def _inputs(m, k, seed, dtype, with_res=True):
    rng = np.random.default_rng(seed)
    x = gen_quant_input(m, k, seed=seed, dtype=dtype)
    res = gen_quant_input(m, k, seed=seed + 1, dtype=dtype) if with_res else None
    return x, (1 + 0.2 * rng.standard_normal(k)).astype(np.float32), res


# every chunk count and thread count: one wave, several, a wave past the row's end, blocks past a word's end
SHAPES = [(1, 128), (1, 7168), (2, 384), (3, 640), (5, 1024), (61, 1536), (17, 2048), (33, 4224), (7, 7168), (4, 16384),
          (2, 12416)]


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("ue", [False, True])
@pytest.mark.parametrize("m,k", SHAPES)
def test_norm_shapes(m, k, dtype, ue):
    x, w, res = _inputs(m, k, 300 + m + k, dtype)
    _check(_run(x, w, dtype, ue, res), dtype, ue, what=f"{m}x{k} {dtype} ue={ue}")


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("m", [1100, 8200])
def test_norm_many_rows(m, dtype):
    """The forms for many rows: fewer threads per row, several rows per workgroup, a last one with fewer."""
    for k in (896, 2048):
        x, w, res = _inputs(m, k, 310 + m, dtype)
        _check(_run(x, w, dtype, False, res), dtype, False, what=f"{m}x{k} {dtype}")
        _check(_run(x, w, dtype, True, None), dtype, True, what=f"{m}x{k} {dtype} ue8m0, no residual")


@pytest.mark.parametrize("m,k,dtype", [(8300, 8320, "bf16"), (20001, 256, "bf16"), (4200, 1152, "fp32"),
                                       (4100, 4224, "bf16")])
def test_norm_rows_per_workgroup(m, k, dtype):
    """Several rows per workgroup (with a shorter last one) and one, streaming operands; rows sampled."""
    gen = torch.Generator(device="cuda:0").manual_seed(m)
    x, res = (torch.randn(m, k, device="cuda:0", generator=gen).to(DT[dtype]) for _ in range(2))
    w = (1 + 0.2 * torch.randn(k, device="cuda:0", generator=gen)).to(DT[dtype])
    o = dict(x=x, w=w, res=res, res_out=_filled(m, k, dtype), y=_filled(m, k, dtype),
             q=torch.full((m, k), 0xAA, dtype=torch.uint8, device="cuda:0"),
             sf=torch.full((k // 128, (m + 3) // 4 * 4), -7.0, device="cuda:0"),
             rstd=torch.full((m,), -1.0, device="cuda:0"))
    dg.add_rms_norm_cast_to_fp8(x, w, 1e-6, o["q"], o["sf"], residual=res, residual_out=o["res_out"], y=o["y"],
                                rstd=o["rstd"])
    rows = torch.cat([torch.arange(40), torch.arange(m // 2, m // 2 + 40), torch.arange(m - 40, m)]).to("cuda:0")
    part = {n: t[rows] if n not in ("w", "sf") else t for n, t in o.items()}
    part["sf"] = o["sf"][:, rows]
    _check(part, dtype, False, what=f"{m}x{k} {dtype}")
    assert torch.equal(o["res_out"], (x.float() + res.float()).to(DT[dtype]))
    g = dict(dy=x, s=o["res_out"], w=w, rstd=o["rstd"], dres=res, dx=_filled(m, k, dtype),
             dw=torch.empty(k, device="cuda:0"))
    dg.rms_norm_backward(g["dy"], g["s"], w, g["rstd"], g["dx"], g["dw"], dresidual=res)
    part = {n: t[rows] if n not in ("w", "dw") else t for n, t in g.items()}
    dx, _, terms, _ = oracle.ref_rms_norm_backward(*(_f64(part[n]) for n in ("dy", "s", "w", "rstd", "dres")))
    bound = 2.0 ** -16 * terms
    bound = bound + (2.0 ** -8 * (np.abs(dx) + bound) if dtype == "bf16" else 0) + 1e-37
    assert (np.abs(_f64(part["dx"]) - dx) <= bound).all()
    t = g["dy"].double() * g["s"].double() * g["rstd"].double()[:, None]
    assert bool(((g["dw"].double() - t.sum(0)).abs() <= 2.0 ** -16 * t.abs().sum(0)).all())


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
def test_norm_strides_weight_types_and_no_residual(dtype):
    x, w, res = _inputs(19, 896, 320, dtype)
    for wdtype in ("bf16", "fp32"):
        _check(_run(x, w, dtype, False, res, wdtype=wdtype, pad=24), dtype, False, what=f"padded, {wdtype} weight")
        _check(_run(x, w, dtype, False, None, wdtype=wdtype, want_y=False), dtype, False, what="no residual, no y")


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
def test_norm_residual_in_place(dtype):
    x, w, res = _inputs(9, 1408, 330, dtype)
    base = _run(x, w, dtype, False, res)
    for alias in ("residual", "x"):
        xd, rd = base["x"].clone(), base["res"].clone()
        q, sf = torch.empty_like(base["q"]), torch.zeros(11, 12, device="cuda:0")
        dg.add_rms_norm_cast_to_fp8(xd, base["w"], 1e-6, q, sf, residual=rd,
                                    residual_out=rd if alias == "residual" else xd)
        assert torch.equal(rd if alias == "residual" else xd, base["res_out"])
        assert torch.equal(q, base["q"]) and torch.equal(sf[:, :9], base["sf"])


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("k", [128, 256])
def test_norm_narrow_rows(k, dtype):
    """Rows of which a wave takes several at a time: counts that end inside a wave, strides, and
    enough rows for workgroups that take more than one turn."""
    for m in (1, 2, 3, 4, 5, 7, 8, 9, 33, 8195, 16391):
        x, w, res = _inputs(m, k, 340 + m, dtype)
        for ue in (False, True):
            _check(_run(x, w, dtype, ue, res, pad=16), dtype, ue, what=f"{m}x{k} {dtype} ue={ue}")
        _check(_run(x, w, dtype, True, None, want_y=dtype == "fp32"), dtype, True, what=f"{m}x{k} {dtype}, no residual")


@pytest.mark.parametrize("ue", [False, True])
@pytest.mark.parametrize("k", [128, 256, 512])
def test_norm_narrow_rows_do_not_mix(k, ue):
    """Zeros, tiny, huge, infinite and NaN rows beside ordinary ones: every row's results are those
    of that row alone, bit for bit."""
    rng = np.random.default_rng(350 + k)
    x = rng.standard_normal((13, k)).astype(np.float32)
    x[1] = 0
    x[2] *= 1e-25
    x[5] *= 1e18
    x[7, 3] = np.inf
    x[8, k - 1] = np.nan
    x[10] *= 1e-38
    w = (1 + 0.1 * rng.standard_normal(k)).astype(np.float32)
    whole = _outputs(x, w, ue)
    for i in range(len(x)):
        one = _outputs(x[i:i + 1], w, ue)
        for a, b, rows in zip(whole, one, (0, 1, 0, 0)):
            assert torch.equal(a.select(rows, i), b.select(rows, 0)), i


def _outputs(x, w, ue):
    """Bits of q, sf, y and 1/rms for FP32 rows."""
    m, k = x.shape
    sf = torch.zeros((k // 128 + 3) // 4 if ue else k // 128, (m + 3) // 4 * 4, device="cuda:0",
                     dtype=torch.int32 if ue else torch.float32)
    q = torch.zeros(m, k, dtype=torch.uint8, device="cuda:0")
    y, rstd = torch.zeros(m, k, device="cuda:0"), torch.zeros(m, device="cuda:0")
    dg.add_rms_norm_cast_to_fp8(to_dev(x), to_dev(w), 1e-6, q, sf, y=y, rstd=rstd)
    return q, sf.view(torch.int32), y.view(torch.int32), rstd.view(torch.int32)


@pytest.mark.parametrize("m,k", [(4339, 8320), (1300, 8448), (1100, 16384), (600, 12544)])
def test_norm_long_rows_per_workgroup(m, k):
    """Numbers of rows that give a workgroup of long rows one to four of them, the last one fewer: every
    row's results are those of a few rows alone, bit for bit."""
    gen = torch.Generator(device="cuda:0").manual_seed(370 + m)
    x, res = (torch.randn(m, k, device="cuda:0", generator=gen).bfloat16() for _ in range(2))
    w = (1 + 0.1 * torch.randn(k, device="cuda:0", generator=gen)).bfloat16()

    def run(rows):
        n = len(rows)
        o = dict(q=torch.zeros(n, k, dtype=torch.uint8, device="cuda:0"), rstd=torch.zeros(n, device="cuda:0"),
                 sf=torch.zeros(k // 128, (n + 3) // 4 * 4, device="cuda:0"), s=torch.zeros_like(x[rows]))
        dg.add_rms_norm_cast_to_fp8(x[rows], w, 1e-6, o["q"], o["sf"], residual=res[rows], residual_out=o["s"],
                                    rstd=o["rstd"])
        return o["q"], o["rstd"], o["sf"].T, o["s"]

    whole = run(torch.arange(m, device="cuda:0"))
    for at in (0, 1, 511, m // 2, m - 4):
        rows = torch.arange(at, at + 4, device="cuda:0")
        for a, b in zip(whole, run(rows)):
            assert torch.equal(a[rows], b), at


@pytest.mark.parametrize("ue", [False, True])
@pytest.mark.parametrize("m,k,dtype", [(6151, 4224, "bf16"), (4099, 640, "bf16"), (2050, 1152, "fp32"),
                                       (3077, 8320, "fp32"), (5200, 4480, "fp32"), (2500, 9216, "bf16")])
def test_norm_codes_alone(m, k, dtype, ue):
    """Neither residual nor y: up to six rows per workgroup, the last one fewer; every row's results are
    those of a few rows alone, bit for bit."""
    gen = torch.Generator(device="cuda:0").manual_seed(380 + m)
    x = torch.randn(m, k, device="cuda:0", generator=gen).to(DT[dtype])
    w = (1 + 0.1 * torch.randn(k, device="cuda:0", generator=gen)).to(DT[dtype])

    def run(x):
        n = len(x)
        sf = torch.zeros((k // 128 + 3) // 4 if ue else k // 128, (n + 3) // 4 * 4, device="cuda:0",
                         dtype=torch.int32 if ue else torch.float32)
        q, rstd = torch.zeros(n, k, dtype=torch.uint8, device="cuda:0"), torch.zeros(n, device="cuda:0")
        dg.add_rms_norm_cast_to_fp8(x, w, 1e-6, q, sf, rstd=rstd)
        return q, rstd, sf.T[:n]

    whole = run(x)
    for at in (0, 5, 767, m // 2, m - 4):
        for a, b in zip(whole, run(x[at:at + 4])):
            assert torch.equal(a[at:at + 4], b), at


@pytest.mark.parametrize("k", [128, 256])
def test_norm_narrow_rows_far_apart(k):
    """Rows 256 MiB apart: too far for 32-bit offsets between the rows of a wave."""
    rng = np.random.default_rng(360 + k)
    x, w = rng.standard_normal((5, k)).astype(np.float32), np.ones(k, np.float32)
    far = torch.empty(5, 1 << 26, device="cuda:0")[:, :k]
    far.copy_(to_dev(x))
    near, out = to_dev(x), []
    for a in (near, far):
        q = torch.zeros(5, k, dtype=torch.uint8, device="cuda:0")
        sf, rstd = torch.zeros(k // 128, 8, device="cuda:0"), torch.zeros(5, device="cuda:0")
        dg.add_rms_norm_cast_to_fp8(a, to_dev(w), 1e-6, q, sf, rstd=rstd)
        dx, dw = torch.zeros(5, k, device="cuda:0"), torch.zeros(k, device="cuda:0")
        dg.rms_norm_backward(near, a, to_dev(w), rstd, dx, dw)
        out.append((q, sf, rstd, dx, dw))
    for i in range(4):  # each row's sums are added in the same order either way
        assert torch.equal(out[0][i], out[1][i]), i
    # five terms of at most 16, added in another order: 4 roundings of 2^-24 each way
    assert bool(((out[0][4] - out[1][4]).abs() <= 5 * 16 * 2.0 ** -21).all())


def test_norm_zero_rows_and_extremes():
    """A zero row (rstd = 1/sqrt(eps), all-zero blocks have scale 1), rows near both ends of the range."""
    rng = np.random.default_rng(340)
    x = rng.standard_normal((6, 512)).astype(np.float32)
    x[0] = 0
    x[1] *= 1e-18
    x[2] *= 1e18
    x[3, 128:256] = 0
    o = _run(x, np.ones(512, np.float32), "fp32", eps=1e-6)
    _check(o, "fp32", False, what="extremes")
    assert not o["q"][0].any() and (o["sf"][:, 0] == 1).all() and o["sf"][1, 3] == 1
    assert not o["q"][3, 128:256].any()


@pytest.mark.parametrize("ue", [False, True])
def test_norm_keeps_nan_and_inf(ue):
    """A NaN spoils its own row only; an Inf shows in its block; neither is clamped away."""
    x = np.random.default_rng(350).standard_normal((5, 512)).astype(np.float32)
    x[1, 130] = np.nan
    x[3, 300] = np.inf
    o = _run(x, np.ones(512, np.float32), "fp32", ue)
    sd = oracle.decode_ue8m0_sf(o["sf"].contiguous().cpu().numpy(), 4, 0) if ue else o["sf"].double().cpu().numpy()
    q = o["q"].contiguous().cpu().numpy()
    assert np.isnan(oracle.decode_e4m3(q[1])).all() and np.isnan(sd[:, 1]).all()
    assert np.isnan(oracle.decode_e4m3(q[3, 300])) and not np.isfinite(sd[2, 3])
    good = [0, 2, 4]
    wq, _ = oracle.quant_per_token(o["y"][good].cpu().numpy(), ue8m0=ue)
    assert np.array_equal(q[good], wq) and np.isfinite(sd[:, good]).all()


def test_norm_no_rows():
    q, sf = torch.empty(0, 256, dtype=torch.uint8, device="cuda:0"), torch.empty(2, 4, device="cuda:0")
    dg.add_rms_norm_cast_to_fp8(torch.empty(0, 256, device="cuda:0"), torch.ones(256, device="cuda:0"), 1e-6, q, sf)


def _spread(rng, k, exponents):
    """Rows of magnitudes 0.5 to 0.99 times 2^e."""
    sign = rng.choice([-1.0, 1.0], (len(exponents), k))
    return sign * rng.uniform(0.5, 0.99, sign.shape) * 2.0 ** np.array(exponents, dtype=np.float64)[:, None]


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("k", [128, 256, 640, 7168, 16384])
def test_norm_rows_at_the_top_of_the_range(k, dtype):
    """Finite rows whose sum of squares passes FP32's range, up to the type's largest values, beside
    ordinary ones: the bounds of every other row."""
    rng = np.random.default_rng(390 + k)
    x = _spread(rng, k, [0, 57, 60, 64, 100, 120, 122, 124, 126, 127, 128])
    x[4, 1:] = rng.standard_normal(k - 1)  # one large value alone
    w = (1 + 0.2 * rng.standard_normal(k)).astype(np.float32)
    for ue in (False, True):
        _check(_run(x, w, dtype, ue), dtype, ue, what=f"K={k} {dtype} ue={ue}")
        _check(_run(0.7 * x, w, dtype, ue, 0.25 * x), dtype, ue, what=f"K={k} {dtype} ue={ue}, residual")


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("k", [128, 256, 640, 7168, 16384])
def test_norm_rows_at_the_bottom_of_the_range(k, dtype):
    """eps = 0 and rows whose squares are denormal or zero in FP32, down to denormal values: the bounds of
    every other row.  (1/rms of a row of 2^-135 is past FP32's range and comes back as Inf; y, of the order
    of 1, is not.  In BF16 that row's values round to zero, and 0 * Inf is NaN on both sides.)"""
    rng = np.random.default_rng(395 + k)
    x = _spread(rng, k, [0, -48, -52, -60, -100, -120, -123, -125, -126, -127])
    w = (1 + 0.2 * rng.standard_normal(k)).astype(np.float32)
    for ue in (False, True):
        _check(_run(x, w, dtype, ue, eps=0.0), dtype, ue, eps=0.0, what=f"K={k} {dtype} ue={ue}")
    o = _run(_spread(rng, k, [0, -135, -130, 3]), w, dtype, eps=0.0)
    _, _, v = oracle.ref_add_rms_norm(_f64(o["x"]), _f64(o["w"]), 0.0)
    tol = 2.0 ** -17 if dtype == "fp32" else 2.0 ** -8 + 2.0 ** -16
    y = _f64(o["y"])
    assert ((np.abs(y - v) <= tol * np.abs(v)) | (np.isnan(v) & np.isnan(y))).all()
    assert torch.isinf(o["rstd"]).tolist() == [False, True, True, False]


@pytest.mark.parametrize("eps", [float("inf"), 3e38])
def test_norm_eps_past_the_range(eps):
    """mean + eps past FP32's range: 1/rms is what the formula gives (0 for an infinite eps)."""
    x = _spread(np.random.default_rng(397), 256, [0, 60, 64, 127])
    o = _run(x, np.ones(256, np.float32), "fp32", eps=eps)
    want = 1 / np.sqrt((_f64(o["x"]) ** 2).mean(1) + float(np.float32(eps)))
    assert (np.abs(_f64(o["rstd"]) - want) <= 2.0 ** -18 * want).all()


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("k", [128, 256, 1024, 4096, 16384])
def test_norm_rstd_is_rounded_once(k, dtype):
    """Rows of small whole numbers: every partial sum of squares is exact in FP32 (< 2^24), so is the mean
    over a power of two, and with eps = 0 only the root is left: half an ulp, and 0.01 for the higher terms."""
    rng = np.random.default_rng(398)
    x = np.stack([rng.integers(-a, a + 1, k) for a in range(1, 31) for _ in range(40)]).astype(np.float64)
    x[:, 0] = 1
    o = _run(x, np.ones(k, np.float32), dtype, eps=0.0, want_y=False)
    want = 1 / np.sqrt((x * x).mean(1))
    ulp = np.spacing(want.astype(np.float32)).astype(np.float64)
    err = np.abs(_f64(o["rstd"]) - want) / ulp
    assert (err <= 0.51).all(), f"{int((err > 0.51).sum())} of {len(err)} rows, worst {err.max():.3f} ulp"


@pytest.mark.parametrize("k", [640, 7168])
def test_norm_rstd_with_a_rounded_mean(k):
    """The same sums over other widths and with eps: the mean and its sum with eps are rounded too, at most
    2^-24 each and halved by the root."""
    rng = np.random.default_rng(399)
    x = np.stack([rng.integers(-a, a + 1, k) for a in range(1, 31) for _ in range(40)]).astype(np.float64)
    x[:, 0] = 1
    o = _run(x, np.ones(k, np.float32), "fp32", eps=1e-6, want_y=False)
    want = 1 / np.sqrt((x * x).mean(1) + float(np.float32(1e-6)))
    ulp = np.spacing(want.astype(np.float32)).astype(np.float64)
    err = np.abs(_f64(o["rstd"]) - want)
    assert (err <= 0.51 * ulp + 2.0 ** -24 * want).all()


# ---- gradient ----

def _run_backward(dy, s, w, rstd, dtype, dres=None, pad=0, wdtype=None, dw0=None, workspace=True):
    m, k = dy.shape

    def up(t):
        d = _filled(m, k, dtype, k + pad)
        d.copy_(to_dev(t.astype(np.float32)))
        return d

    o = dict(dy=up(dy), s=up(s), w=to_dev(w.astype(np.float32)).to(DT[wdtype or dtype]),
             rstd=to_dev(rstd.astype(np.float32)), dres=up(dres) if dres is not None else None,
             dx=_filled(m, k, dtype, k + pad),
             dw=torch.full((k,), float("nan"), device="cuda:0") if dw0 is None else to_dev(dw0.astype(np.float32)))
    ws = dg.alloc_rms_norm_backward_workspace(m, k) if workspace else None
    if ws is not None:
        ws.fill_(0xFF)  # any contents
    dg.rms_norm_backward(o["dy"], o["s"], o["w"], o["rstd"], o["dx"], o["dw"], dresidual=o["dres"],
                         accumulate=dw0 is not None, workspace=ws)
    torch.cuda.synchronize()
    assert _pad_kept(o["dx"], k)
    return o


def _check_backward(o, dtype, dw0=None, what=""):
    dx, dw, terms, mag = oracle.ref_rms_norm_backward(_f64(o["dy"]), _f64(o["s"]), _f64(o["w"]), _f64(o["rstd"]),
                                                      _f64(o["dres"]) if o["dres"] is not None else None)
    bound = 2.0 ** -16 * terms
    bound = bound + (2.0 ** -8 * (np.abs(dx) + bound) if dtype == "bf16" else 0) + 1e-37
    assert (np.abs(_f64(o["dx"]) - dx) <= bound).all(), f"{what}: dx"
    if dw0 is not None:
        dw, mag = dw + dw0, mag + np.abs(dw0)
    assert (np.abs(_f64(o["dw"]) - dw) <= 2.0 ** -16 * mag + 1e-37).all(), f"{what}: dw"


def _grad_inputs(m, k, seed):
    rng = np.random.default_rng(seed)
    s = rng.standard_normal((m, k)) * np.exp(rng.uniform(-3, 3, (m, 1)))
    rstd = 1 / np.sqrt((s * s).mean(1) + 1e-6)
    return rng.standard_normal((m, k)), s, 1 + 0.2 * rng.standard_normal(k), rstd, rng.standard_normal((m, k))


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("m,k", SHAPES + [(1100, 896), (2500, 256)])
def test_gradient_shapes(m, k, dtype):
    dy, s, w, rstd, dres = _grad_inputs(m, k, 400 + m + k)
    _check_backward(_run_backward(dy, s, w, rstd, dtype, dres), dtype, what=f"{m}x{k} {dtype}")
    _check_backward(_run_backward(dy, s, w, rstd, dtype), dtype, what=f"{m}x{k} {dtype}, no skip path")


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("k", [128, 256])
def test_gradient_narrow_rows(k, dtype):
    """Rows of which a wave takes several at a time: counts that end inside a wave, and many turns."""
    for m in (1, 2, 3, 4, 5, 7, 8, 9, 33, 8195, 30001):
        dy, s, w, rstd, dres = _grad_inputs(m, k, 440 + m)
        _check_backward(_run_backward(dy, s, w, rstd, dtype, dres, pad=16), dtype, what=f"{m}x{k} {dtype}")


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("k", [128, 256, 640, 16384])
def test_gradient_of_rows_at_the_ends_of_the_range(k, dtype):
    """Rows up to the type's largest values (1/rms denormal) and, with eps = 0, down to 2^-120."""
    rng = np.random.default_rng(460 + k)
    s = _spread(rng, k, [0, 60, 64, 121, 126, 127, 128, -60, -100, -120])
    rstd = (1 / np.sqrt((s * s).mean(1))).astype(np.float32)
    w = 1 + 0.2 * rng.standard_normal(k)
    _check_backward(_run_backward(rng.standard_normal(s.shape), s, w, rstd, dtype), dtype, what=f"K={k} {dtype}")


@pytest.mark.parametrize("skip", [False, True])
@pytest.mark.parametrize("m,k", [(300, 16384), (1000, 8320), (1500, 7168), (150, 16384), (230, 12416)])
def test_gradient_long_fp32_rows_in_turns(m, k, skip):
    """FP32 rows past 4096 and past 8192 values in several turns per workgroup, operands above and below
    32 MiB; every value of dx and dw against FP64."""
    gen = torch.Generator(device="cuda:0").manual_seed(450 + m)
    dy, s, dres = (torch.randn(m, k, device="cuda:0", generator=gen) for _ in range(3))
    w = 1 + 0.2 * torch.randn(k, device="cuda:0", generator=gen)
    rstd = torch.rsqrt(s.double().square().mean(1) + 1e-6).float()
    dx, dw = torch.full_like(dy, float("nan")), torch.full_like(w, float("nan"))
    dg.rms_norm_backward(dy, s, w, rstd, dx, dw, dresidual=dres if skip else None)
    r = rstd.double()[:, None]
    xhat, g = s.double() * r, dy.double() * w.double()
    want = r * (g - xhat * (g * xhat).mean(1, keepdim=True))
    terms = r * (g.abs() + xhat.abs() * (g * xhat).abs().mean(1, keepdim=True))
    if skip:
        want, terms = want + dres.double(), terms + dres.double().abs()
    assert bool(((dx.double() - want).abs() <= 2.0 ** -16 * terms).all())
    t = dy.double() * xhat
    assert bool(((dw.double() - t.sum(0)).abs() <= 2.0 ** -16 * t.abs().sum(0)).all())


def test_gradient_strides_accumulation_and_own_workspace():
    dy, s, w, rstd, dres = _grad_inputs(45, 640, 410)
    dw0 = np.random.default_rng(411).standard_normal(640).astype(np.float32)
    for dtype in ("bf16", "fp32"):
        for wdtype in ("bf16", "fp32"):
            o = _run_backward(dy, s, w, rstd, dtype, dres, pad=16, wdtype=wdtype, dw0=dw0, workspace=False)
            _check_backward(o, dtype, dw0=dw0, what=f"{dtype}, {wdtype} weight")


def test_gradient_in_place_and_repeatable():
    dy, s, w, rstd, dres = _grad_inputs(300, 1152, 420)
    base = _run_backward(dy, s, w, rstd, "bf16", dres)
    again = _run_backward(dy, s, w, rstd, "bf16", dres)
    assert torch.equal(base["dx"], again["dx"]) and torch.equal(base["dw"], again["dw"])
    for name in ("dy", "dres"):
        t = {n: base[n].clone() for n in ("dy", "dres")}
        dw = torch.empty_like(base["dw"])
        dg.rms_norm_backward(t["dy"], base["s"], base["w"], base["rstd"], t[name], dw, dresidual=t["dres"])
        assert torch.equal(t[name], base["dx"]) and torch.equal(dw, base["dw"])


def test_gradient_no_rows():
    """No rows: dw is overwritten with zeros, or kept when it is added to."""
    e = torch.empty(0, 256, device="cuda:0")
    dw = torch.ones(256, device="cuda:0")
    args = (e, e, torch.ones(256, device="cuda:0"), torch.empty(0, device="cuda:0"), torch.empty_like(e), dw)
    dg.rms_norm_backward(*args, accumulate=True)
    assert (dw == 1).all()
    dg.rms_norm_backward(*args)
    assert (dw == 0).all()


def test_gradient_matches_differences_of_the_forward():
    """Central differences of sum(dy * y) through the forward kernel (FP32), in five directions.
    With |d| = 1 per element and h = 2^-5 relative to |x| ~ 1 the third-order term is about
    h^2 / 6 * |dL| < 2^-12 of the terms' magnitude; y's rounding, 2^-22 of each of the 512 terms, over
    2h gives 2^-18 of the sum of magnitudes."""
    m, k, h = 2, 256, 2.0 ** -5
    rng = np.random.default_rng(430)
    x, dy = rng.standard_normal((m, k)), rng.standard_normal((m, k))
    w = 1 + 0.2 * rng.standard_normal(k)
    base = _run(x, w, "fp32")
    g = _run_backward(dy, x, w, _f64(base["rstd"]), "fp32")
    dy64 = _f64(g["dy"])

    def loss(x_, w_):
        return float((dy64 * _f64(_run(x_, w_, "fp32")["y"])).sum())

    scale = float(np.abs(dy64 * _f64(base["y"])).sum())
    tol = scale * (2.0 ** -10 + 2.0 ** -18)
    for _ in range(5):
        d = rng.choice([-1.0, 1.0], (m, k)) * 2.0 ** -1
        xp, xm = (x + h * d).astype(np.float32), (x - h * d).astype(np.float32)
        got = (loss(xp, w) - loss(xm, w)) / (2 * h)
        want = float((_f64(g["dx"]) * ((xp.astype(np.float64) - xm) / (2 * h))).sum())
        assert abs(got - want) <= tol, (got, want, tol)
        d = rng.choice([-1.0, 1.0], k)
        wp, wm = (w + h * d).astype(np.float32), (w - h * d).astype(np.float32)
        got = (loss(x, wp) - loss(x, wm)) / (2 * h)
        want = float((_f64(g["dw"]) * ((wp.astype(np.float64) - wm) / (2 * h))).sum())
        assert abs(got - want) <= tol, (got, want, tol)
    note(f"differences agree within {tol:.2e} of {scale:.2e}")


def test_norm_on_another_stream_and_in_a_graph():
    """On a side stream, and captured: forward and gradient replayed four times between eager calls."""
    x, w, res = _inputs(70, 896, 440, "bf16")
    base = _run(x, w, "bf16", False, res)
    q, sf = torch.empty_like(base["q"]).contiguous(), torch.zeros(7, 72, device="cuda:0")
    ro, rstd = torch.empty_like(base["res_out"]).contiguous(), torch.empty(70, device="cuda:0")
    dx, dw = torch.empty_like(ro), torch.empty(896, device="cuda:0")
    ws = dg.alloc_rms_norm_backward_workspace(70, 896)

    def both():
        dg.add_rms_norm_cast_to_fp8(base["x"], base["w"], 1e-6, q, sf, residual=base["res"], residual_out=ro, rstd=rstd)
        dg.rms_norm_backward(base["x"], ro, base["w"], rstd, dx, dw, workspace=ws)

    st = torch.cuda.Stream()
    st.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(st):
        both()
    torch.cuda.current_stream().wait_stream(st)
    torch.cuda.synchronize()
    assert torch.equal(q, base["q"]) and torch.equal(sf[:, :70], base["sf"]) and torch.equal(ro, base["res_out"])
    want = dx.clone(), dw.clone()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        both()
    for _ in range(4):
        for t in (q, ro, dx, dw, sf):
            t.zero_()
        ws.fill_(0xFF)
        g.replay()
        torch.cuda.synchronize()
        assert torch.equal(q, base["q"]) and torch.equal(ro, base["res_out"])
        assert torch.equal(dx, want[0]) and torch.equal(dw, want[1])
        _run(x, w, "bf16", True, res)
