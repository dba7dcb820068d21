"""GPU parity of the global gradient norm and clipping against the oracle
(``oracle/clip.py``).  The squares are summed in FP64 and the norm is rounded
once to FP32 (2^-24); the factor takes two more FP32 roundings and each product
one: 2^-22 relative for the norm, 2^-21 for FP32 results, half a BF16 ulp (2^-8 of
the value) more for BF16 ones."""

import math

import numpy as np
import pytest
import torch

import oracle

pytestmark = pytest.mark.gpu

if torch.cuda.is_available():  # pragma: no cover - GPU only
    import moe_grouped_gemm_tiles_amd as dg
    from tests._gpu_harness import note, to_dev

DT = {"bf16": torch.bfloat16, "fp32": torch.float32}


def _grads(sizes, dtypes, seed, scale=1.0):
    rng = np.random.default_rng(seed)
    return [to_dev((scale * rng.standard_normal(n)).astype(np.float32)).to(DT[d]) for n, d in zip(sizes, dtypes)]


def _check(grads, max_norm, norm, out, what=""):
    want, scaled = oracle.ref_clip([g.double().cpu().numpy() for g in grads], max_norm)
    assert abs(float(norm) - want) <= 2.0 ** -22 * want, f"{what}: norm {float(norm)} {want}"
    for i, (o, s) in enumerate(zip(out, scaled)):
        tol = 2.0 ** -21 if o.dtype == torch.float32 else 2.0 ** -8 + 2.0 ** -20
        assert (np.abs(o.double().cpu().numpy() - s) <= tol * np.abs(s) + 1e-38).all(), f"{what}: tensor {i}"


def _norm():
    return torch.full((1,), -1.0, device="cuda:0")


SIZES = [
    [1], [7], [8], [8191, 8192, 8193], [0, 5, 0, 0, 3, 0], [100000, 1, 17, 65536 * 4 + 3],
    [33] * 127, [40] * 128, [9] * 300, [3_000_001],
]


@pytest.mark.parametrize("kind", ["fp32", "bf16", "mixed"])
@pytest.mark.parametrize("sizes", SIZES, ids=lambda s: f"{len(s)}x{max(s)}")
def test_clip_sizes(sizes, kind):
    dtypes = [kind if kind != "mixed" else ("bf16", "fp32")[i % 2] for i in range(len(sizes))]
    grads = _grads(sizes, dtypes, 700 + len(sizes))
    out = [torch.full_like(g, float("nan")) for g in grads]
    norm = _norm()
    dg.clip_grad_norm(grads, 0.5, norm, out=out)
    _check(grads, 0.5, norm, out, "out of place")
    mine = [g.clone() for g in grads]
    dg.clip_grad_norm(mine, 0.5, norm)
    _check(grads, 0.5, norm, mine, "in place")
    for a, b in zip(mine, out):
        assert torch.equal(a, b)


def test_clip_not_needed():
    """A norm below the limit: the same bits, also out of place."""
    grads = _grads([1000, 3], ["fp32", "bf16"], 710, scale=1e-3)
    out = [torch.zeros_like(g) for g in grads]
    norm = _norm()
    dg.clip_grad_norm(grads, 100.0, norm, out=out)
    _check(grads, 100.0, norm, out)
    for g, o in zip(grads, out):
        assert torch.equal(g, o)
    mine = [g.clone() for g in grads]
    dg.clip_grad_norm(mine, math.inf, norm)
    assert all(torch.equal(a, b) for a, b in zip(mine, grads))


@pytest.mark.parametrize("shift_in", range(4))
@pytest.mark.parametrize("shift_out", [0, 1, 4])
def test_clip_unaligned_tensors(shift_in, shift_out):
    """Tensors that start anywhere: views into one flat buffer, the neighbours untouched."""
    for dtype in ("fp32", "bf16"):
        flat = _grads([20000], [dtype], 720 + shift_in)[0]
        dst = torch.full_like(flat, 7.0)
        grads = [flat[shift_in:shift_in + 9001], flat[9100 + shift_in:9103 + shift_in]]
        out = [dst[shift_out:shift_out + 9001], dst[9200 + shift_out:9203 + shift_out]]
        norm = _norm()
        dg.clip_grad_norm(grads, 1.0, norm, out=out)
        _check(grads, 1.0, norm, out, f"{dtype} {shift_in} {shift_out}")
        kept = torch.ones(20000, dtype=torch.bool, device="cuda:0")
        kept[shift_out:shift_out + 9001] = False
        kept[9200 + shift_out:9203 + shift_out] = False
        assert (dst[kept] == 7.0).all()


def test_clip_large_and_small_values():
    """Squares past FP32's range, and below it: the FP64 sum holds them."""
    for scale in (1e25, 1e-30):
        grads = _grads([5000, 77], ["fp32", "fp32"], 730, scale=scale)
        out = [torch.empty_like(g) for g in grads]
        norm = _norm()
        dg.clip_grad_norm(grads, 1.0, norm, out=out)
        _check(grads, 1.0, norm, out, f"scale {scale}")


def test_clip_norm_not_finite():
    grads = _grads([100, 100], ["fp32", "fp32"], 740)
    grads[1][3] = math.inf
    out = [torch.empty_like(g) for g in grads]
    norm = _norm()
    dg.clip_grad_norm(grads, 1.0, norm, out=out)
    assert math.isinf(float(norm)) and (out[0] == 0).all() and math.isnan(float(out[1][3]))
    grads[1][3] = math.nan
    dg.clip_grad_norm(grads, 1.0, norm, out=out)
    assert math.isnan(float(norm)) and torch.isnan(out[0]).all()
    kept = [g.clone() for g in grads]
    dg.clip_grad_norm(grads, math.inf, norm)  # only measured
    assert math.isnan(float(norm)) and torch.equal(grads[0], kept[0])


def test_clip_no_tensors_and_all_zero():
    norm = _norm()
    dg.clip_grad_norm([], 1.0, norm)
    assert float(norm) == 0.0
    z = [torch.zeros(5, device="cuda:0")]
    dg.clip_grad_norm(z, 0.0, norm)
    assert float(norm) == 0.0 and (z[0] == 0).all()


def test_clip_repeatable_on_another_stream_and_in_a_graph():
    grads = _grads([50000, 3, 70001], ["fp32", "bf16", "bf16"], 750)
    out = [torch.empty_like(g) for g in grads]
    ws, norm = dg.alloc_clip_workspace(), _norm()
    lists = dg.tensor_list(grads), dg.tensor_list(out)
    dg.clip_grad_norm(lists[0], 0.7, norm, out=lists[1], workspace=ws)
    want = [o.clone() for o in out] + [norm.clone()]
    st = torch.cuda.Stream()
    st.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(st):
        dg.clip_grad_norm(lists[0], 0.7, norm, out=lists[1], workspace=ws)
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(out + [norm], want))
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        dg.clip_grad_norm(lists[0], 0.7, norm, out=lists[1], workspace=ws)
    for _ in range(4):
        for o in out:
            o.zero_()
        ws.fill_(0xFF)
        g.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(out + [norm], want))
        dg.clip_grad_norm([o.clone() for o in out], 0.1, torch.empty(1, device="cuda:0"))


def test_clip_large():
    """256 MiB in three tensors (FP64 reference on the GPU)."""
    gen = torch.Generator(device="cuda:0").manual_seed(760)
    grads = [torch.randn(n, device="cuda:0", generator=gen) for n in (40_000_001, 25_000_000, 2_000_000)]
    out = [torch.empty_like(g) for g in grads]
    norm = _norm()
    dg.clip_grad_norm(grads, 1.0, norm, out=out)
    want = math.sqrt(sum(float(g.double().square().sum()) for g in grads))
    assert abs(float(norm) - want) <= 2.0 ** -22 * want
    for g, o in zip(grads, out):
        ref = g.double() / (want + 1e-6)
        assert bool(((o.double() - ref).abs() <= 2.0 ** -21 * ref.abs()).all())
    note(f"norm {float(norm)}")


def test_clip_large_with_empty_tensors_at_the_end():
    """More tensors than one launch takes, the last ones without elements but with addresses."""
    gen = torch.Generator(device="cuda:0").manual_seed(770)
    data = torch.randn(10_000_000, device="cuda:0", generator=gen)
    lists = []
    for t in (data, torch.empty_like(data)):
        tensors = dg.tensor_list([t] + [t[:0]] * 140)
        for i in range(1, 141):
            tensors.table[i].data = t.data_ptr()
        lists.append(tensors)
    norm = _norm()
    dg.clip_grad_norm(lists[0], 1.0, norm, out=lists[1])
    want = math.sqrt(float(data.double().square().sum()))
    assert abs(float(norm) - want) <= 2.0 ** -22 * want
    ref = data.double() / (want + 1e-6)
    assert bool(((lists[1].tensors[0].double() - ref).abs() <= 2.0 ** -21 * ref.abs()).all())


def _replace_data(t):
    t.data = torch.ones(t.numel(), dtype=t.dtype, device="cuda:0")


CHANGES = {
    "data replaced": _replace_data,
    "set to another storage": lambda t: t.set_(torch.ones(t.numel(), dtype=t.dtype, device="cuda:0")),
    "grown": lambda t: t.resize_(t.numel() * 64),
    "shrunk in place": lambda t: t.resize_(t.numel() - 1),
    "narrowed": lambda t: setattr(t, "data", t.data[:-2]),
}


@pytest.mark.parametrize("role", ["grads", "out"])
@pytest.mark.parametrize("how", list(CHANGES))
def test_clip_refuses_a_list_whose_tensors_have_moved(how, role):
    """Descriptors made before a tensor got another storage or size are not used: the call raises and
    launches nothing.  A new list over the same tensors works."""
    sets = {n: _grads([300, 5000, 40], ["fp32", "bf16", "fp32"], 790) for n in ("grads", "out")}
    lists = {n: dg.tensor_list(t) for n, t in sets.items()}
    norm = _norm()
    dg.clip_grad_norm(lists["grads"], 0.5, norm, out=lists["out"])  # as made
    dg.clip_grad_norm(lists["grads"], 0.5, norm, out=lists["out"])
    before = float(norm)
    kept = [t.clone() for t in sets["grads"]]
    norm.fill_(-1.0)
    CHANGES[how](sets[role][1])
    with pytest.raises(ValueError, match=role):
        dg.clip_grad_norm(lists["grads"], 0.5, norm, out=lists["out"])
    if role == "grads":
        with pytest.raises(ValueError, match=role):
            dg.clip_grad_norm(lists["grads"], 0.5, norm)
    torch.cuda.synchronize()
    assert float(norm) == -1.0
    for i in (0, 2):
        assert torch.equal(sets["grads"][i], kept[i])
    sets[role][1].resize_(5000).copy_(kept[1] if role == "out" else _grads([5000], ["bf16"], 791)[0])
    dg.clip_grad_norm(dg.tensor_list(sets["grads"]), 0.5, norm, out=dg.tensor_list(sets["out"]))
    _check(sets["grads"], 0.5, norm, sets["out"], how)
    assert before > 0.5


def _check_large(grads, kept, max_norm, norm, out, what):
    """The bounds of the small sets, with FP64 sums on the GPU; ``kept`` are the gradients as they were."""
    want = math.sqrt(sum(float(g.double().square().sum()) for g in kept))
    assert abs(float(norm) - want) <= 2.0 ** -22 * want, what
    c = min(1.0, max_norm / (want + 1e-6))
    for i, (g, o) in enumerate(zip(kept, out)):
        ref = g.double() * c
        tol = 2.0 ** -21 if o.dtype == torch.float32 else 2.0 ** -8 + 2.0 ** -20
        assert bool(((o.double() - ref).abs() <= tol * ref.abs() + 1e-38).all()), f"{what}: tensor {i}"


def _large_set(kind, shift):
    """360 to 460 MB in 150 tensors, two launches; each tensor starts ``shift`` elements into its own buffer."""
    gen = torch.Generator(device="cuda:0").manual_seed(780 + shift)
    sizes = [20_000_003, 0, 13_000_001, 1, 4097] + [(i * 7919) % 90_000 + 1 for i in range(140)] + [14_999_999] * 5
    grads = []
    for i, n in enumerate(sizes):
        half = kind == "bf16" or (kind == "mixed" and i % 2 == 1)
        n = 2 * n if kind == "bf16" else n
        t = torch.randn(n + 8, device="cuda:0", generator=gen)
        grads.append((t.bfloat16() if half else t)[shift:shift + n])
    return grads


@pytest.mark.parametrize("shift", [0, 3])
@pytest.mark.parametrize("kind", ["fp32", "bf16", "mixed"])
def test_clip_past_the_last_level_cache(kind, shift):
    """More than 256 MiB over two launches, so that the first pass streams and then stops streaming: out of
    place (inputs and outputs that start alike and differently), in place, and in place with nothing to clip."""
    grads = _large_set(kind, shift)
    size = sum(g.numel() * g.element_size() for g in grads)
    assert size > (256 << 20) + (32 << 20) and len(grads) > 128
    norm = _norm()
    for back in (shift, 1):
        out = [torch.full((g.numel() + 8,), float("nan"), dtype=g.dtype, device="cuda:0")[back:back + g.numel()]
               for g in grads]
        dg.clip_grad_norm(grads, 0.5, norm, out=out)
        _check_large(grads, grads, 0.5, norm, out, f"{kind}, starts {shift} and {back}")
    whole = [g.as_strided((g.numel() + 8,), (1,), 0).clone() for g in grads]
    mine = [t[shift:shift + g.numel()] for t, g in zip(whole, grads)]
    dg.clip_grad_norm(mine, 1e9, norm)
    assert all(torch.equal(a, b) for a, b in zip(mine, grads)), "a factor of 1"
    dg.clip_grad_norm(mine, 0.5, norm)
    _check_large(mine, grads, 0.5, norm, mine, f"{kind}, in place")
    assert all(torch.equal(a, b) for a, b in zip(mine, out)), "in place and out of place"
    for t, g in zip(whole, grads):
        full = g.as_strided((g.numel() + 8,), (1,), 0)
        assert torch.equal(t[:shift], full[:shift]) and torch.equal(t[shift + g.numel():], full[shift + g.numel():])


@pytest.mark.parametrize("kind", ["fp32", "bf16", "mixed"])
def test_clip_streamed_sets_below_the_last_level_cache(kind):
    """Between 32 and 256 MiB, one launch: in place and out of place."""
    grads = _large_set(kind, 0)[2:100]
    assert 32 << 20 < sum(g.numel() * g.element_size() for g in grads) < 256 << 20
    out, mine, norm = [torch.empty_like(g) for g in grads], [g.clone() for g in grads], _norm()
    dg.clip_grad_norm(grads, 2.0, norm, out=out)
    _check_large(grads, grads, 2.0, norm, out, kind)
    dg.clip_grad_norm(mine, 2.0, norm)
    assert all(torch.equal(a, b) for a, b in zip(mine, out))
