"""GPU parity of the few-token expert layer against the FP64 oracle (``oracle/moe.py``).

Bound per element, derived from the arithmetic:
  2^-8 |out|      the output's rounding to BF16 (half an ulp is at most 2^-8 of a value),
  2^-8 second     the activation's rounding to BF16, each term of the second sum,
  2^-16 first     the first product's FP32 sums: at most hidden / 128 scaled partial sums and
                  two products per value (< 128 roundings of 2^-24, 2^-17), and the
                  exponential's few ulps,
  2^-16 second    the same for the second product,
and 2^-6 of the first two for each rounding acting on what the others left.  The 2-norm
of the error is held to 2^-8 of the result's: a BF16 rounding's is about 2^-9.2, two
of them 2^-8.7.
"""

import numpy as np
import pytest
import torch

import oracle
from workloads import gen_moe

pytestmark = pytest.mark.gpu

if torch.cuda.is_available():  # pragma: no cover - GPU only
    import moe_grouped_gemm_tiles_amd as dg
    from tests._gpu_harness import SENT_BF16, fp8_dev, note, to_dev


def _dev(x):
    return dict(x=(fp8_dev(x["x"]), to_dev(x["sfx"])), w13=(fp8_dev(x["w13"]), to_dev(x["sf13"])),
                w2=(fp8_dev(x["w2"]), to_dev(x["sf2"])), ids=to_dev(x["ids"]), weights=to_dev(x["weights"]))


def _run(x, ld=None, workspace=None):
    d = _dev(x)
    h = x["hidden"]
    out = torch.full((x["m"], h if ld is None else ld), SENT_BF16, dtype=torch.int16, device="cuda:0")
    out = out.view(torch.bfloat16)
    dg.fp8_moe_few_tokens(d["x"], d["w13"], d["w2"], d["ids"], d["weights"], out[:, :h], workspace=workspace)
    torch.cuda.synchronize()
    assert (out[:, h:].contiguous().view(torch.int16) == SENT_BF16).all(), "columns past hidden were written"
    return out[:, :h]


def _check(x, out, what=""):
    ref, second, first = oracle.ref_moe(x["x"], x["sfx"], x["w13"], x["sf13"], x["w2"], x["sf2"], x["ids"],
                                        x["weights"], ue8m0=x["scale_fmt"] == "ue8m0")
    got = out.double().cpu().numpy()
    assert np.isfinite(got).all(), f"{what}: not finite"
    err = np.abs(got - ref)
    bound = 2.0 ** -8 * (np.abs(ref) + second) * (1 + 2.0 ** -6) + 2.0 ** -16 * (first + second)
    worst = float((err / np.where(bound > 0, bound, 1)).max()) if err.size else 0.0
    assert (err <= bound).all(), f"{what}: worst error / bound {worst:.3f}"
    norm = float(np.linalg.norm(ref))
    rel = float(np.linalg.norm(got - ref)) / norm if norm else 0.0
    assert rel <= 2.0 ** -8, f"{what}: 2-norm error {rel:.2e}"
    idle = ~((x["ids"] >= 0) & (x["ids"] < x["experts"])).any(1)
    assert (got[idle] == 0).all(), f"{what}: tokens without an expert here"
    note(f"{what}: worst={worst:.3f} rel={rel:.2e}")


@pytest.mark.parametrize("fmt", ["fp32", "ue8m0"])
@pytest.mark.parametrize("m,experts,top_k,hidden,inter,routed", [
    (1, 4, 2, 256, 128, None),      # one K block in the second product
    (1, 8, 8, 1024, 384, None),     # one token, every expert
    (3, 8, 1, 128, 256, None),      # one K block in the first product, one slot
    (17, 4, 3, 640, 640, None),     # K blocks that fill no round of the waves
    (16, 2, 2, 256, 256, None),     # every expert has 16 tokens: exactly one MFMA's columns
    (40, 3, 2, 384, 128, None),     # more than 16 tokens per expert
    (70, 2, 1, 256, 256, None),     # more than 32
    (9, 8, 4, 512, 256, 32),        # most ids are not of this device
    (5, 100, 6, 256, 128, None),    # more experts than pairs
    (13, 1, 1, 256, 128, None),     # one expert
])
def test_moe_shapes(m, experts, top_k, hidden, inter, routed, fmt):
    x = gen_moe(m, experts, top_k, hidden, inter, seed=500 + m, scale_fmt=fmt, routed=routed, poison=True)
    _check(x, _run(x), what=f"m={m} E={experts} top_k={top_k} H={hidden} I={inter} {fmt}")


@pytest.mark.parametrize("cus", [0, 64, 8])
@pytest.mark.parametrize("fmt", ["fp32", "ue8m0"])
@pytest.mark.parametrize("m,experts", [(3, 1), (7, 1), (15, 1), (20, 1), (30, 1), (45, 1), (70, 1), (24, 3)])
def test_moe_tile_forms(m, experts, fmt, cus):
    """Every number of output columns per workgroup (fewer usable CUs: wider tiles, more units per
    workgroup) with every amount of tokens per stage, up to several passes."""
    x = gen_moe(m, experts, 1, 1024, 384, seed=510 + m, scale_fmt=fmt)
    dg.set_num_cus(cus)
    try:
        _check(x, _run(x), what=f"m={m} E={experts} {fmt} cus={cus}")
    finally:
        dg.set_num_cus(0)


@pytest.mark.parametrize("m,experts,top_k", [(40, 2, 1), (17, 3, 3), (128, 2, 2)])
def test_moe_widest_rows(m, experts, top_k):
    x = gen_moe(m, experts, top_k, 7168, 128, seed=515 + m, scale_fmt="ue8m0" if m == 17 else "fp32")
    _check(x, _run(x), what=f"m={m} H=7168 I=128")


@pytest.mark.parametrize("fmt", ["fp32", "ue8m0"])
@pytest.mark.parametrize("m", [28, 33, 50, 64, 65, 90, 130])
def test_moe_many_tokens_per_expert(m, fmt):
    """Every token at both experts: 64 tokens a pass in the first product with 16 and, where each CU gets
    two units, 32 columns; 24 or 32 tokens a stage in the second."""
    x = gen_moe(m, 2, 2, 1152, 640, seed=530 + m, scale_fmt=fmt)
    for cus in (8, 0):
        dg.set_num_cus(cus)
        try:
            _check(x, _run(x), what=f"m={m} {fmt} cus={cus}")
        finally:
            dg.set_num_cus(0)


def test_moe_full_chunk_with_wide_tiles():
    """512 pairs of one expert in 32-column tiles: the sums take the most LDS, the rings the least."""
    x = gen_moe(512, 1, 1, 512, 256, seed=518)
    dg.set_num_cus(4)
    try:
        _check(x, _run(x), what="512 pairs, 32 columns")
    finally:
        dg.set_num_cus(0)


def test_moe_larger_than_one_chunk_of_pairs():
    """More than 512 (token, slot) pairs: several chunks, the last with one token."""
    x = gen_moe(2 * 128 + 1, 5, 4, 256, 128, seed=520)
    _check(x, _run(x), what="257 tokens, top 4")
    x = gen_moe(20, 70, 64, 128, 128, seed=521)
    _check(x, _run(x), what="top 64")
    x = gen_moe(520, 1, 1, 128, 128, seed=522)
    _check(x, _run(x), what="one expert, 520 tokens")


def test_moe_many_experts():
    x = gen_moe(6, 1024, 8, 128, 128, seed=530, poison=True)
    _check(x, _run(x), what="1024 experts")


def test_moe_same_expert_in_two_slots():
    x = gen_moe(6, 3, 2, 256, 128, seed=540)
    x["ids"][:, 1] = x["ids"][:, 0]
    _check(x, _run(x), what="an expert twice")


def test_moe_nothing_routed_here():
    x = gen_moe(5, 2, 2, 256, 128, seed=541)
    x["ids"][:] = -1
    x["weights"][:] = np.nan
    assert (_run(x).cpu() == 0).all()


def test_moe_row_strides_and_workspace_contents():
    """x and out with padded rows, a workspace of NaN bytes; bit-identical to the packed call."""
    x = gen_moe(7, 4, 2, 384, 256, seed=550)
    base = _run(x)
    ws = torch.full((dg.get_moe_workspace_size(7, 2, 256),), 0xFF, dtype=torch.uint8, device="cuda:0")
    assert torch.equal(base, _run(x, ld=408, workspace=ws))
    d = _dev(x)
    wide = torch.full((7, 400), 0x7F, dtype=torch.uint8, device="cuda:0")
    wide[:, :384] = d["x"][0].view(torch.uint8)
    sfx = torch.full((3, 16), float("nan"), device="cuda:0")
    sfx[:, :7] = d["x"][1][:, :7]
    out = torch.empty(7, 384, dtype=torch.bfloat16, device="cuda:0")
    dg.fp8_moe_few_tokens((wide[:, :384], sfx), d["w13"], d["w2"], d["ids"], d["weights"], out)
    assert torch.equal(base, out)


def test_moe_one_token_equals_its_row_of_a_batch():
    """A token's result does not depend on the other tokens' data (only, in the last bit, on how K is split)."""
    x = gen_moe(4, 4, 2, 512, 256, seed=560)
    full = _run(x).double().cpu().numpy()
    one = {**x, "m": 1, "x": x["x"][2:3].copy(), "ids": x["ids"][2:3].copy(), "weights": x["weights"][2:3].copy()}
    sf = np.zeros((4, 4), np.float32)
    sf[:, 0] = x["sfx"][:, 2]
    one["sfx"] = sf
    got = _run(one)
    _check(one, got, what="token 2 alone")
    assert np.abs(got.double().cpu().numpy()[0] - full[2]).max() <= 2.0 ** -7 * np.abs(full[2]).max()


def test_moe_extreme_activations():
    """Gates far from zero: silu goes to g and to 0, no overflow of the exponential reaches the result."""
    x = gen_moe(3, 2, 2, 256, 128, seed=570)
    x["sf13"] *= np.float32(400.0)
    x["sf2"] *= np.float32(1e-4)
    _check(x, _run(x), what="wide gates")


def test_moe_repeatable_on_another_stream_and_in_a_graph():
    x = gen_moe(11, 6, 3, 512, 256, seed=580, routed=8)
    d = _dev(x)
    base = _run(x)
    out = torch.empty(11, 512, dtype=torch.bfloat16, device="cuda:0")
    ws = dg.alloc_moe_workspace(11, 3, 256)

    def call():
        dg.fp8_moe_few_tokens(d["x"], d["w13"], d["w2"], d["ids"], d["weights"], out, workspace=ws)

    st = torch.cuda.Stream()
    st.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(st):
        call()
    torch.cuda.synchronize()
    assert torch.equal(out, base)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        call()
    for _ in range(4):
        out.zero_()
        ws.fill_(0xFF)
        g.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, base)
        assert torch.equal(_run(x), base)


def test_moe_no_tokens():
    x = gen_moe(1, 2, 1, 128, 128, seed=590)
    d = _dev(x)
    e = torch.empty(0, 128, dtype=torch.bfloat16, device="cuda:0")
    dg.fp8_moe_few_tokens((d["x"][0][:0], d["x"][1]), d["w13"], d["w2"], d["ids"][:0], d["weights"][:0], e)


@pytest.mark.parametrize("m,experts,top_k,hidden,inter", [(1, 16, 8, 7168, 2048), (33, 16, 4, 4096, 1024)])
def test_moe_full_size(m, experts, top_k, hidden, inter):
    x = gen_moe(m, experts, top_k, hidden, inter, seed=600 + m)
    _check(x, _run(x), what=f"m={m} H={hidden} I={inter}")
