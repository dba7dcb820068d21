"""Measured cases of the 4-bit operands with their products and of the router with its balance loss.

Four operators of the library, reached as a user reaches them:

* ``cast``  microscaled 4-bit quantisation: E2M1 codes, a power-of-two scale for each row and 32
  columns, and the values they stand for (``dg.cast_to_mxfp4``);
* ``product``  the product of two such operands, dense, over contiguous groups of rows or over
  masked groups (``dg.mxfp4_gemm_nt``, ``dg.m_grouped_mxfp4_gemm_nt_contiguous`` / ``_masked``);
* ``route``  scores, the choice of experts and their weights, tokens per expert and the balance
  loss (``dg.moe_router``);
* ``route_grad``  the gradient of both (``dg.moe_router_backward``).

With ``own`` false, ``run`` computes the same from elementary torch operations in FP32 (scores that
are compared with each other in FP64), rounded once at the end; with ``own`` true it calls the
library.  ``exact`` is the definition in FP64.
"""

import math
import random

import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "fp32": torch.float32}
E2M1 = [0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0]
TINY = 1e-20  # added to the sums that scores are divided by


# ---------------------------------------------------------------------------
# cases
# ---------------------------------------------------------------------------

def listed():
    return [
        # one decode step of one request: its hidden state quantised, latency only
        dict(name="cast decode 1x7168", op="cast", groups=0, m=1, k=7168, dtype="bf16", masked=False),
        # the FP32 activations of a ragged batch, an odd number of 128-column blocks
        dict(name="cast 4099x1408 fp32", op="cast", groups=0, m=4099, k=1408, dtype="fp32", masked=False),
        # eight experts' BF16 weights, once per optimizer step, with the values that a straight-through forward uses
        dict(name="cast weights 8x4096x7168", op="cast", groups=8, m=4096, k=7168, dtype="bf16", masked=False),
        # decode of a few requests: the reading of the weight
        dict(name="product decode 5x7168x16384", op="product", kind="dense", groups=0, m=5, n=7168, k=16384, layout=0,
             dtype="bf16", c=False),
        # an odd-sized weight gradient added to an FP32 accumulator
        dict(name="product 333x1000x1408 fp32 +C", op="product", kind="dense", groups=0, m=333, n=1000, k=1408, layout=0,
             dtype="fp32", c=True),
        # prefill through a large projection
        dict(name="product 4096x7168x16384", op="product", kind="dense", groups=0, m=4096, n=7168, k=16384, layout=0,
             dtype="bf16", c=False),
        # prefill through eight experts, tokens sorted by expert
        dict(name="product contiguous 8x4096x7168", op="product", kind="contiguous", groups=8, m=8192, n=4096, k=7168,
             layout=2, dtype="bf16", c=False),
        # decode through sixteen experts with up to 256 tokens each
        dict(name="product masked 16x4096x7168", op="product", kind="masked", groups=16, m=256, n=4096, k=7168, layout=30,
             dtype="bf16", c=False),
        # decode of a few requests: choice only, latency
        dict(name="route 7x64", op="route", m=7, experts=64, top_k=6, dtype="bf16", score="softmax", bias=False, mask=False,
             dead=0, normalize=True, loss=False),
        # a training step of a large expert layer: sigmoid scores, a bias that steers the choice, a padded batch
        dict(name="route 33280x256 sigmoid", op="route", m=33280, experts=256, top_k=8, dtype="fp32", score="sigmoid",
             bias=True, mask=True, dead=0, normalize=True, loss=True),
        # backward of a short ragged batch over an odd number of experts, two of them out of service
        dict(name="route grad 333x60", op="route_grad", m=333, experts=60, top_k=4, dtype="fp32", score="softmax", dead=2,
             normalize=False),
        # backward of the training step, BF16 logits
        dict(name="route grad 33280x256 sigmoid", op="route_grad", m=33280, experts=256, top_k=8, dtype="bf16",
             score="sigmoid", dead=0, normalize=True),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def _width(rng, lo, hi):
    """A multiple of 128 between lo and hi."""
    return max(lo, min(hi, _log(rng, lo, hi) // 128 * 128))


def draw(rng: random.Random):
    op = rng.choice(["cast", "product", "product", "route", "route_grad"])
    if op == "cast":
        k, dtype = _width(rng, 128, 16384), rng.choice(["bf16", "bf16", "fp32"])
        groups = rng.choice([0, 0, _log(rng, 2, 32)])
        most = 8 * 4096 * 7168 // (1 if dtype == "bf16" else 2) // max(1, groups)
        return dict(op=op, groups=groups, m=max(1, min(_log(rng, 1, 33280), most // k)), k=k, dtype=dtype,
                    masked=groups > 0 and rng.random() < 0.5)
    if op == "product":
        kind, dtype = rng.choice(["dense", "dense", "contiguous", "masked"]), rng.choice(["bf16", "bf16", "fp32"])
        k = _width(rng, 128, 16384)
        if kind == "dense":
            m, n = _log(rng, 1, 8192), _log(rng, 16, 24576)
            return dict(op=op, kind=kind, groups=0, m=max(1, min(m, 4096 * 7168 * 16384 // (n * k))), n=n, k=k, layout=0,
                        dtype=dtype, c=rng.random() < 0.3)
        groups, n = _log(rng, 2, 32), _log(rng, 2, 512) * 16
        rows = min(32768 if kind == "contiguous" else 8192, 32768 * 4096 * 7168 // (n * k))
        weights = max(1, 16 * 4096 * 7168 // (n * k))
        groups = max(1, min(groups, weights))
        return dict(op=op, kind=kind, groups=groups, m=max(1, min(_log(rng, 16, 8192), rows // groups)), n=n, k=k,
                    layout=rng.randint(0, 1 << 30), dtype=dtype, c=False)
    experts = _log(rng, 4, 512)
    top_k = rng.randint(1, min(12, experts))
    case = dict(op=op, m=min(_log(rng, 1, 33280), 33280 * 256 // experts), experts=experts, top_k=top_k,
                dtype=rng.choice(["bf16", "fp32"]), score=rng.choice(["softmax", "sigmoid"]),
                dead=rng.choice([0, 0, rng.randint(0, experts - top_k)]), normalize=rng.random() < 0.7)
    if op == "route":
        case.update(bias=rng.random() < 0.5, mask=rng.random() < 0.5, loss=rng.random() < 0.6)
    return case


def _rows(case):
    """Rows of each group, drawn from the case's layout."""
    r = random.Random(case["layout"])
    if case["kind"] == "contiguous":
        return [r.randint(1, case["m"]) for _ in range(case["groups"])]
    return [r.randint(0, case["m"]) for _ in range(case["groups"])]


def _padded(n, to):
    return -(-n // to) * to


def work(case):
    if case["op"] == "cast":
        rows, k = case["m"] * max(1, case["groups"]), case["k"]
        if case["masked"]:
            rows //= 2  # on average
        es = 2 if case["dtype"] == "bf16" else 4
        return dict(bytes=rows * k * (2 * es + 0.5 + 1 / 32), flops=4 * rows * k)
    if case["op"] == "product":
        n, k, es = case["n"], case["k"], 2 if case["dtype"] == "bf16" else 4
        rows = case["m"] if case["kind"] == "dense" else sum(_rows(case))
        weights = 1 if case["kind"] == "dense" else sum(r > 0 for r in _rows(case))
        return dict(bytes=(rows + weights * n) * k * (0.5 + 1 / 32) + rows * n * es * (2 if case["c"] else 1),
                    flops=2 * rows * n * k)
    m, e, k, es = case["m"], case["experts"], case["top_k"], 2 if case["dtype"] == "bf16" else 4
    if case["op"] == "route":
        return dict(bytes=m * e * es + m * k * 8 + 4 * e + (4 * e + 4 if case["loss"] else 0) + (4 * e if case["bias"] else 0)
                    + (m if case["mask"] else 0), flops=8 * m * e)
    return dict(bytes=2 * m * e * es + m * k * 8 + 8 * e, flops=10 * m * e)


# ---------------------------------------------------------------------------
# inputs
# ---------------------------------------------------------------------------

def _scale_byte(amax):
    """Exponent byte of the smallest power of two s with amax / s <= 6 (127 for an empty block)."""
    mant, ex = torch.frexp(amax)  # amax = mant * 2^ex, mant in [0.5, 1): 6 = 0.75 * 2^3
    e = torch.where(mant > 0.75, ex - 2, ex - 3) + 127
    return torch.where(amax == 0, torch.full_like(e, 127), e.clamp(0, 254)).to(torch.int64)


def _pack(b):
    """Exponent bytes along the last axis, four to a word, 127 past the end."""
    b = torch.nn.functional.pad(b, (0, (-b.shape[-1]) % 4), value=127).unflatten(-1, (-1, 4))
    return (b << torch.tensor([0, 8, 16, 24], device=b.device)).sum(-1).to(torch.int32)


def _quantise(x):
    """x [..., rows, K] in FP32 -> packed codes [..., rows, K / 2], scale words [..., K / 128, rows] and the values
    they stand for."""
    blocks = x.unflatten(-1, (-1, 32))
    byte = _scale_byte(blocks.abs().amax(-1))
    scale = torch.ldexp(torch.ones_like(blocks[..., 0]), byte - 127)
    v = (blocks.abs() / scale[..., None]).flatten(-2)
    code = ((v > 0.25).to(torch.uint8) + (v >= 0.75) + (v > 1.25) + (v >= 1.75) + (v > 2.5) + (v >= 3.5) + (v > 5)).to(torch.uint8)
    value = torch.tensor(E2M1, device=x.device)[code.int()].copysign(x)
    code += 8 * torch.signbit(x).to(torch.uint8)
    value = (value.unflatten(-1, (-1, 32)) * scale[..., None]).flatten(-2)
    return code[..., 0::2] + 16 * code[..., 1::2], _pack(byte).transpose(-1, -2), value


def _values(q, sf):
    """The FP32 values of packed codes [..., rows, K / 2] with scale words [..., K / 128, ld]."""
    code = torch.stack((q & 15, q >> 4), -1).flatten(-2).int()
    value = torch.tensor(E2M1 + [-v for v in E2M1], device=q.device)[code]
    words = sf[..., :q.shape[-2]].transpose(-1, -2).to(torch.int64)
    byte = ((words[..., None] >> torch.tensor([0, 8, 16, 24], device=q.device)) & 255).flatten(-2)
    return (value.unflatten(-1, (-1, 32)) * torch.exp2(byte.float() - 127)[..., None]).flatten(-2)


def _operand(x):
    """x [..., rows, K] as a quantised operand: codes and scale words whose rows are padded to 16 bytes."""
    q, words, _ = _quantise(x)
    rows = words.shape[-1]
    sf = torch.full((*words.shape[:-1], _padded(rows, 4)), 0x7F7F7F7F, dtype=torch.int32, device=x.device)
    sf[..., :rows] = words
    return q.contiguous(), sf


def _operands(gen, groups, rows, k):
    """`groups` random quantised operands, made one by one."""
    q, sf = zip(*[_operand(torch.randn(rows, k, device="cuda", generator=gen)) for _ in range(groups)])
    return torch.stack(q), torch.stack(sf)


def _logits(case, gen):
    m, e = case["m"], case["experts"]
    x = torch.randn(m, e, device="cuda", generator=gen) + 0.5 * torch.randn(e, device="cuda", generator=gen)
    if case["dead"]:
        x[:, torch.randperm(e, device="cuda", generator=gen)[:case["dead"]]] = -math.inf
    return x.to(DTYPES[case["dtype"]])


def _scores64(case, logits):
    x = logits.double()
    return torch.softmax(x, 1) if case["score"] == "softmax" else torch.sigmoid(x)


def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    op = case["op"]

    def empty(*shape, dtype):
        return torch.zeros(shape, dtype=dtype, device="cuda")

    if op == "cast":
        g, m, k, dt = case["groups"], case["m"], case["k"], DTYPES[case["dtype"]]
        lead = (g,) if g else ()
        x = torch.randn(*lead, m, k, device="cuda", generator=gen)
        x.mul_(torch.exp(torch.randn(*lead, m, 1, device="cuda", generator=gen)))
        masked_m = torch.randint(0, m + 1, (g,), device="cuda", generator=gen, dtype=torch.int32) if case["masked"] else None
        return dict(op=op, case=case, x=x.to(dt), masked_m=masked_m, q=empty(*lead, m, k // 2, dtype=torch.uint8),
                    sf=empty(*lead, k // 128, _padded(m, 4), dtype=torch.int32), y=empty(*lead, m, k, dtype=dt))

    if op == "product":
        m, n, k, dt = case["m"], case["n"], case["k"], DTYPES[case["dtype"]]
        state = dict(op=op, case=case, c=None)
        if case["kind"] == "dense":
            state["a"] = _operand(torch.randn(m, k, device="cuda", generator=gen))
            state["b"] = _operand(torch.randn(n, k, device="cuda", generator=gen))
            ld = _padded(n, 8)
            if case["c"]:
                state["c"] = torch.randn(m, ld, device="cuda", generator=gen).to(dt)[:, :n]
            state["d"] = empty(m, ld, dtype=dt)[:, :n]
            if own:
                import moe_grouped_gemm_tiles_amd as dg
                state["workspace"] = dg.alloc_mxfp4_workspace(m, n, k)
            return state
        rows = _rows(case)
        state["b"] = _operands(gen, case["groups"], n, k)
        if case["kind"] == "contiguous":
            index = torch.full((sum(_padded(r, 128) for r in rows),), -1, dtype=torch.int32)
            at = 0
            for g, r in enumerate(rows):
                index[at:at + r] = g
                at += _padded(r, 128)
            state["a"] = _operand(torch.randn(len(index), k, device="cuda", generator=gen))
            state["m_indices"] = index.cuda()
            state["d"] = empty(len(index), n, dtype=dt)
        else:
            state["a"] = _operands(gen, case["groups"], m, k)
            state["masked_m"] = torch.tensor(rows, dtype=torch.int32, device="cuda")
            state["expected_m"] = max(1, sum(rows) // len(rows))
            state["d"] = empty(case["groups"], m, n, dtype=dt)
        return state

    m, e, k = case["m"], case["experts"], case["top_k"]
    state = dict(op=op, case=case, logits=_logits(case, gen))
    if op == "route":
        state["bias"] = 0.05 * torch.randn(e, device="cuda", generator=gen) if case["bias"] else None
        state["mask"] = torch.rand(m, device="cuda", generator=gen) < 0.9 if case["mask"] else None
        state["ids"], state["weights"] = empty(m, k, dtype=torch.int32), empty(m, k, dtype=torch.float32)
        state["counts"] = empty(e, dtype=torch.int32)
        state["prob_sum"] = empty(e, dtype=torch.float32) if case["loss"] else None
        state["loss"] = empty(1, dtype=torch.float32) if case["loss"] else None
        if own:
            import moe_grouped_gemm_tiles_amd as dg
            state["workspace"] = dg.alloc_moe_router_workspace(m, e)
        return state
    p = _scores64(case, state["logits"])
    state["ids"] = torch.sort(state["logits"].double(), dim=1, descending=True, stable=True)[1][:, :k].to(torch.int32).contiguous()
    state["dweights"] = torch.randn(m, k, device="cuda", generator=gen)
    state["dloss"] = torch.rand(1, device="cuda", generator=gen) * m
    state["counts"] = torch.bincount(state["ids"].flatten().long(), minlength=e).to(torch.int32)
    state["prob_sum"] = (p / (p.sum(1, keepdim=True) + TINY)).sum(0).float()
    state["dlogits"] = torch.empty_like(state["logits"])
    return state


# ---------------------------------------------------------------------------
# one pass
# ---------------------------------------------------------------------------

def _plain_cast(st):
    q, sf, y = _quantise(st["x"].float())
    y = y.to(st["x"].dtype)
    if st["masked_m"] is not None:
        live = torch.arange(st["case"]["m"], device=q.device) < st["masked_m"][:, None]
        q, y, sf = q * live[..., None], torch.where(live[..., None], y, torch.zeros_like(y)), sf * live[:, None]
    return dict(q=q, sf=sf, y=y)


def _plain_product(st):
    case, dt = st["case"], st["d"].dtype
    if case["kind"] == "dense":
        d = _values(*st["a"]) @ _values(*st["b"]).t()
        return dict(d=(d if st["c"] is None else d + st["c"].float()).to(dt))
    d = torch.zeros_like(st["d"])
    (qa, sfa), (qb, sfb) = st["a"], st["b"]
    at = 0
    for g, r in enumerate(_rows(case)):
        b = _values(qb[g], sfb[g])
        if case["kind"] == "contiguous":
            d[at:at + r] = (_values(qa[at:at + r], sfa[:, at:at + r]) @ b.t()).to(dt)
            at += _padded(r, 128)
        else:
            d[g, :r] = (_values(qa[g, :r], sfa[g]) @ b.t()).to(dt)
    return dict(d=d)


def _plain_scores(case, logits):
    """Scores and their share of the row's sum, FP32; nothing for a row without a live expert."""
    x = logits.float()
    if case["score"] == "softmax":
        top = x.amax(1, keepdim=True)
        p = torch.exp(x - torch.where(torch.isinf(top), torch.zeros_like(top), top))
        p = p / p.sum(1, keepdim=True).clamp(min=1e-38)
        return p, p
    p = torch.sigmoid(x)
    return p, p / (p.sum(1, keepdim=True) + TINY)


def _plain_route(st):
    case, x = st["case"], st["logits"]
    e, k = case["experts"], case["top_k"]
    key = x.double()
    if st["bias"] is not None:
        key = torch.where(torch.isinf(key), key, _scores64(case, x) + st["bias"].double())
    key, order = torch.sort(key, dim=1, descending=True, stable=True)
    live = ~torch.isinf(key[:, :k])
    p, share = _plain_scores(case, x)
    if st["mask"] is not None:
        live = live & st["mask"][:, None]
        share = share * st["mask"][:, None]
    ids = torch.where(live, order[:, :k], torch.full_like(order[:, :k], -1))
    weights = torch.where(live, torch.gather(p, 1, order[:, :k]), torch.zeros_like(p[:, :k]))
    if case["normalize"]:
        weights = weights / (weights.sum(1, keepdim=True) + TINY)
    counts = (ids.flatten()[:, None] == torch.arange(e, device=x.device)).sum(0) if len(ids) * k * e < 1 << 22 \
        else torch.zeros(e + 1, dtype=torch.int64, device=x.device).index_add_(
            0, torch.where(live, ids, torch.full_like(ids, e)).flatten(), torch.ones_like(ids).flatten())[:e]
    out = dict(ids=ids.to(torch.int32), weights=weights, counts=counts.to(torch.int32))
    if case["loss"]:
        s = share.double().sum(0)
        loss = e * (counts.double() * s).sum() / (counts.sum() * s.sum()).clamp(min=1e-300)
        out.update(prob_sum=s.float(), loss=loss.float().view(1))
    return out


def _plain_route_grad(st):
    case, x = st["case"], st["logits"]
    ids = st["ids"].long()
    p, share = _plain_scores(case, x)
    chosen = torch.gather(p, 1, ids)
    dw = st["dweights"]
    if case["normalize"]:
        total = chosen.sum(1, keepdim=True) + TINY
        dw = (dw - (dw * chosen).sum(1, keepdim=True) / total) / total
    c, s = st["counts"].double(), st["prob_sum"].double()
    g = (st["dloss"].double() * case["experts"] * c / (c.sum() * s.sum())).float()
    if case["score"] == "softmax":
        dp = (g + torch.zeros_like(p)).scatter_add(1, ids, dw)
        dx = p * (dp - (p * dp).sum(1, keepdim=True))
    else:
        dp = ((g - (g * share).sum(1, keepdim=True)) / (p.sum(1, keepdim=True) + TINY)).scatter_add(1, ids, dw)
        dx = dp * p * torch.sigmoid(-x.float())
    return dict(dlogits=dx.to(x.dtype))


def _own(st):
    import moe_grouped_gemm_tiles_amd as dg
    case = st["case"]
    if st["op"] == "cast":
        dg.cast_to_mxfp4(st["x"], st["q"], st["sf"], y=st["y"], masked_m=st["masked_m"])
        return dict(q=st["q"], sf=st["sf"][..., :case["m"]], y=st["y"])
    if st["op"] == "product":
        if case["kind"] == "dense":
            dg.mxfp4_gemm_nt(st["a"], st["b"], st["d"], c=st["c"], workspace=st["workspace"])
        elif case["kind"] == "contiguous":
            dg.m_grouped_mxfp4_gemm_nt_contiguous(st["a"], st["b"], st["d"], st["m_indices"])
        else:
            dg.m_grouped_mxfp4_gemm_nt_masked(st["a"], st["b"], st["d"], st["masked_m"], st["expected_m"])
        return dict(d=st["d"])
    if st["op"] == "route":
        dg.moe_router(st["logits"], st["ids"], st["weights"], counts=st["counts"], prob_sum=st["prob_sum"], loss=st["loss"],
                      score=case["score"], bias=st["bias"], mask=st["mask"], normalize=case["normalize"],
                      workspace=st["workspace"])
        out = dict(ids=st["ids"], weights=st["weights"], counts=st["counts"])
        if case["loss"]:
            out.update(prob_sum=st["prob_sum"], loss=st["loss"])
        return out
    dg.moe_router_backward(st["logits"], st["ids"], st["dweights"], st["dlogits"], counts=st["counts"],
                           prob_sum=st["prob_sum"], dloss=st["dloss"], score=case["score"], normalize=case["normalize"])
    return dict(dlogits=st["dlogits"])


def run(state):
    if own:
        return _own(state)
    return {"cast": _plain_cast, "product": _plain_product, "route": _plain_route,
            "route_grad": _plain_route_grad}[state["op"]](state)


# ---------------------------------------------------------------------------
# the definition in FP64
# ---------------------------------------------------------------------------

def _exact_cast(st):
    """The nearest value on the grid of the block's scale, ties to the even one."""
    case = st["case"]
    x = st["x"].view(-1, case["m"], case["k"])
    y = torch.zeros(x.shape, dtype=torch.float64, device=x.device)
    for g in range(x.shape[0]):
        rows = case["m"] if st["masked_m"] is None else int(st["masked_m"][g])
        for at in range(0, rows, 4096):
            b = x[g, at:min(rows, at + 4096)].double().unflatten(-1, (-1, 32))
            amax = b.abs().amax(-1, keepdim=True)
            s = torch.exp2(torch.ceil(torch.log2(torch.where(amax == 0, 6.0, amax) / 6)).clamp(min=-127))
            v = b / s
            step = torch.where(v.abs() < 2, 0.5, torch.where(v.abs() < 4, 1.0, 2.0))
            y[g, at:min(rows, at + 4096)] = (torch.round(v / step) * step * s).flatten(-2)
    return dict(q=None, sf=None, y=y.view(st["y"].shape))


def _exact_values(q, sf, rows):
    lut = torch.tensor(E2M1, dtype=torch.float64, device=q.device)
    out = torch.empty(rows, 2 * q.shape[1], dtype=torch.float64, device=q.device)
    for half in (0, 1):
        c = ((q[:rows] >> (4 * half)) & 15).long()
        out[:, half::2] = lut[c & 7] * (1 - 2 * (c >> 3))
    for j in range(q.shape[1] // 16):
        e = ((sf[j // 4, :rows].long() >> (8 * (j % 4))) & 255).double() - 127
        out[:, 32 * j:32 * j + 32] *= torch.exp2(e)[:, None]
    return out


def _exact_product(st):
    case = st["case"]
    d = torch.zeros(st["d"].shape, dtype=torch.float64, device="cuda")
    (qa, sfa), (qb, sfb) = st["a"], st["b"]
    if case["kind"] == "dense":
        d[:] = _exact_values(qa, sfa, case["m"]) @ _exact_values(qb, sfb, case["n"]).t()
        if st["c"] is not None:
            d += st["c"].double()
        return dict(d=d)
    for g in range(case["groups"]):
        b = _exact_values(qb[g], sfb[g], case["n"]).t()
        if case["kind"] == "contiguous":
            at = torch.nonzero(st["m_indices"] == g).flatten()
            d[at] = _exact_values(qa[at], sfa[:, at].contiguous(), len(at)) @ b
        else:
            r = int(st["masked_m"][g])
            d[g, :r] = _exact_values(qa[g], sfa[g], r) @ b
    return dict(d=d)


def _exact_scores(case, x):
    e = torch.exp(x - x.amax(1, keepdim=True).nan_to_num(neginf=0.0)) if case["score"] == "softmax" else 1 / (1 + torch.exp(-x))
    total = e.sum(1, keepdim=True)
    return (e / total, e / total) if case["score"] == "softmax" else (e, e / (total + TINY))


def _exact_route(st):
    case, x = st["case"], st["logits"].double()
    m, e, k = case["m"], case["experts"], case["top_k"]
    p, share = _exact_scores(case, x)
    key = x if st["bias"] is None else torch.where(x == -math.inf, x, p + st["bias"].double())
    # expert j is chosen as number (experts ahead of it), if that is below k
    left = key.clone()
    weights = torch.zeros(m, k, dtype=torch.float64, device="cuda")
    counts = torch.zeros(e, dtype=torch.float64, device="cuda")
    rows = torch.arange(m, device="cuda")
    alive = torch.ones(m, dtype=torch.bool, device="cuda") if st["mask"] is None else st["mask"]
    for j in range(k):
        best = left.amax(1, keepdim=True)
        first = (left == best).to(torch.int8).argmax(1)
        ok = alive & (best[:, 0] > -math.inf)
        weights[:, j] = torch.where(ok, p[rows, first], 0.0)
        counts += torch.bincount(first[ok], minlength=e)
        left[rows, first] = -math.inf
    if case["normalize"]:
        weights /= weights.sum(1, keepdim=True) + TINY
    out = dict(ids=None, weights=weights, counts=None)
    if case["loss"]:
        s = share[alive].sum(0)
        some = counts.sum() > 0  # no loss in a batch whose rows are all padding
        out.update(prob_sum=s, loss=torch.where(some, e * (counts / counts.sum() * (s / s.sum())).sum(), 0.0).view(1))
    return out


def _exact_route_grad(st):
    case, x = st["case"], st["logits"].double()
    p, share = _exact_scores(case, x)
    c, s = st["counts"].double(), st["prob_sum"].double()
    g = st["dloss"].double() * case["experts"] * (c / c.sum()) / s.sum()
    dw = torch.zeros_like(p)
    chosen = torch.zeros_like(p)
    for j in range(case["top_k"]):
        at = st["ids"][:, j:j + 1].long()
        dw.scatter_(1, at, st["dweights"][:, j:j + 1].double())
        chosen.scatter_(1, at, 1.0)
    if case["normalize"]:
        total = (p * chosen).sum(1, keepdim=True) + TINY
        dw = chosen * (dw / total - (dw * p).sum(1, keepdim=True) / total ** 2)
    if case["score"] == "softmax":
        dp = g + dw
        return dict(dlogits=p * dp - p * (p * dp).sum(1, keepdim=True))
    dp = dw + (g - share @ g[:, None]) / (p.sum(1, keepdim=True) + TINY)
    return dict(dlogits=dp * p * (1 / (1 + torch.exp(x))))


def exact(case, seed):
    global own
    before, own = own, False
    try:
        state = prepare(case, seed)
    finally:
        own = before
    return {"cast": _exact_cast, "product": _exact_product, "route": _exact_route,
            "route_grad": _exact_route_grad}[state["op"]](state)
