"""An expert layer with 4-bit operands behind its router, put together as a model uses them.

``python examples/mxfp4_experts.py serve``  a decode step, captured once in a HIP graph and replayed: norm,
router (choice, weights, rows per expert), the chosen rows laid out by expert, 4-bit cast, both masked
products, the weighted sum over a token's experts.

``python examples/mxfp4_experts.py train``  one training step of router and experts' first weights: balance
loss and straight-through 4-bit values forward, their gradients backward.

Inputs and weights are random.
"""

import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

import moe_grouped_gemm_tiles_amd as dg  # noqa: E402


def quantised(x, masked_m=None):
    """x [.., rows, K] as a product's operand."""
    *lead, rows, k = x.shape
    q = torch.empty(*lead, rows, k // 2, dtype=torch.uint8, device=x.device)
    sf = torch.empty(*lead, k // 128, dg.get_sf_aligned_size(rows), dtype=torch.int32, device=x.device)
    return dg.cast_to_mxfp4(x, q, sf, masked_m=masked_m)


class Experts:
    """Norm, router and gated 4-bit experts of one layer for batches of m tokens."""

    def __init__(self, m, hidden, inter, experts, top_k, dev):
        g = lambda *s: torch.randn(*s, device=dev)  # noqa: E731
        self.m, self.experts, self.top_k, self.inter = m, experts, top_k, inter
        self.norm = (1 + 0.1 * g(hidden)).bfloat16()
        self.router = (g(experts, hidden) * hidden ** -0.5).bfloat16()
        self.bias = 0.02 * g(experts)
        self.w13 = quantised((g(experts, 2 * inter, hidden) * hidden ** -0.5).bfloat16())
        self.w2 = quantised((g(experts, hidden, inter) * inter ** -0.5).bfloat16())
        empty = lambda *s, dt=torch.bfloat16: torch.empty(*s, dtype=dt, device=dev)  # noqa: E731
        self.y, self.q8 = empty(m, hidden), empty(m, hidden, dt=torch.uint8)
        self.sf8 = empty(hidden // 128, dg.get_sf_aligned_size(m), dt=torch.float32)
        self.ids, self.weights = empty(m, top_k, dt=torch.int32), empty(m, top_k, dt=torch.float32)
        self.counts = empty(experts, dt=torch.int32)
        self.workspace = dg.alloc_moe_router_workspace(m, experts, dev)
        # rows of each expert (a token chooses one once, so m at most), and one row for slots without an expert
        self.rows = torch.zeros(experts * m + 1, hidden, dtype=torch.bfloat16, device=dev)
        self.hid, self.out = empty(experts, m, 2 * inter), torch.zeros(experts * m + 1, hidden, dtype=torch.bfloat16, device=dev)
        self.order = torch.arange(experts, device=dev, dtype=torch.int32)

    def __call__(self, x):
        m, e, k = self.m, self.experts, self.top_k
        dg.add_rms_norm_cast_to_fp8(x, self.norm, 1e-6, self.q8, self.sf8, y=self.y)
        dg.moe_router(self.y @ self.router.t(), self.ids, self.weights, self.counts, score="sigmoid", bias=self.bias,
                      workspace=self.workspace)
        # row of each (token, slot): its expert's block, in the order of the pairs
        flat = self.ids.view(-1)
        mine = flat[:, None] == self.order
        rank = (mine.int().cumsum(0) * mine).sum(1) - 1
        row = torch.where(flat >= 0, flat * m + rank, e * m).long()
        self.rows.index_copy_(0, row, self.y.repeat_interleave(k, 0))
        a = quantised(self.rows[:-1].view(e, m, -1), self.counts)
        dg.m_grouped_mxfp4_gemm_nt_masked(a, self.w13, self.hid, self.counts)
        act = (torch.nn.functional.silu(self.hid[..., :self.inter].float()) * self.hid[..., self.inter:]).bfloat16()
        dg.m_grouped_mxfp4_gemm_nt_masked(quantised(act, self.counts), self.w2, self.out[:-1].view(e, m, -1), self.counts)
        return (self.out[row].view(m, k, -1).float() * self.weights[..., None]).sum(1).bfloat16()


def serve(tokens=16, hidden=2048, inter=1024, experts=32, top_k=4, steps=8, dev="cuda:0"):
    """Returns (outputs of `steps` replays with inputs of their own, eager outputs of the same inputs, the layer)."""
    torch.manual_seed(0)
    layer = Experts(tokens, hidden, inter, experts, top_k, dev)
    inputs = [torch.randn(tokens, hidden, device=dev).bfloat16() for _ in range(steps)]
    eager = [layer(x).clone() for x in inputs]
    x = inputs[0].clone()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = layer(x)
    replayed = []
    t = [torch.cuda.Event(enable_timing=True) for _ in range(2)]
    t[0].record()
    for src in inputs:
        x.copy_(src)
        graph.replay()
        replayed.append(out.clone())
    t[1].record()
    torch.cuda.synchronize()
    print(f"{tokens} tokens through {top_k} of {experts} 4-bit experts: {t[0].elapsed_time(t[1]) / steps * 1e3:.1f} us a step")
    return replayed, eager, layer


def train(tokens=512, hidden=1024, experts=16, top_k=2, alpha=0.01, dev="cuda:0"):
    """One step: returns the tensors and gradients of the router (its logits' and weight's) and of a 4-bit product's weight."""
    torch.manual_seed(1)
    x = torch.randn(tokens, hidden, device=dev).bfloat16()
    wr = torch.randn(experts, hidden, device=dev) * hidden ** -0.5
    logits = x.float() @ wr.t()
    ids, w = torch.empty(tokens, top_k, dtype=torch.int32, device=dev), torch.empty(tokens, top_k, device=dev)
    counts, prob_sum = torch.empty(experts, dtype=torch.int32, device=dev), torch.empty(experts, device=dev)
    loss = torch.empty(1, device=dev)
    dg.moe_router(logits, ids, w, counts, prob_sum, loss)
    dw = torch.randn(tokens, top_k, device=dev)  # what came back from the experts' outputs
    dlogits = torch.empty_like(logits)
    dg.moe_router_backward(logits, ids, dw, dlogits, counts, prob_sum, torch.full((1,), alpha, device=dev))
    # a projection of the tokens of expert 0 in 4 bits, straight through: out = Q(x) Q(w)^T, dw += Q(dout^T) Q(x^T)^T
    weight = (torch.randn(256, hidden, device=dev) * hidden ** -0.5)
    values = torch.empty_like(weight)
    wq = (torch.empty(256, hidden // 2, dtype=torch.uint8, device=dev),
          torch.empty(hidden // 128, 256, dtype=torch.int32, device=dev))
    dg.cast_to_mxfp4(weight, *wq, y=values)
    out = torch.empty(tokens, 256, device=dev)
    dg.mxfp4_gemm_nt(quantised(x), wq, out)
    dout = torch.randn(tokens, 256, device=dev).bfloat16()
    dweight = torch.zeros(256, hidden, device=dev)
    dg.mxfp4_gemm_nt(quantised(dout.t().contiguous()), quantised(x.t().contiguous()), dweight, c=dweight)
    print(f"balance loss {float(loss):.3f}, gradient norms {float(dlogits.norm()):.4f} and {float(dweight.norm()):.1f}")
    return dict(x=x, logits=logits, ids=ids, dw=dw, alpha=alpha, dlogits=dlogits, loss=loss, dout=dout, dweight=dweight,
                out=out, values=values)


if __name__ == "__main__":
    for name in sys.argv[1:] or ("serve", "train"):
        {"serve": serve, "train": train}[name]()
