"""The operators around an expert layer, put together as a model uses them.

``python examples/decoder_block.py serve``  decode steps of a stack of expert
layers: residual addition + norm + FP8 cast, router, whole expert layer, captured
once in a HIP graph and replayed.

``python examples/decoder_block.py train``  training steps of a norm and an FP8
projection: fused norm, FP8 GEMMs forward and backward, FP32 weight gradient, the
norm's gradient, clipping by the global norm, update of the FP32 master weights.

Inputs and weights are random.
"""

import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

import moe_grouped_gemm_tiles_amd as dg  # noqa: E402

F8 = torch.float8_e4m3fn


def cast_rows(x):
    """(codes, transposed scales) of x [M, K]: a GEMM's a operand."""
    m, k = x.shape
    q = torch.empty(m, k, dtype=F8, device=x.device)
    sf = torch.empty(k // 128, dg.get_sf_aligned_size(m), device=x.device)
    return dg.per_token_cast_to_fp8(x, q, sf)


def cast_blocks(w):
    """(codes, block scales) of w [N, K]: a GEMM's b operand."""
    n, k = w.shape
    q = torch.empty(n, k, dtype=F8, device=w.device)
    sf = torch.empty((n + 127) // 128, k // 128, device=w.device)
    return dg.per_block_cast_to_fp8(w, q, sf)


class ExpertLayer:
    """Norm, router and gated experts of one layer, with the buffers of a batch of m tokens."""

    def __init__(self, m, hidden, inter, experts, top_k, dev):
        g = lambda *s: torch.randn(*s, device=dev)  # noqa: E731
        self.top_k, self.weight = top_k, (1 + 0.1 * g(hidden)).bfloat16()
        self.router = (g(experts, hidden) * hidden ** -0.5).bfloat16()
        pairs = [(cast_blocks((g(2 * inter, hidden) * hidden ** -0.5).bfloat16()),
                  cast_blocks((g(hidden, inter) * inter ** -0.5).bfloat16())) for _ in range(experts)]
        self.w13 = tuple(torch.stack([p[0][i] for p in pairs]) for i in (0, 1))
        self.w2 = tuple(torch.stack([p[1][i] for p in pairs]) for i in (0, 1))
        self.q = torch.empty(m, hidden, dtype=F8, device=dev)
        self.sf = torch.empty(hidden // 128, dg.get_sf_aligned_size(m), device=dev)
        self.y = torch.empty(m, hidden, dtype=torch.bfloat16, device=dev)
        self.out = torch.empty(m, hidden, dtype=torch.bfloat16, device=dev)
        self.workspace = dg.alloc_moe_workspace(m, top_k, inter, dev)

    def __call__(self, x, residual):
        """Adds x to the residual stream (in place) and returns the layer's output."""
        dg.add_rms_norm_cast_to_fp8(x, self.weight, 1e-6, self.q, self.sf, residual=residual, residual_out=residual,
                                    y=self.y)
        top, ids = torch.topk(self.y @ self.router.t(), self.top_k, dim=1)
        weights = torch.softmax(top.float(), dim=1)
        return dg.fp8_moe_few_tokens((self.q, self.sf), self.w13, self.w2, ids.int(), weights, self.out,
                                     workspace=self.workspace)


def serve(tokens=4, hidden=2048, inter=1024, experts=16, top_k=4, layers=3, steps=8, dev="cuda:0"):
    """Decode steps through the captured stack; returns the last residual stream and an eager run's."""
    torch.manual_seed(0)
    stack = [ExpertLayer(tokens, hidden, inter, experts, top_k, dev) for _ in range(layers)]
    x0 = torch.randn(tokens, hidden, device=dev).bfloat16()
    residual = torch.empty_like(x0)

    def step():
        x = x0
        residual.zero_()
        for layer in stack:
            x = layer(x, residual)
        residual.add_(x)

    step()
    eager = residual.clone()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    t = [torch.cuda.Event(enable_timing=True) for _ in range(2)]
    t[0].record()
    for _ in range(steps):
        graph.replay()
    t[1].record()
    torch.cuda.synchronize()
    print(f"{layers} expert layers, {tokens} tokens: {t[0].elapsed_time(t[1]) / steps * 1e3:.1f} us a step")
    return residual, eager


def train(tokens=512, hidden=1024, out=512, steps=20, lr=2.0, max_norm=1.0, dev="cuda:0"):
    """Training steps of out = FP8(norm(x + residual)) @ FP8(W).T against a fixed target; returns the losses."""
    torch.manual_seed(1)
    x, residual = (torch.randn(tokens, hidden, device=dev).bfloat16() for _ in range(2))
    target = torch.randn(tokens, out, device=dev) * 0.5
    master = {"w": torch.randn(out, hidden, device=dev) * hidden ** -0.5, "norm": torch.ones(hidden, device=dev)}
    grads = {k: torch.zeros_like(v) for k, v in master.items()}
    grad_list, total = dg.tensor_list(grads.values()), torch.empty(1, device=dev)
    like = lambda dt=torch.bfloat16: torch.empty(tokens, hidden, dtype=dt, device=dev)  # noqa: E731
    s, y, dx, q = like(), like(), like(), like(F8)
    sf = torch.empty(hidden // 128, dg.get_sf_aligned_size(tokens), device=dev)
    rstd = torch.empty(tokens, device=dev)
    workspace, clip_workspace = dg.alloc_rms_norm_backward_workspace(tokens, hidden, dev), dg.alloc_clip_workspace(dev)
    losses = []
    for step in range(steps):
        # forward
        dg.add_rms_norm_cast_to_fp8(x, master["norm"], 1e-6, q, sf, residual=residual, residual_out=s, y=y, rstd=rstd)
        w = master["w"].bfloat16()
        o = torch.empty(tokens, out, device=dev)
        dg.fp8_gemm_nt((q, sf), cast_blocks(w), o)
        diff = o - target
        losses.append(float(diff.square().mean()))
        do = (diff * (2.0 / diff.numel() * tokens)).bfloat16()
        # backward: gradient of the norm's output, of the projection, of the norm
        dy = torch.empty_like(s)
        dg.fp8_gemm_nt(cast_rows(do), cast_blocks(w.t().contiguous()), dy)
        grads["w"].zero_()
        dg.wgrad_fp8_gemm_nt(cast_rows(do.t().contiguous()), cast_blocks(y.t().contiguous()), grads["w"])
        dg.rms_norm_backward(dy, s, master["norm"], rstd, dx, grads["norm"], workspace=workspace)
        dg.clip_grad_norm(grad_list, max_norm, total, workspace=clip_workspace)
        for k, v in master.items():
            v.sub_(grads[k], alpha=lr / max_norm * 0.2)
    print(f"loss {losses[0]:.4f} -> {losses[-1]:.4f}, last gradient norm {float(total):.3f}")
    return losses


if __name__ == "__main__":
    for name in sys.argv[1:] or ("serve", "train"):
        {"serve": serve, "train": train}[name]()
