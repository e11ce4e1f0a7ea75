"""A residual expert block, trained in MXFP8 and served from 4-bit weights: norms, routing, experts' products, gradients.

    python examples/expert_block.py [--tokens 4096] [--hidden 2048] [--ffn 1024] [--experts 64] [--top-k 8]

    x = norm(h)                            block_norm of the block before (or without one)
    y = combine(experts(x))                each expert SwiGLU: (silu(a) * b) W2^T with [a | b] = x W1^T
    h' = scale h + gate norm(y), x' = norm(h')    block_norm

``forward`` and ``backward`` run the experts' products from grouped MXFP8 casts (activations in E4M3, gradients in E5M2) and give
the gradients of every parameter: experts' weights, router, norm weights and gate.  ``serve`` runs a few tokens, uncast,
against the same weights in 4 bits.  The router's product and the SwiGLU are plain torch; every other step is one call of
the package.
"""
from __future__ import annotations

import argparse
import os
import sys
from typing import NamedTuple

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import mxfp8_block_scaled_04_gb300 as mx  # noqa: E402

BF16 = torch.bfloat16


def cast_experts8(w: torch.Tensor) -> mx.MXFP8Tensor:
    """w [E, N, K] bf16 in 8 bits, both ways: E groups of N rows."""
    E, N, K = w.shape
    return mx.quantize_grouped(w.view(E * N, K), torch.arange(E + 1, device=w.device) * N, mx.E4M3, swizzled=True)


def cast_experts4(w: torch.Tensor) -> mx.MXFP4Matrix:
    """The same in 4 bits along K."""
    casts = [mx.quantize_mxfp4(m).row for m in w]
    return mx.MXFP4Matrix(torch.stack([c.codes for c in casts]), torch.stack([c.scales for c in casts]), w.shape[1], w.shape[2])


def swiglu(ab: torch.Tensor) -> torch.Tensor:
    a, b = ab.float().chunk(2, dim=1)
    return (torch.nn.functional.silu(a) * b).to(BF16)


def swiglu_backward(ab: torch.Tensor, dh: torch.Tensor) -> torch.Tensor:
    a, b = ab.float().chunk(2, dim=1)
    s, d = torch.sigmoid(a), dh.float()
    return torch.cat((d * b * s * (1 + a * (1 - s)), d * a * s), dim=1).to(BF16)


class Saved(NamedTuple):
    x: torch.Tensor
    logits: torch.Tensor
    route: mx.MoERoute
    plan: mx.MoEPlan
    rows: mx.MXFP8Tensor    # cast of the gathered tokens
    ab: torch.Tensor
    inner: mx.MXFP8Tensor   # cast of the SwiGLU's output
    y: torch.Tensor         # the experts' rows
    out: torch.Tensor       # combined: the block's output before its norm
    h: torch.Tensor         # the stream behind the block


class ExpertBlock:
    def __init__(self, hidden: int, ffn: int, experts: int, top_k: int, scale: float = 1.0, seed: int = 0, device: str = "cuda"):
        g = torch.Generator(device=device).manual_seed(seed)

        def init(*shape):
            return (torch.randn(*shape, generator=g, device=device) * shape[-1] ** -0.5).to(BF16)
        self.experts, self.top_k, self.scale = experts, top_k, scale
        self.how = dict(score="sigmoid", renormalize=True, scale=1.0)
        self.router = init(experts, hidden)
        self.w1, self.w2 = init(experts, 2 * ffn, hidden), init(experts, hidden, ffn)
        self.pre = 1.0 + 0.1 * torch.randn(hidden, generator=g, device=device)   # weight of the next block's norm
        self.post = 1.0 + 0.1 * torch.randn(hidden, generator=g, device=device)  # of the norm behind this one
        self.gate = 0.5 + 0.1 * torch.randn(hidden, generator=g, device=device)
        self.q1, self.q2 = cast_experts8(self.w1), cast_experts8(self.w2)
        self.s1, self.s2 = cast_experts4(self.w1), cast_experts4(self.w2)

    def norm(self, y, h) -> mx.BlockNorm:
        return mx.block_norm(y, h, self.pre, self.post, self.gate, self.scale)

    def forward(self, x: torch.Tensor, h: torch.Tensor):
        """x [T, hidden] bf16 (the stream's norm), h [T, hidden]: (the next block's x and h, what backward needs)."""
        logits = x.float() @ self.router.float().t()
        route = mx.moe_route(logits, self.top_k, **self.how)
        plan = mx.moe_plan(route.indices, self.experts)
        rows = mx.quantize_grouped(x[plan.tokens.long()], plan.offsets, mx.E4M3, swizzled=True)
        ab = mx.matmul_mxfp8_grouped(rows, plan.offsets, self.q1)
        inner = mx.quantize_grouped(swiglu(ab), plan.offsets, mx.E4M3, swizzled=True)
        y = mx.matmul_mxfp8_grouped(inner, plan.offsets, self.q2)
        out = mx.moe_combine(y, plan.slots, route.weights)
        n = self.norm(out, h)
        return n.x, n.h, Saved(x, logits, route, plan, rows, ab, inner, y, out, n.h)

    def backward(self, grad_x, grad_h, s: Saved) -> dict:
        """Gradients of forward's results -> those of its inputs and of the parameters."""
        off = s.plan.offsets
        n = mx.block_norm_backward(grad_h, grad_x, s.out, s.h, self.pre, self.post, self.gate, self.scale)
        dy, dweights = mx.moe_combine_backward(n.y, s.y, s.plan.slots, s.route.weights)
        dlogits = mx.moe_route_backward(s.logits, s.route.indices, dweights, **self.how)
        qdy = mx.quantize_grouped(dy, off, mx.E5M2, swizzled=True)
        dw2 = mx.matmul_mxfp8_grouped_wgrad(qdy, s.inner, off)
        dab = swiglu_backward(s.ab, mx.matmul_mxfp8_grouped_dgrad(qdy, off, self.q2))
        qdab = mx.quantize_grouped(dab, off, mx.E5M2, swizzled=True)
        dw1 = mx.matmul_mxfp8_grouped_wgrad(qdab, s.rows, off)
        dx = mx.moe_combine(mx.matmul_mxfp8_grouped_dgrad(qdab, off, self.q1), s.plan.slots).float()
        dx = dx + dlogits @ self.router.float()
        return {"x": dx.to(BF16), "h": n.h, "w1": dw1, "w2": dw2, "router": dlogits.t() @ s.x.float(), "pre": n.pre_weight,
                "post": n.post_weight, "gate": n.gate}

    def serve(self, x: torch.Tensor, h: torch.Tensor) -> mx.BlockNorm:
        """The forward pass of a few tokens from 4-bit weights, without casting the tokens and without reading the host."""
        route = mx.moe_route(x.float() @ self.router.float().t(), self.top_k, **self.how)
        plan = mx.moe_plan(route.indices, self.experts)
        ab = mx.linear_mxfp4_grouped(x, plan.offsets, self.s1, rows=plan.tokens)
        y = mx.linear_mxfp4_grouped(swiglu(ab), plan.offsets, self.s2)
        return self.norm(mx.moe_combine(y, plan.slots, route.weights), h)


def plain_block(block: ExpertBlock, p: dict, x: torch.Tensor, h: torch.Tensor, indices: torch.Tensor):
    """The same block without any cast, differentiable in the parameters p (fp32), x and h, for the experts that were chosen."""
    score = torch.sigmoid(x @ p["router"].t()).gather(1, indices.long())
    w = score / score.sum(1, keepdim=True)
    out = torch.zeros_like(x)
    for e in range(block.experts):
        t, j = torch.where(indices == e)
        if t.numel():
            a, b = (x[t] @ p["w1"][e].t()).chunk(2, dim=1)
            out = out.index_add(0, t, w[t, j, None] * ((torch.nn.functional.silu(a) * b) @ p["w2"][e].t()))

    def rms(v):
        return v * torch.rsqrt((v * v).mean(1, keepdim=True) + 1e-6)
    h = block.scale * h + p["gate"] * rms(out) * p["post"]
    return rms(h) * p["pre"], h


def compare(block: ExpertBlock, x, h, grad_x, grad_h) -> dict:
    """Cosine of each result and gradient with the block's that casts nothing."""
    nx, nh, saved = block.forward(x, h)
    grads = block.backward(grad_x, grad_h, saved)
    leaves = {k: getattr(block, k).float().requires_grad_() for k in ("router", "w1", "w2", "pre", "post", "gate")}
    leaves |= {"x": x.float().requires_grad_(), "h": h.float().requires_grad_()}
    want_x, want_h = plain_block(block, leaves, leaves["x"], leaves["h"], saved.route.indices)
    loss = (want_x * grad_x.float()).sum() + (want_h * grad_h.float()).sum()
    want = dict(zip(leaves, torch.autograd.grad(loss, list(leaves.values()))))

    def cosine(u, v):
        return float(torch.nn.functional.cosine_similarity(u.detach().float().flatten(), v.detach().float().flatten(), dim=0))
    served = block.serve(x, h)
    return {"x": cosine(nx, want_x), "h": cosine(nh, want_h), "served x": cosine(served.x, want_x),
            **{f"grad {k}": cosine(grads[k], want[k]) for k in want}}


def main() -> None:
    ap = argparse.ArgumentParser(description=__doc__, formatter_class=argparse.RawDescriptionHelpFormatter)
    for name, default in (("tokens", 4096), ("hidden", 2048), ("ffn", 1024), ("experts", 64), ("top-k", 8)):
        ap.add_argument("--" + name, type=int, default=default)
    a = ap.parse_args()
    block = ExpertBlock(a.hidden, a.ffn, a.experts, a.top_k)
    h, gh, gx = (torch.randn(a.tokens, a.hidden, device="cuda").to(BF16) for _ in range(3))
    x = mx.block_norm(None, h, block.pre).x  # before the first block
    print("cosine with the block that casts nothing:")
    for k, v in compare(block, x, h, gx, gh).items():
        print(f"  {k:12s} {v:.4f}")
    few = slice(0, 16)
    for what, call in (("forward", lambda: block.forward(x, h)), ("forward + backward", lambda: block.backward(gx, gh, block.forward(x, h)[2])),
                       ("serving 16 tokens", lambda: block.serve(x[few], h[few]))):
        for _ in range(3):
            call()
        start, end = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
        start.record()
        for _ in range(10):
            call()
        end.record()
        torch.cuda.synchronize()
        print(f"{what}: {start.elapsed_time(end) / 10 * 1e3:.0f} us")


if __name__ == "__main__":
    main()
