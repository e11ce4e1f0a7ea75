"""A mixture-of-experts MLP with MXFP4 experts: routing, plan, gathered cast, experts' products, combination, gradients.

    python examples/expert_layer.py [--tokens 4096] [--hidden 2048] [--ffn 1024] [--experts 64] [--top-k 8]

Each expert is SwiGLU: y = (silu(a) * b) W2^T with [a | b] = x W1^T.  Weights are cast once, both ways: along
their inputs for the forward products and transposed for the input gradients; backward gives the gradients of x and of
the router's logits (the package has no call for the experts' weight gradients).  Every step is one call of the
package; only the router's own product and the SwiGLU are plain torch.
"""
from __future__ import annotations

import argparse
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import mxfp8_block_scaled_04_gb300 as mx  # noqa: E402


def cast_experts(w: torch.Tensor):
    """w [E, N, K] bf16 as the experts' matrices: (along K, transposed along N), each held as one MXFP4Matrix."""
    E, N, K = w.shape
    casts = [mx.quantize_mxfp4(w[e], rowwise=True, colwise=True) for e in range(E)]

    def stack(ms, rows, cols):
        return mx.MXFP4Matrix(torch.stack([m.codes for m in ms]), torch.stack([m.scales for m in ms]), rows, cols)
    return stack([c.row for c in casts], N, K), stack([c.col for c in casts], K, N)


class ExpertLayer:
    def __init__(self, hidden: int, ffn: int, experts: int, top_k: int, score: str = "sigmoid", groups: int = 1,
                 topk_groups: int = 1, seed: int = 0, device: str = "cuda"):
        g = torch.Generator(device=device).manual_seed(seed)

        def init(*shape):
            return (torch.randn(*shape, generator=g, device=device) * shape[-1] ** -0.5).to(torch.bfloat16)
        self.experts, self.top_k = experts, top_k
        self.how = dict(score=score, renormalize=True, scale=1.0)
        self.groups = dict(groups=groups, topk_groups=topk_groups)
        self.bias = torch.zeros(experts, device=device)  # moved by the training loop towards an even load
        self.router = init(experts, hidden)
        self.w1, self.w2 = init(experts, 2 * ffn, hidden), init(experts, hidden, ffn)
        (self.q1, self.q1t), (self.q2, self.q2t) = cast_experts(self.w1), cast_experts(self.w2)

    def forward(self, x: torch.Tensor):
        """x [T, hidden] bf16 -> (output [T, hidden] bf16, what backward needs)."""
        logits = x.float() @ self.router.float().t()
        route = mx.moe_route(logits, self.top_k, bias=self.bias, **self.how, **self.groups)
        plan = mx.moe_plan(route.indices, self.experts)
        gathered = mx.quantize_mxfp4_grouped(x, plan.offsets, rows=plan.tokens)  # dropped choices would be rows of zeros
        ab = mx.matmul_mxfp4_grouped(gathered, plan.offsets, self.q1)
        a, b = ab.float().chunk(2, dim=1)
        h = (torch.nn.functional.silu(a) * b).to(torch.bfloat16)
        y = mx.matmul_mxfp4_grouped(mx.quantize_mxfp4_grouped(h, plan.offsets), plan.offsets, self.q2)
        out = mx.moe_combine(y, plan.slots, route.weights)
        return out, (logits, route, plan, ab, y)

    def backward(self, grad: torch.Tensor, saved):
        """grad [T, hidden] bf16 -> gradients of x (bf16) and of the router's logits (fp32)."""
        logits, route, plan, ab, y = saved
        dy, dweights = mx.moe_combine_backward(grad, y, plan.slots, route.weights)
        dlogits = mx.moe_route_backward(logits, route.indices, dweights, **self.how)
        dh = mx.matmul_mxfp4_grouped(mx.quantize_mxfp4_grouped(dy, plan.offsets), plan.offsets, self.q2t).float()
        a, b = ab.float().chunk(2, dim=1)
        s = torch.sigmoid(a)
        dab = torch.cat((dh * b * s * (1 + a * (1 - s)), dh * a * s), dim=1).to(torch.bfloat16)
        dx = mx.matmul_mxfp4_grouped(mx.quantize_mxfp4_grouped(dab, plan.offsets), plan.offsets, self.q1t)
        dx = mx.moe_combine(dx, plan.slots).float() + dlogits @ self.router.float()
        return dx.to(torch.bfloat16), dlogits


def plain_layer(layer: ExpertLayer, x: torch.Tensor, indices: torch.Tensor) -> torch.Tensor:
    """The same layer without any 4-bit cast, differentiable, for the experts that were chosen."""
    score = torch.sigmoid if layer.how["score"] == "sigmoid" else (lambda l: torch.softmax(l, 1))
    p = score(x.float() @ layer.router.float().t()).gather(1, indices.long())
    w = p / p.sum(1, keepdim=True)
    out = torch.zeros_like(x, dtype=torch.float32)
    for e in range(layer.experts):
        t, j = torch.where(indices == e)
        if t.numel():
            a, b = (x[t].float() @ layer.w1[e].float().t()).chunk(2, dim=1)
            y = (torch.nn.functional.silu(a) * b) @ layer.w2[e].float().t()
            out = out.index_add(0, t, w[t, j, None] * y)
    return out


def compare(layer: ExpertLayer, x: torch.Tensor, grad: torch.Tensor) -> dict:
    """Cosine of each result with the layer's that casts nothing to 4 bits."""
    out, saved = layer.forward(x)
    dx, dlogits = layer.backward(grad, saved)
    leaf = x.float().requires_grad_()
    want = plain_layer(layer, leaf, saved[1].indices)
    want_dx = torch.autograd.grad((want * grad.float()).sum(), leaf)[0]

    def cosine(u, v):
        return float(torch.nn.functional.cosine_similarity(u.detach().float().flatten(), v.detach().float().flatten(), dim=0))
    return {"out": cosine(out, want), "dx": cosine(dx, want_dx), "finite": bool(torch.isfinite(dlogits).all())}


def main() -> None:
    ap = argparse.ArgumentParser(description=__doc__, formatter_class=argparse.RawDescriptionHelpFormatter)
    for name, default in (("tokens", 4096), ("hidden", 2048), ("ffn", 1024), ("experts", 64), ("top-k", 8)):
        ap.add_argument("--" + name, type=int, default=default)
    a = ap.parse_args()
    layer = ExpertLayer(a.hidden, a.ffn, a.experts, a.top_k)
    x = torch.randn(a.tokens, a.hidden, device="cuda").to(torch.bfloat16)
    grad = torch.randn(a.tokens, a.hidden, device="cuda").to(torch.bfloat16)
    print("cosine with the layer that casts nothing to 4 bits:", compare(layer, x, grad))
    for what, call in (("forward", lambda: layer.forward(x)), ("forward + backward", lambda: layer.backward(grad, layer.forward(x)[1]))):
        for _ in range(3):
            call()
        start, end = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
        start.record()
        for _ in range(10):
            call()
        end.record()
        torch.cuda.synchronize()
        print(f"{what}: {start.elapsed_time(end) / 10 * 1e3:.0f} us for {a.tokens} tokens")


if __name__ == "__main__":
    main()
