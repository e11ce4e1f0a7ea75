"""examples/expert_layer.py: the operators together, step by step against 64-bit references of the cast operands.

Every product of the layer reads casts of what the step before it left, so each step is recomputed from the layer's
own intermediate results, with the tolerances of the single operators' tests.
"""
import importlib.util
import os

import pytest
import torch

import mxfp4_ref as ref

pytestmark = pytest.mark.gpu

PATH = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples", "expert_layer.py")
spec = importlib.util.spec_from_file_location("expert_layer", PATH)
example = importlib.util.module_from_spec(spec)
spec.loader.exec_module(example)


def check_product(got, a, b, offsets):
    """Rows [offsets[g], offsets[g + 1]) of got are cast(a) times cast(b[g]) transposed."""
    av = ref.cast(a.cpu())
    for g in range(b.shape[0]):
        s = slice(int(offsets[g]), int(offsets[g + 1]))
        want, tol = ref.product_bound(av[s], ref.cast(b[g].cpu()), True)
        assert bool(((got[s].cpu().double() - want).abs() <= tol).all()), g


@pytest.mark.parametrize("tokens,hidden,ffn,experts,k,score,groups,topk_groups", [
    (1, 256, 128, 8, 2, "softmax", 1, 1), (37, 264, 136, 8, 3, "sigmoid", 4, 2), (900, 512, 264, 4, 2, "sigmoid", 1, 1)])
def test_layer_step_by_step(tokens, hidden, ffn, experts, k, score, groups, topk_groups):
    layer = example.ExpertLayer(hidden, ffn, experts, k, score, groups, topk_groups)
    gen = torch.Generator(device="cuda").manual_seed(1)
    x = torch.randn(tokens, hidden, generator=gen, device="cuda").to(torch.bfloat16)
    grad = torch.randn(tokens, hidden, generator=gen, device="cuda").to(torch.bfloat16)
    out, saved = layer.forward(x)
    logits, route, plan, ab, y = saved
    p = ref.scores(logits.cpu(), score)
    want = ref.route_weights(p, route.indices.cpu(), True, 1.0)
    assert bool(((route.weights.cpu().double() - want).abs() <= 1e-6 * want).all())
    off, slots, tok = ref.plan(route.indices.cpu(), experts)
    assert torch.equal(plan.offsets.cpu(), off) and torch.equal(plan.slots.cpu(), slots) and torch.equal(plan.tokens.cpu(), tok)
    check_product(ab, x[plan.tokens.long()], layer.w1, off)
    a, b = ab.float().chunk(2, dim=1)
    check_product(y, (torch.nn.functional.silu(a) * b).to(torch.bfloat16), layer.w2, off)
    rows, w = y.cpu().double()[slots.long()], route.weights.cpu().double()[:, :, None]
    tol = k * 2.0 ** -23 * (w * rows.abs()).sum(1)
    want = (w * rows).sum(1)
    assert bool(((out.cpu().double() - want).abs() <= tol + 2.0 ** -8 * (want.abs() + tol)).all())
    dx, dlogits = layer.backward(grad, saved)
    assert dx.shape == x.shape and bool(torch.isfinite(dx).all())
    # the router's gradient against autograd in 64 bits, from the combination's own weights' gradient
    dw = (rows * grad.cpu().double()[:, None]).sum(2)
    leaf = logits.cpu().double().requires_grad_()
    wv = ref.route_weights(ref.scores(leaf, score), route.indices.cpu(), True, 1.0)
    want = torch.autograd.grad(wv, leaf, dw)[0]
    # dw's own rounding (hidden additions of 2^-23) and the gradient's 4e-6, of the magnitudes summed
    mag = (rows.abs() * grad.cpu().double().abs()[:, None]).sum(2)
    total = p.gather(1, route.indices.cpu().long()).sum(1, keepdim=True)
    tol = (hidden * 2.0 ** -23 + 4e-6) * mag.sum(1, keepdim=True) / total * p
    assert bool(((dlogits.cpu().double() - want).abs() <= tol + 1e-12).all())
