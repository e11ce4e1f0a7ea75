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


@pytest.mark.parametrize("tokens,hidden,ffn,experts,k,score", [(1, 256, 128, 8, 2, "softmax"), (37, 264, 136, 8, 3, "sigmoid"),
                                                               (900, 512, 264, 4, 2, "sigmoid")])
def test_layer_input_gradient_step_by_step(tokens, hidden, ffn, experts, k, score):
    """The gradient of x, each step against 64 bits of its own operands, and the layer's result against the steps'."""
    layer = example.ExpertLayer(hidden, ffn, experts, k, score)
    gen = torch.Generator(device="cuda").manual_seed(2)
    x = torch.randn(tokens, hidden, generator=gen, device="cuda").to(torch.bfloat16)
    grad = torch.randn(tokens, hidden, generator=gen, device="cuda").to(torch.bfloat16)
    _, saved = layer.forward(x)
    logits, route, plan, ab, y = saved
    dx, dlogits = layer.backward(grad, saved)
    mx, off = example.mx, plan.offsets.cpu()
    dy, _ = mx.moe_combine_backward(grad, y, plan.slots, route.weights)
    want = (route.weights.double()[:, :, None] * grad.double()[:, None]).flatten(0, 1)
    rows = dy.double()[plan.slots.flatten().long()]
    assert bool(((rows - want).abs() <= 2.0 ** -8 * want.abs()).all())
    dh = mx.matmul_mxfp4_grouped(mx.quantize_mxfp4_grouped(dy, plan.offsets), plan.offsets, layer.q2t)
    check_product(dh, dy, layer.w2.transpose(1, 2), off)
    leaf = ab.double().requires_grad_()
    a, b = leaf.chunk(2, dim=1)
    want = torch.autograd.grad(torch.nn.functional.silu(a) * b, leaf, dh.double())[0]
    a, b, d = ab.float().chunk(2, dim=1)[0], ab.float().chunk(2, dim=1)[1], dh.float()
    s = torch.sigmoid(a)
    dab = torch.cat((d * b * s * (1 + a * (1 - s)), d * a * s), dim=1).to(torch.bfloat16)  # as the layer computes it
    # fewer than 16 fp32 roundings of products below |d b| (1 + |a|) and |d a|, then one to bf16
    mag = torch.cat(((d * b).abs() * (1 + a.abs()), (d * a).abs()), dim=1).double()
    assert bool(((dab.double() - want).abs() <= 16 * 2.0 ** -23 * mag + 2.0 ** -8 * (want.abs() + 16 * 2.0 ** -23 * mag)).all())
    dr = mx.matmul_mxfp4_grouped(mx.quantize_mxfp4_grouped(dab, plan.offsets), plan.offsets, layer.q1t)
    check_product(dr, dab, layer.w1.transpose(1, 2), off)
    summed = mx.moe_combine(dr, plan.slots)
    parts = dr.double()[plan.slots.long()]
    tol = k * 2.0 ** -23 * parts.abs().sum(1)
    assert bool(((summed.double() - parts.sum(1)).abs() <= tol + 2.0 ** -8 * (parts.sum(1).abs() + tol)).all())
    want = summed.double() + dlogits.double() @ layer.router.double()
    tol = (experts + 2) * 2.0 ** -23 * (summed.double().abs() + dlogits.double().abs() @ layer.router.double().abs())
    assert bool(((dx.double() - want).abs() <= tol + 2.0 ** -8 * (want.abs() + tol)).all())


def test_layer_against_the_one_that_casts_nothing():
    """The example's own comparison.  A cast to levels spaced as E2M1's errs by about 0.12 of a normal block's rms: four
    casts on the way to the output (those of x and w1 count twice, in a and in b) make an error of at most 0.3 of
    its rms, a cosine of at least 0.95; the input gradient adds those of a and b again and two products, 0.4 and 0.92.  Held to
    0.9 and 0.85: an operand in the wrong place gives nearly 0."""
    layer = example.ExpertLayer(512, 256, 8, 2)
    gen = torch.Generator(device="cuda").manual_seed(3)
    x, grad = (torch.randn(600, 512, generator=gen, device="cuda").to(torch.bfloat16) for _ in range(2))
    got = example.compare(layer, x, grad)
    assert got["finite"] and got["out"] >= 0.9 and got["dx"] >= 0.85, got
