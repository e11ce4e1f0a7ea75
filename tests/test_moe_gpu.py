"""Expert routing, plan and combination against the 64-bit reference (tests/mxfp4_ref.py).

Tolerances.  A score or weight is a chain of fewer than 512 + 16 fp32 operations with relative error
2^-24 each and expf within 2 ulps, all on positive terms: 1e-6 covers logits up to |l| = 8 (the argument's
rounding adds |l| 2^-24).  Gradients subtract: their error is held to 4e-6 of the sum of the magnitudes.
Combination: k fp32 additions (k 2^-23 of sum |w y|) and half a unit of bf16's 8 bits.
"""
import pytest
import torch

import mxfp4_ref as ref
import mxfp8_block_scaled_04_gb300 as mx

pytestmark = pytest.mark.gpu

BF16, F32 = torch.bfloat16, torch.float32


def draw_logits(T, E, dtype, seed, bias, score, k, groups, topk_groups):
    """Logits whose choices are wider apart than fp32 scores resolve: rows whose order of keys (or of group ranks)
    is closer than 1e-5 anywhere are drawn again."""
    g = torch.Generator().manual_seed(seed)
    b = torch.randn(E, generator=g) * 0.1 if bias else None
    l = (torch.randn(T, E, generator=g) * 1.5).to(dtype)
    for _ in range(200):
        key = l.double() if b is None else ref.scores(l, score) + b.double()
        near = (key.sort(1).values.diff(dim=1) < 1e-5)
        if b is None:
            near &= key.sort(1).values.diff(dim=1) != 0  # equal logits are ties, by index
        near = near.any(1) if E <= 64 else (near[:, -2 * k * groups // topk_groups - 8:]).any(1)
        if groups > topk_groups:
            top = key.view(T, groups, -1).sort(2, descending=True).values
            rank = top[:, :, :2].sum(2) if b is not None else top[:, :, 0]
            d = rank.sort(1).values.diff(dim=1)
            near |= ((d < 1e-5) & ((d != 0) | (b is not None))).any(1)
        if not near.any():
            break
        l[near] = (torch.randn(int(near.sum()), E, generator=g) * 1.5).to(dtype)
    return l, b


CASES = [  # T, E, k, groups, topk_groups
    (1, 1, 1, 1, 1), (1, 8, 2, 1, 1), (17, 64, 8, 1, 1), (5, 64, 6, 8, 3), (9, 96, 4, 4, 2), (33, 160, 6, 8, 3),
    (12, 256, 8, 8, 4), (3, 512, 32, 1, 1), (4, 512, 8, 16, 4), (6, 60, 4, 60, 5), (7, 20, 3, 10, 2), (2, 33, 33 - 1, 1, 1)]


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("bias", [False, True])
@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("T,E,k,groups,topk_groups", CASES)
def test_route_and_gradient(T, E, k, groups, topk_groups, dtype, bias, score):
    l, b = draw_logits(T, E, dtype, E + k, bias, score, k, groups, topk_groups)
    p = ref.scores(l, score)
    key = l.double() if b is None else p + b.double()
    idx = ref.choose(key, k, groups, topk_groups, two=b is not None)
    for renorm in (True, False):
        r = mx.moe_route(l.cuda(), k, score, None if b is None else b.cuda(), groups, topk_groups, renorm, 2.5)
        assert torch.equal(r.indices.cpu(), idx)
        want = ref.route_weights(p, idx, renorm, 2.5)
        assert bool(((r.weights.cpu().double() - want).abs() <= 1e-6 * want.abs()).all())
        # gradient against autograd in 64 bits
        g = torch.Generator().manual_seed(7)
        dw = torch.randn(T, k, generator=g)
        leaf = l.double().requires_grad_()
        w = ref.route_weights(ref.scores(leaf, score), idx, renorm, 2.5)
        want = torch.autograd.grad(w, leaf, dw.double())[0]
        got = mx.moe_route_backward(l.cuda(), r.indices, dw.cuda(), score, renorm, 2.5).cpu()
        assert got.dtype == dtype
        total = p.gather(1, idx.long()).sum(1, keepdim=True) if renorm else 1.0
        mag = 2.5 * dw.abs().double().sum(1, keepdim=True) / total * p
        tol = 4e-6 * mag + (2.0 ** -8 * want.abs() if dtype == BF16 else 0.0)
        assert bool(((got.double() - want).abs() <= tol + 1e-12).all())


def test_route_gradient_against_differences():
    """Central differences of the weights themselves (64-bit reference of the same formula), h = 1e-4."""
    l, _ = draw_logits(6, 24, F32, 1, False, "softmax", 4, 1, 1)
    dw = torch.randn(6, 4, generator=torch.Generator().manual_seed(2))
    for score in ("softmax", "sigmoid"):
        for renorm in (True, False):
            r = mx.moe_route(l.cuda(), 4, score, renormalize=renorm)
            got = mx.moe_route_backward(l.cuda(), r.indices, dw.cuda(), score, renorm).cpu().double()
            idx = r.indices.cpu()
            for t, e in ((0, int(idx[0, 1])), (3, 5), (5, 23)):
                f = []
                for h in (1e-4, -1e-4):
                    m = l.double().clone()
                    m[t, e] += h
                    f.append((ref.route_weights(ref.scores(m, score), idx, renorm, 1.0) * dw.double()).sum())
                slope = (f[0] - f[1]) / 2e-4
                # differences: O(h^2) times a third derivative below 10 |dw|, and 1e-12 of rounding over h
                assert abs(slope - got[t, e]) <= 1e-6 * dw[t].abs().sum() + 1e-7


def test_route_ties_masks_and_nan():
    inf = float("inf")
    l = torch.zeros(6, 8)
    l[1] = torch.tensor([1.0, 3, 3, 2, 3, -1, 0, 3])
    l[2] = -inf                                   # nothing left
    l[3] = torch.tensor([-inf, -inf, 5, -inf, -inf, 1, -inf, -inf])
    l[4] = torch.finfo(F32).min                   # masked with the lowest value
    l[4, 6] = 1.0
    l[5] = torch.tensor([-0.0, 0.0, -1, -1, -1, -1, -1, -1])
    r = mx.moe_route(l.cuda(), 3)
    idx, w = r.indices.cpu(), r.weights.cpu()
    assert idx.tolist() == [[0, 1, 2], [1, 2, 4], [0, 1, 2], [2, 5, 0], [6, 0, 1], [0, 1, 2]]
    assert torch.equal(w[2], torch.zeros(3))
    assert torch.equal(w[0], torch.full((3,), 1 / 3)) and float(w[3, 2]) == 0 and w[4].tolist() == [1.0, 0.0, 0.0]
    d = mx.moe_route_backward(l.cuda(), r.indices, torch.ones(6, 3).cuda(), renormalize=True)
    assert bool((d[2] == 0).all()) and bool(torch.isfinite(d).all())
    # NaN ranks last and reaches the weights; indices stay in range
    l[0, 3] = float("nan")
    r = mx.moe_route(l.cuda(), 8)
    assert r.indices[0].tolist() == [0, 1, 2, 4, 5, 6, 7, 3]
    assert bool(torch.isnan(r.weights[0]).all()) and bool(torch.isfinite(r.weights[1]).all())
    # sigmoid of very negative logits: scores 0, weights 0
    r = mx.moe_route(torch.full((1, 8), -200.0).cuda(), 2, "sigmoid")
    assert r.indices.tolist() == [[0, 1]] and r.weights.tolist() == [[0.0, 0.0]]


@pytest.mark.parametrize("E", [8, 32, 60, 256, 512])
@pytest.mark.parametrize("bias", [False, True])
def test_route_many_equal_keys(E, bias):
    """Logits of a few values only: ties within and across lanes, all the way down the order."""
    g = torch.Generator().manual_seed(E)
    l = torch.randint(-2, 3, (300, E), generator=g).float()
    b = (torch.randint(0, 2, (E,), generator=g).float() * 0.5) if bias else None
    k = min(E, 32)
    r = mx.moe_route(l.cuda(), k, "sigmoid", None if b is None else b.cuda())
    key = l.double() if b is None else torch.sigmoid(l.double()).float().double() + b.double()
    # sigmoid(-x) + 0.5 and sigmoid(x) are never closer than 1e-3 on these values: equal keys are equal logits and biases
    assert torch.equal(r.indices.cpu().long(), key.sort(dim=1, descending=True, stable=True).indices[:, :k])


def test_route_extreme_logits():
    """Infinite, huge and tiny logits among others: scores 0, 1 and subnormal, in every lane."""
    inf = float("inf")
    l = torch.randn(64, 64, generator=torch.Generator().manual_seed(3))
    for i, v in enumerate((inf, -inf, 100.0, -100.0, -88.0, -87.5, -103.0, 3e38, -3e38, 0.0)):
        l[i * 3, (i * 7) % 64] = v
    want = torch.sigmoid(l.double())
    r = mx.moe_route(l.cuda(), 16, "sigmoid", renormalize=False)
    assert torch.equal(r.indices.cpu().long(), l.sort(dim=1, descending=True, stable=True).indices[:, :16])
    w = want.gather(1, r.indices.cpu().long())
    assert bool(((r.weights.cpu().double() - w).abs() <= 1e-6 * w + 1.5e-45).all())
    # scores near the end of fp32: exp(-l) overflows beyond l = -88.72, where the score, below 2^-127, becomes 0; before
    # that the argument's rounding adds |l| 2^-24 and a subnormal score half its spacing
    low = torch.full((4, 64), -200.0)
    low[:, 1], low[:, 9] = -88.2, -95.0
    r = mx.moe_route(low.cuda(), 2, "sigmoid", renormalize=False)
    assert r.indices.tolist() == [[1, 9]] * 4
    w = torch.sigmoid(low.double()).gather(1, r.indices.cpu().long())
    got = r.weights.cpu().double()
    assert bool(((got - w).abs()[:, 0] <= (1e-6 + 88.2 * 2.0 ** -24) * w[:, 0] + 1.5e-45).all()) and bool((w[:, 0] > 0).all())
    assert bool(((got - w).abs()[:, 1] <= 2.0 ** -127).all())


def test_route_strided_logits_and_many_tokens():
    l, _ = draw_logits(3000, 64, F32, 4, False, "softmax", 8, 1, 1)
    big = torch.zeros(3000, 72)
    big[:, 3:67] = l
    got = mx.moe_route(big.cuda()[:, 3:67], 8)
    want = mx.moe_route(l.cuda(), 8)
    assert torch.equal(got.indices, want.indices) and torch.equal(got.weights, want.weights)
    assert torch.equal(got.indices.cpu().long(), l.sort(dim=1, descending=True, stable=True).indices[:, :8])
    dw = torch.randn(3000, 8).cuda()
    assert torch.equal(mx.moe_route_backward(big.cuda()[:, 3:67], got.indices, dw), mx.moe_route_backward(l.cuda(), got.indices, dw))


@pytest.mark.parametrize("T,k,E", [(0, 2, 4), (1, 1, 1), (16, 8, 64), (100, 3, 7), (513, 8, 512), (5000, 2, 33), (30000, 8, 160)])
def test_plan(T, k, E):
    g = torch.Generator().manual_seed(T + E)
    idx = torch.randint(0, E, (T, k), generator=g, dtype=torch.int32)
    p = mx.moe_plan(idx.cuda(), E)
    off, slots, tokens = ref.plan(idx, E)
    assert torch.equal(p.offsets.cpu(), off) and torch.equal(p.slots.cpu(), slots) and torch.equal(p.tokens.cpu(), tokens)


@pytest.mark.parametrize("T", [3, 900])
def test_plan_dropped_choices(T):
    """Indices outside [0, E) have no row; their slots name the rows left over, and the gradient there is zero."""
    g = torch.Generator().manual_seed(T)
    idx = torch.randint(-2, 12, (T, 4), generator=g, dtype=torch.int32)
    idx[0] = torch.tensor([-1, 2 ** 31 - 1, -2 ** 31, 10], dtype=torch.int32)
    p = mx.moe_plan(idx.cuda(), 10)
    off, slots, tokens = ref.plan(idx, 10)
    assert torch.equal(p.offsets.cpu(), off) and torch.equal(p.slots.cpu(), slots) and torch.equal(p.tokens.cpu(), tokens)
    y = torch.randn(T * 4, 16, generator=g).to(BF16)
    d = torch.randn(T, 16, generator=g).to(BF16)
    dy, dw = mx.moe_combine_backward(d.cuda(), y.cuda(), p.slots, torch.ones(T, 4).cuda())
    want = torch.zeros(T * 4, 16, dtype=BF16)
    want[:int(off[-1])] = d[tokens[:int(off[-1])].long()]
    assert torch.equal(dy.cpu(), want)
    assert bool((dw.cpu()[slots < 0] == 0).all())
    out = mx.moe_combine(y.cuda(), p.slots)
    assert bool((out[0] == 0).all())


@pytest.mark.parametrize("T,k,H", [(0, 2, 8), (1, 1, 8), (5, 3, 24), (16, 8, 7168), (40, 32, 1032), (700, 2, 264), (9, 9, 2048)])
@pytest.mark.parametrize("weighted", [True, False])
def test_combine_and_gradient(T, k, H, weighted):
    g = torch.Generator().manual_seed(T + H)
    R = T * k
    slots = torch.randperm(R, generator=g).to(torch.int32).view(T, k)
    y, d = torch.randn(R, H, generator=g).to(BF16), torch.randn(T, H, generator=g).to(BF16)
    w = torch.randn(T, k, generator=g) if weighted else None
    wd = w.double() if weighted else torch.ones(T, k, dtype=torch.float64)
    out = mx.moe_combine(y.cuda(), slots.cuda(), w.cuda() if weighted else None).cpu().double()
    rows = y.double()[slots.long()]
    want, mag = (wd[:, :, None] * rows).sum(1), (wd.abs()[:, :, None] * rows.abs()).sum(1)
    tol = k * 2.0 ** -23 * mag
    assert bool(((out - want).abs() <= tol + 2.0 ** -8 * (want.abs() + tol)).all())
    dy, dw = mx.moe_combine_backward(d.cuda(), y.cuda(), slots.cuda(), w.cuda() if weighted else None)
    want = (rows * d.double()[:, None]).sum(2)
    mag = (rows.abs() * d.double().abs()[:, None]).sum(2)
    assert bool(((dw.cpu().double() - want).abs() <= H * 2.0 ** -23 * mag).all())
    want = torch.zeros(R, H, dtype=torch.float64)
    want[slots.flatten().long()] = (wd[:, :, None] * d.double()[:, None]).reshape(-1, H)
    assert bool(((dy.cpu().double() - want).abs() <= 2.0 ** -8 * want.abs()).all())
    # the same bits again
    dy2, dw2 = mx.moe_combine_backward(d.cuda(), y.cuda(), slots.cuda(), w.cuda() if weighted else None)
    assert torch.equal(dy, dy2) and torch.equal(dw, dw2)


def test_combine_gradient_against_differences():
    """out is linear in w and y: a difference over h is the derivative up to 64-bit rounding."""
    g = torch.Generator().manual_seed(1)
    y, d, w = torch.randn(6, 16, generator=g).to(BF16), torch.randn(3, 16, generator=g).to(BF16), torch.randn(3, 2, generator=g)
    slots = torch.tensor([[4, 0], [1, 5], [3, 2]], dtype=torch.int32)
    dy, dw = mx.moe_combine_backward(d.cuda(), y.cuda(), slots.cuda(), w.cuda())

    def loss(yv, wv):
        return ((wv[:, :, None] * yv[slots.long()]).sum(1) * d.double()).sum()
    yv, wv, h = y.double(), w.double(), 0.5
    for t, j in ((0, 0), (2, 1)):
        m = wv.clone()
        m[t, j] += h
        slope = (loss(yv, m) - loss(yv, wv)) / h
        assert abs(slope - float(dw[t, j])) <= 16 * 2.0 ** -23 * (yv[slots[t, j]].abs() @ d[t].double().abs()) + 1e-12
    m = yv.clone()
    m[5, 7] += h
    slope = (loss(m, wv) - loss(yv, wv)) / h
    assert abs(slope - float(dy[5, 7])) <= 2.0 ** -8 * abs(slope)


@pytest.mark.parametrize("E", [8, 40, 256])
def test_route_nan_among_masked_logits(E):
    """A NaN makes the sum of its row's softmax NaN whatever the other logits are, -inf alone included; a row of -inf only
    keeps its zeros."""
    inf, nan = float("inf"), float("nan")
    l = torch.full((3, E), -inf)
    l[0, 3] = nan
    l[1, E - 1], l[1, 0] = nan, 1.0
    for renorm in (False, True):
        r = mx.moe_route(l.cuda(), 4, renormalize=renorm)
        assert r.indices[0].tolist() == [0, 1, 2, 4] and int(r.indices[1, 0]) == 0
        assert bool(torch.isnan(r.weights[:2]).all()) and bool((r.weights[2] == 0).all())
        d = mx.moe_route_backward(l.cuda(), r.indices, torch.ones(3, 4).cuda(), renormalize=renorm)
        assert bool(torch.isnan(d[:2]).all()) and bool((d[2] == 0).all())
