"""The norms around a block with gate and residual scale, and their gradients, against 64-bit formulas, autograd and differences.

Roundings that the tolerances count: a row's sum passes at most 32 additions in a thread and 10 in two trees, each off by
2^-24 of what it adds up; rsqrtf is good to 2 units of the last of 24 bits; a dozen more products follow.  64 * 2^-24
= 2^-18 of the magnitudes covers them.  A sum over tokens adds a CTA's rows, then the CTAs in eight
strands or more.  Outputs in bf16 are off by half a unit of the last of 8 bits, 2^-8.
"""
import math

import pytest
import torch

import mxfp8_block_scaled_04_gb300 as mx

pytestmark = pytest.mark.gpu

BF16, F32 = torch.bfloat16, torch.float32
HALF = {BF16: 2.0 ** -8, F32: 2.0 ** -24}
EPS = 1e-6


def draw(T, H, dtype, seed, spread=0.5):
    g = torch.Generator(device="cuda").manual_seed(seed)
    x = torch.randn(T, H, generator=g, device="cuda") * torch.exp(spread * torch.randn(T, 1, generator=g, device="cuda"))
    return x.to(dtype)


def vec(H, seed, mean=1.0):
    return mean + 0.3 * torch.randn(H, generator=torch.Generator(device="cuda").manual_seed(seed), device="cuda")


def rms(v, eps):
    return v / torch.sqrt((v * v).mean(1, keepdim=True) + eps)


def gate_of(kind, T, H):
    return {"none": None, "channel": vec(H, 7, 0.4), "token": vec(T, 8, 0.4)[:, None].contiguous()}[kind]


def behind(y, post, gate, eps):
    u = y if post is None else rms(y, eps) * post
    return u if gate is None else u * gate


def inside(got, want, tol, what):
    bad = ~((got.double() - want).abs() <= tol)
    assert not bool(bad.any()), (what, int(bad.sum()), float((got.double() - want).abs().max()), float(want.abs().max()))


def d(t):
    return None if t is None else t.double()


def check_forward(T, H, yt, ht, post, kind, scale, eps=EPS, y=None, h=None):
    y = draw(T, H, yt, 1) if y is None else y
    h = draw(T, H, ht, 2) if h is None else h
    w1, w2, gate = vec(H, 3) if post else None, vec(H, 4), gate_of(kind, T, H)
    r = mx.block_norm(y, h, w2, w1, gate, scale, eps)
    assert r.h.dtype == ht and r.x.dtype == BF16 and r.h.shape == r.x.shape == (T, H)
    v = behind(y.double(), d(w1), d(gate), eps)
    want = scale * h.double() + v
    mag = (scale * h.double()).abs() + v.abs()
    inside(r.h, want, 2.0 ** -18 * mag + HALF[ht] * (want.abs() + 2.0 ** -18 * mag), "h")
    want = rms(r.h.double(), eps) * w2.double()  # of the stream as it is kept
    inside(r.x, want, (2.0 ** -18 + 2.0 ** -8 * (1 + 2.0 ** -18)) * want.abs(), "x")
    return r


TYPES = [(BF16, BF16), (BF16, F32), (F32, BF16), (F32, F32)]
SIZES = [(1, 8), (3, 40), (5, 256), (7, 264), (2, 4096), (9, 4104), (400, 4104), (33, 7168), (310, 7168), (4, 8192), (6, 8200), (3, 16384), (700, 264)]


@pytest.mark.parametrize("yt,ht", TYPES)
@pytest.mark.parametrize("T,H", SIZES)
def test_forward(T, H, yt, ht):
    check_forward(T, H, yt, ht, True, "channel", 0.7)


@pytest.mark.parametrize("post", [True, False])
@pytest.mark.parametrize("kind", ["none", "channel", "token"])
@pytest.mark.parametrize("scale", [1.0, 0.25, 0.0, -1.5])
def test_forward_options(post, kind, scale):
    check_forward(37, 1032, BF16, F32, post, kind, scale)
    check_forward(350, 4800, BF16, BF16, post, kind, scale)


def test_forward_without_a_block_or_a_next_norm():
    h, y, w = draw(20, 520, BF16, 1), draw(20, 520, BF16, 2), vec(520, 3)
    r = mx.block_norm(None, h, w)
    assert torch.equal(r.h, h)
    want = rms(h.double(), EPS) * w.double()
    inside(r.x, want, 2.0 ** -7 * want.abs(), "x")
    last = mx.block_norm(y, h, None, w)
    assert last.x is None and torch.equal(last.h, mx.block_norm(y, h, w, w).h)


def test_forward_extremes():
    """Rows of zeros, of one value, tiny and large ones, and NaN or infinity in one row alone."""
    T, H = 12, 512
    y, h = draw(T, H, F32, 1), draw(T, H, F32, 2)
    y[0] = 0.0
    y[1], h[1] = 0.0, 0.0
    y[2] *= 1e-20
    y[3] *= 1e15
    h[4] *= 1e15
    y[5], h[5] = 3.0, 0.0
    r = check_forward(T, H, F32, F32, True, "channel", 1.0, y=y, h=h)
    assert bool((r.x[1] == 0).all()) and bool((r.h[1] == 0).all())
    y[7, 100], h[9, 3] = float("nan"), float("inf")
    bad = mx.block_norm(y, h, vec(H, 4), vec(H, 3), gate_of("channel", T, H), 1.0)
    keep = torch.ones(T, dtype=torch.bool, device="cuda")
    keep[[7, 9]] = False
    assert torch.equal(bad.x[keep], r.x[keep]) and torch.equal(bad.h[keep], r.h[keep])
    assert bool(torch.isnan(bad.x[7]).all()) and bool(torch.isnan(bad.x[9, 3]))


@pytest.mark.parametrize("ht", [BF16, F32])
def test_forward_pitches_and_guards(ht):
    T, H = 23, 136
    yb, hb = draw(T, H + 16, BF16, 1), draw(T, H + 24, ht, 2)
    y, h = yb[:, 8:8 + H], hb[:, 16:16 + H]
    w1, w2, gate = vec(H, 3), vec(H, 4), vec(T, 5)[:, None].contiguous()
    want = mx.block_norm(y.contiguous(), h.contiguous(), w2, w1, gate, 0.5)
    got = mx.block_norm(y, h, w2, w1, gate, 0.5)
    assert torch.equal(got.h, want.h) and torch.equal(got.x, want.x)
    cfg = mx.BlockNormConfig(0, 0 if ht == BF16 else 1, 2, 0.5, EPS, w2.data_ptr(), w1.data_ptr(), gate.data_ptr())
    out = [torch.full((T + 2, H), 9.0, dtype=t, device="cuda") for t in (ht, BF16)]
    assert mx.block_norm_c(cfg, T, H, y, H + 16, h, H + 24, out[0][1:T + 1], out[1][1:T + 1]) == 0
    assert torch.equal(out[0][1:T + 1], want.h) and torch.equal(out[1][1:T + 1], want.x)
    for o in out:
        assert bool((o[0] == 9).all() and (o[-1] == 9).all())
    stream = h.contiguous().clone()  # in place
    assert mx.block_norm_c(cfg, T, H, y, H + 16, stream, H, stream, out[1][1:T + 1]) == 0
    assert torch.equal(stream, want.h)


# ---- gradients -----------------------------------------------------------------------------------------

def formulas(gh, gx, y, h, w2, w1, gate, scale, eps):
    """(gradients, magnitudes of what each adds up) in float64, term by term."""
    T, H = h.shape
    y, h, w2, w1, gate = y.double(), h.double(), w2.double(), d(w1), d(gate)
    total, mag, out, mags = torch.zeros_like(h), torch.zeros_like(h), {}, {}
    if gh is not None:
        total, mag = gh.double(), gh.double().abs()
    if gx is not None:
        r = 1 / torch.sqrt((h * h).mean(1, keepdim=True) + eps)
        t, n = gx.double() * w2, h * r
        total = total + r * (t - n * (t * n).mean(1, keepdim=True))
        mag = mag + r * (t.abs() + n.abs() * (t * n).abs().mean(1, keepdim=True))
        out["pre"], mags["pre"] = (gx.double() * n).sum(0), (gx.double() * n).abs().sum(0)
    out["h"], mags["h"] = scale * total, abs(scale) * mag
    g = torch.ones(1, 1, dtype=torch.float64, device="cuda") if gate is None else gate
    u, ud = y, mag * g.abs()
    if w1 is not None:
        r = 1 / torch.sqrt((y * y).mean(1, keepdim=True) + eps)
        n = y * r
        u = n * w1
        b, bm = total * g * w1, mag * (g * w1).abs()
        out["y"] = r * (b - n * (b * n).mean(1, keepdim=True))
        mags["y"] = r * (bm + n.abs() * (bm * n.abs()).mean(1, keepdim=True))
        out["post"], mags["post"] = (g * total * n).sum(0), (mag * (g * n).abs()).sum(0)
    else:
        out["y"], mags["y"] = g * total, ud
    if gate is not None:
        dim = 0 if gate.dim() == 1 else 1
        out["gate"], mags["gate"] = (total * u).sum(dim), (mag * u.abs()).sum(dim)
    return out, mags


def check_backward(T, H, yt, ht, post, kind, scale, gh=True, gx=True, eps=EPS):
    y, h = draw(T, H, yt, 11), draw(T, H, ht, 12)
    w1, w2, gate = vec(H, 3) if post else None, vec(H, 4), gate_of(kind, T, H)
    dh = draw(T, H, ht, 13) if gh else None
    dx = draw(T, H, BF16, 14) if gx else None
    got = mx.block_norm_backward(dh, dx, y, h, w2, w1, gate, scale, eps)
    want, mags = formulas(dh, dx, y, h, w2, w1, gate, scale, eps)
    path = (T + 151) // 152 + 38 + 8 + 64  # additions of a sum over tokens, and its terms' own roundings
    for name, t in (("h", got.h), ("y", got.y)):
        tol = 2.0 ** -17 * mags[name]
        inside(t, want[name], tol + HALF[t.dtype] * (want[name].abs() + tol), name)
    if gx:
        inside(got.pre_weight, want["pre"], path * 2.0 ** -23 * mags["pre"], "pre_weight")
    else:
        assert bool((got.pre_weight == 0).all())
    if post:
        inside(got.post_weight, want["post"], (path + 64) * 2.0 ** -23 * mags["post"], "post_weight")
    if kind != "none":
        assert got.gate.shape == gate.shape
        inside(got.gate.view(-1), want["gate"], ((path if kind == "channel" else 64) + 64) * 2.0 ** -23 * mags["gate"], "gate")
    return got


@pytest.mark.parametrize("yt,ht", TYPES)
@pytest.mark.parametrize("T,H", SIZES)
def test_backward(T, H, yt, ht):
    check_backward(T, H, yt, ht, True, "channel", 0.7)


@pytest.mark.parametrize("post", [True, False])
@pytest.mark.parametrize("kind", ["none", "channel", "token"])
@pytest.mark.parametrize("gh,gx", [(True, True), (True, False), (False, True)])
def test_backward_options(post, kind, gh, gx):
    check_backward(61, 1032, BF16, F32, post, kind, 0.25, gh, gx)
    check_backward(900, 520, F32, BF16, post, kind, 1.0, gh, gx)


def test_backward_without_a_block():
    h, w, dx = draw(50, 264, F32, 1), vec(264, 2), draw(50, 264, BF16, 3)
    got = mx.block_norm_backward(None, dx, None, h, w)
    assert got.y is None and got.gate is None and got.post_weight is None
    want, mags = formulas(None, dx, torch.zeros_like(h), h, w, None, None, 1.0, EPS)
    inside(got.h, want["h"], 2.0 ** -17 * mags["h"], "h")
    inside(got.pre_weight, want["pre"], 120 * 2.0 ** -23 * mags["pre"], "pre_weight")


@pytest.mark.parametrize("post,kind", [(True, "channel"), (True, "token"), (False, "token"), (True, "none")])
def test_gradients_against_autograd_and_differences(post, kind):
    """The formulas used above are autograd's, and the package's gradients the slopes of the function in 64 bits."""
    T, H, scale = 5, 48, 0.6
    y, h = draw(T, H, F32, 21), draw(T, H, F32, 22)
    w1, w2, gate = vec(H, 3) if post else None, vec(H, 4), gate_of(kind, T, H)
    gh, gx = draw(T, H, F32, 23), draw(T, H, BF16, 24)
    leaves = {"y": y.double(), "h": h.double(), "pre": w2.double(), "post": d(w1), "gate": d(gate)}
    leaves = {k: v.clone().requires_grad_() for k, v in leaves.items() if v is not None}

    def loss(l):
        s = scale * l["h"] + behind(l["y"], l.get("post"), l.get("gate"), EPS)
        return (s * gh.double()).sum() + (rms(s, EPS) * l["pre"] * gx.double()).sum()
    want = dict(zip(leaves, torch.autograd.grad(loss(leaves), list(leaves.values()))))
    stream = (scale * h.double() + behind(y.double(), d(w1), d(gate), EPS)).float()
    got = mx.block_norm_backward(gh, gx, y, stream, w2, w1, gate, scale)
    got = {"y": got.y, "h": got.h, "pre": got.pre_weight, "post": got.post_weight, "gate": got.gate}
    step = 2.0 ** -12
    for name, leaf in leaves.items():
        top = want[name].abs().max()
        assert bool(((got[name].double() - want[name]).abs() <= 1e-5 * top).all()), name
        for at in (0, leaf.numel() // 2, leaf.numel() - 1):
            moved = []
            for sign in (1, -1):
                m = {k: v.detach().clone() for k, v in leaves.items()}
                m[name].view(-1)[at] += sign * step
                moved.append(loss(m))
            slope = float(moved[0] - moved[1]) / (2 * step)
            assert abs(slope - float(got[name].reshape(-1)[at])) <= 1e-4 * float(top) + 1e-5, (name, at)


def test_backward_pitches_repeats_and_parts():
    """Inputs with larger pitches, results equal in every repeat, and each output wanted alone."""
    T, H = 410, 264
    big = [draw(T, H + 8 * (i + 1), t, 30 + i) for i, t in enumerate((BF16, BF16, BF16, F32, F32))]
    dx, y = big[0][:, 8:8 + H], big[1][:, :H]
    h, dh = big[3][:, 8:8 + H], big[4][:, 16:16 + H]
    w1, w2, gate = vec(H, 3), vec(H, 4), vec(H, 5)
    want = mx.block_norm_backward(dh.contiguous(), dx.contiguous(), y.contiguous(), h.contiguous(), w2, w1, gate, 0.5)
    for _ in range(3):
        got = mx.block_norm_backward(dh, dx, y, h, w2, w1, gate, 0.5)
        assert all(torch.equal(a, b) for a, b in zip(got, want))
    cfg = mx.BlockNormConfig(0, 1, 1, 0.5, EPS, w2.data_ptr(), w1.data_ptr(), gate.data_ptr())
    ws = torch.empty(mx.block_norm_backward_workspace_bytes(T, H), dtype=torch.uint8, device="cuda")
    names = ("dh", "dy", "dpre", "dpost", "dgate")
    whole = dict(zip(names, (want.h, want.y, want.pre_weight, want.post_weight, want.gate)))
    for alone in names:
        out = {n: torch.full_like(whole[n], 9.0) if n == alone else None for n in names}
        assert mx.block_norm_backward_c(cfg, T, H, dh, H + 40, dx, H + 8, y, H + 16, h, H + 32, *(out[n] for n in names), ws) == 0
        assert torch.equal(out[alone], whole[alone]), alone


def test_no_rows():
    H = 72
    e = torch.empty(0, H, dtype=BF16, device="cuda")
    w = vec(H, 1)
    assert mx.block_norm(e, e, w, w, w).x.shape == (0, H)
    g = mx.block_norm_backward(e, e, e, e, w, w, w)
    assert all(bool((t == 0).all()) and t.shape == (H,) for t in (g.pre_weight, g.post_weight, g.gate))
    z = torch.empty(4, 0, dtype=BF16, device="cuda")
    assert mx.block_norm(z, z, torch.empty(0, device="cuda")).x.shape == (4, 0)
    assert math.prod(mx.block_norm_backward(z, z, z, z, torch.empty(0, device="cuda")).h.shape) == 0


@pytest.mark.parametrize("T", [1, 300])
def test_a_gate_per_token_of_rows_without_columns(T):
    """Sums over nothing are zeros."""
    z, w = torch.empty(T, 0, dtype=BF16, device="cuda"), torch.empty(0, device="cuda")
    gate = torch.ones(T, 1, device="cuda")
    torch.full((T, 1), 7.0, device="cuda")  # what the gradient's memory may hold
    assert bool((mx.block_norm_backward(z, z, z, z, w, w, gate).gate == 0).all())
    cfg, out = mx.BlockNormConfig(0, 0, 2, 1.0, EPS, None, None, gate.data_ptr()), torch.full((T + 2,), 9.0, device="cuda")
    assert mx.block_norm_backward_c(cfg, T, 0, None, 0, None, 0, None, 0, None, 0, None, None, None, None, out[1:T + 1], None) == 0
    assert bool((out[1:T + 1] == 0).all()) and bool((out[[0, -1]] == 9).all())


# Layouts of the gradients that the options meet: two vectors per thread with the weights kept in shared memory, a row shared by
# two CTAs with an odd split and with whole ones.
@pytest.mark.parametrize("yt,ht", TYPES)
@pytest.mark.parametrize("post", [True, False])
@pytest.mark.parametrize("kind", ["none", "channel", "token"])
@pytest.mark.parametrize("T,H", [(61, 4800), (331, 5000), (37, 8200), (170, 8208), (9, 16384)])
def test_backward_options_of_long_rows(T, H, kind, post, yt, ht):
    for gh, gx in ((True, True), (True, False), (False, True)):
        check_backward(T, H, yt, ht, post, kind, 0.25, gh, gx)
    assert mx.mxfp8_device_fault_word() == 0


@pytest.mark.parametrize("yt,ht", TYPES)
@pytest.mark.parametrize("T,H", [(61, 4800), (170, 8208), (9, 16384)])
def test_forward_options_of_long_rows(T, H, yt, ht):
    for post in (True, False):
        for kind in ("none", "channel", "token"):
            check_forward(T, H, yt, ht, post, kind, -0.5)
    assert mx.mxfp8_device_fault_word() == 0


@pytest.mark.parametrize("T,H", [(40, 520), (200, 4800), (170, 8208)])
def test_outputs_of_long_rows_alone(T, H):
    """Each output wanted alone is what it is among the others, without the inputs that it does not need."""
    y, h, dh, dx = draw(T, H, BF16, 1), draw(T, H, F32, 2), draw(T, H, F32, 3), draw(T, H, BF16, 4)
    w1, w2 = vec(H, 5), vec(H, 6)
    names = ("dh", "dy", "dpre", "dpost", "dgate")
    ws = torch.empty(mx.block_norm_backward_workspace_bytes(T, H), dtype=torch.uint8, device="cuda")
    for kind, number in (("channel", 1), ("token", 2), ("none", 0)):
        for post in (w1, None):
            gate = gate_of(kind, T, H)
            cfg = mx.BlockNormConfig(0, 1, number, 0.5, EPS, w2.data_ptr(), None if post is None else post.data_ptr(), None if gate is None else gate.data_ptr())
            whole = dict(zip(names, (lambda g: (g.h, g.y, g.pre_weight, g.post_weight, g.gate))(mx.block_norm_backward(dh, dx, y, h, w2, post, gate, 0.5))))
            for alone in (n for n in names if whole[n] is not None):
                out = {n: torch.full_like(whole[n], 9.0) if n == alone else None for n in names}
                needs_y = alone == "dgate" or (post is not None and alone in ("dy", "dpost"))
                assert mx.block_norm_backward_c(cfg, T, H, dh, H, dx, H, y if needs_y else None, H, h, H, *(out[n] for n in names), ws) == 0
                assert torch.equal(out[alone], whole[alone]), (kind, alone)
    assert mx.mxfp8_device_fault_word() == 0
