"""The expert block's operators where element numbers pass 2^31, at the most experts, and with the stream written in place.

Operands are casts of normal values; of outputs too large to check whole, some rows and columns are compared with 64-bit
products of the operands' values, at the ends above all.  The bounds are those of the operators' own tests.
"""
import ctypes

import pytest
import torch

import mxfp8_ref as ref
import test_block_norm_gpu as norms
import mxfp8_block_scaled_04_gb300 as mx
from mxfp8_block_scaled_04_gb300 import norm

pytestmark = pytest.mark.gpu

BF16, F32 = torch.bfloat16, torch.float32


@pytest.fixture(autouse=True)
def free_memory():
    yield
    torch.cuda.empty_cache()


def randn(*shape, seed=0):
    return torch.randn(*shape, generator=torch.Generator(device="cuda").manual_seed(seed), device="cuda", dtype=BF16)


def grouped(x, offsets, fmt):
    return mx.quantize_grouped(x, torch.tensor(offsets).cuda(), fmt, swizzled=True)


def compare(got, a, b, bf16):
    want, tol = ref.product_bound(a, b, bf16)
    err = (got.cpu().double() - want).abs()
    assert bool((err <= tol).all()), (float((err - tol).max()), float(err.max()))


def some(n):
    return sorted({0, 1, n // 3, n // 2 + 7, n - 2, n - 1})


def plane_rows(codes, plane, rows, cols_blocks, fmt):
    """Values [len(rows), C] of rows of one rowwise plane."""
    at = torch.tensor(rows)
    v = ref.elements(codes[at.cuda()], fmt)
    byte = torch.empty(len(rows), cols_blocks, dtype=torch.long)
    for i, r in enumerate(rows):
        b = torch.arange(cols_blocks)
        where = ((r // 128) * -(-cols_blocks // 4) + b // 4) * 512 + 16 * (r % 32) + 4 * (r % 128 // 32) + b % 4
        byte[i] = plane[where.cuda()].cpu().long()
    return v * (2.0 ** (byte - 127).double()).repeat_interleave(32, 1)[:, :codes.shape[1]]


def test_products_with_long_outputs():
    """Forward and input gradient: 2.2e9 elements out, one expert; their rows' numbers times the pitch pass 2^31."""
    R, wide, thin = 137000, 16400, 48
    x, dy = grouped(randn(R, thin, seed=1), [0, R], "e4m3"), grouped(randn(R, thin, seed=2), [0, R], "e5m2")
    w, v = grouped(randn(wide, thin, seed=3), [0, wide], "e4m3"), grouped(randn(thin, wide, seed=4), [0, thin], "e4m3")
    off = torch.tensor([0, R]).cuda()
    rows = some(R)
    y = mx.matmul_mxfp8_grouped(x, off, w)
    assert y.numel() > 1 << 31 and mx.mxfp8_device_fault_word() == 0
    a = plane_rows(x.out_row, x.scale_row, rows, 2, "e4m3")
    compare(y[torch.tensor(rows).cuda()], a, ref.groups(w.out_row, w.scale_row, [0, wide], "e4m3", True)[0], True)
    del y
    dx = mx.matmul_mxfp8_grouped_dgrad(dy, off, v)
    assert dx.shape == (R, wide) and mx.mxfp8_device_fault_word() == 0
    a = plane_rows(dy.out_row, dy.scale_row, rows, 2, "e5m2")
    compare(dx[torch.tensor(rows).cuda()], a, ref.groups(v.out_col, v.scale_col, [0, thin], "e4m3", False)[0].t(), True)


def test_weight_gradients_past_2_to_31_elements():
    sizes, N, K = [40, 0, 3, 65], 16400, 40016
    off = torch.tensor([0] + sizes).cumsum(0)
    R = int(off[-1])
    dy, x = grouped(randn(R, N, seed=1), off.tolist(), "e5m2"), grouped(randn(R, K, seed=2), off.tolist(), "e4m3")
    dw = mx.matmul_mxfp8_grouped_wgrad(dy, x, off.cuda(), BF16)
    assert dw.numel() > 1 << 31 and mx.mxfp8_device_fault_word() == 0
    cols = torch.tensor(some(K))
    d, v = ref.groups(dy.out_col, dy.scale_col, off.tolist(), "e5m2", False), ref.groups(x.out_col, x.scale_col, off.tolist(), "e4m3", False)
    for e in range(len(sizes)):
        compare(dw[e][:, cols.cuda()], d[e].t(), v[e][:, cols].t(), True)
        compare(dw[e][some(N)], d[e].t()[some(N)], v[e].t(), True)


def test_linear_with_a_long_output():
    M, N, K = 300, (1 << 23) + 40, 40
    w = mx.quantize_mxfp4(randn(N, K, seed=1)).row
    x = randn(M, K, seed=2)
    y = mx.linear_mxfp4(x, w)
    assert y.numel() > 1 << 31 and mx.mxfp8_device_fault_word() == 0
    xd, plane = x.double(), 512  # one scale tile along K: 128 rows of w
    for tile in (0, N // 256, N // 128):
        r0, r1 = 128 * tile, min(128 * tile + 128, N)
        part = mx.MXFP4Matrix(w.codes[r0:r1], w.scales[plane * tile:plane * (tile + 1)].clone(), r1 - r0, K)
        wd = mx.dequantize_mxfp4(part, F32).double()
        want = xd @ wd.t()
        amax = torch.nn.functional.pad(xd, (0, 24)).unflatten(1, (2, 32)).abs().amax(2).repeat_interleave(32, 1)[:, :K]
        tol = ((K + 8) * 2.0 ** -23 * 4 * xd.abs() + amax * 2.0 ** -22 + 2.0 ** -126) @ wd.abs().t()
        err = (y[:, r0:r1].double() - want).abs()
        assert bool((err <= tol + 2.0 ** -8 * (want.abs() + tol)).all()), (tile, float(err.max()))


@pytest.mark.parametrize("M,K", [(1, (1 << 31) - 8), (3, (1 << 29) + 264)])
def test_linear_of_long_rows(M, K):
    """A few elements of x are not zero, and the weights' levels times powers of two: the sums are exact."""
    N, pitch = 2, mx.mxfp4_row_bytes(K)
    codes = torch.full((N, pitch), 0x22, dtype=torch.uint8, device="cuda")  # 1.0 throughout
    codes[1] = 0x45                                                          # 3.0 at even columns, 2.0 at odd ones
    w = mx.MXFP4Matrix(codes, torch.full((-(-K // 128) * 512,), 127, dtype=torch.uint8, device="cuda"), N, K)
    x = torch.zeros(M, K, dtype=BF16, device="cuda")
    at = [0, 31, (1 << 28) + 5, (1 << 29) + 100, K // 2 + 1, K - 9, K - 1]
    for m in range(M):
        for i, c in enumerate(at):
            x[m, c] = (m + 1) * 2.0 ** -i
    y = mx.linear_mxfp4(x, w, F32)
    assert mx.mxfp8_device_fault_word() == 0
    for m in range(M):
        one = sum((m + 1) * 2.0 ** -i for i in range(len(at)))
        other = sum((m + 1) * 2.0 ** -i * (2.0 if c % 2 else 3.0) for i, c in enumerate(at))
        assert y[m].tolist() == [one, other]


@pytest.mark.parametrize("T,H", [(270000, 8192), (132000, 16384)])
def test_norms_past_2_to_31_elements(T, H):
    y, h = randn(T, H, seed=1), randn(T, H, seed=2)
    w1, w2 = 1 + 0.3 * randn(H, seed=3).float(), 1 + 0.3 * randn(H, seed=4).float()
    gate = 0.4 + 0.1 * randn(T, 1, seed=5).float()
    r = mx.block_norm(y, h, w2, w1, gate)
    rows = torch.tensor(some(T)).cuda()

    def rms(v):
        return v / torch.sqrt((v * v).mean(1, keepdim=True) + 1e-6)
    u = gate[rows].double() * rms(y[rows].double()) * w1.double()
    want = h[rows].double() + u
    mag = h[rows].double().abs() + u.abs()
    assert bool(((r.h[rows].double() - want).abs() <= 2.0 ** -18 * mag + 2.0 ** -8 * (want.abs() + 2.0 ** -18 * mag)).all())
    want = rms(r.h[rows].double()) * w2.double()
    assert bool(((r.x[rows].double() - want).abs() <= (2.0 ** -18 + 2.0 ** -8 * (1 + 2.0 ** -18)) * want.abs()).all())
    del h
    dh, dx = randn(T, H, seed=6), randn(T, H, seed=7)
    g = mx.block_norm_backward(dh, dx, y, r.h, w2, w1, gate)
    assert mx.mxfp8_device_fault_word() == 0
    # (r2 and the row's mean are good to 2^-18 of their magnitudes each)
    n2, t = rms(r.h[rows].double()), dx[rows].double() * w2.double()
    r2 = n2 / r.h[rows].double()
    r2 = r2.nanmean(1, keepdim=True)
    c2 = (t * n2).mean(1, keepdim=True)
    want = dh[rows].double() + r2 * (t - n2 * c2)
    mag = dh[rows].double().abs() + r2 * (t.abs() + n2.abs() * (t * n2).abs().mean(1, keepdim=True))
    assert bool(((g.h[rows].double() - want).abs() <= 2.0 ** -17 * mag + 2.0 ** -8 * (want.abs() + 2.0 ** -17 * mag)).all())
    # the sums over tokens: a CTA's rows one after the other, the CTAs' sums in eight strands
    total, bound = torch.zeros(H, dtype=torch.float64, device="cuda"), torch.zeros(H, dtype=torch.float64, device="cuda")
    for a in range(0, T, 8192):
        term = dx[a:a + 8192].double() * rms(r.h[a:a + 8192].double())
        total += term.sum(0)
        bound += term.abs().sum(0)
    steps = T / 76 + 19 + 8 + 64
    assert bool(((g.pre_weight.double() - total).abs() <= steps * 2.0 ** -24 * bound).all())


def test_products_of_512_experts():
    sizes = [(7 * i) % 5 for i in range(512)]
    N, K = 16, 32
    off = torch.tensor([0] + sizes).cumsum(0)
    R, w_off = int(off[-1]), [N * e for e in range(513)]
    x, dy = grouped(randn(R, K, seed=1), off.tolist(), "e4m3"), grouped(randn(R, N, seed=2), off.tolist(), "e5m2")
    w = grouped(randn(512 * N, K, seed=3), w_off, "e4m3")
    y = mx.matmul_mxfp8_grouped(x, off.cuda(), w, F32)
    dx = mx.matmul_mxfp8_grouped_dgrad(dy, off.cuda(), w, F32)
    dw = mx.matmul_mxfp8_grouped_wgrad(dy, x, off.cuda())
    assert mx.mxfp8_device_fault_word() == 0
    xs, ws = ref.groups(x.out_row, x.scale_row, off.tolist(), "e4m3", True), ref.groups(w.out_row, w.scale_row, w_off, "e4m3", True)
    ds, wc = ref.groups(dy.out_row, dy.scale_row, off.tolist(), "e5m2", True), ref.groups(w.out_col, w.scale_col, w_off, "e4m3", False)
    dc, xc = ref.groups(dy.out_col, dy.scale_col, off.tolist(), "e5m2", False), ref.groups(x.out_col, x.scale_col, off.tolist(), "e4m3", False)
    for e in range(512):
        a, b = int(off[e]), int(off[e + 1])
        compare(y[a:b], xs[e], ws[e], False)
        compare(dx[a:b], ds[e], wc[e].t(), False)
        compare(dw[e], dc[e].t(), xc[e].t(), False)
    # the same experts in 4 bits, uncast tokens: each row as the dense call on its expert's weights
    m = [mx.quantize_mxfp4(v).row for v in randn(512 * N, K, seed=3).view(512, N, K)]
    w4 = mx.MXFP4Matrix(torch.stack([c.codes for c in m]), torch.stack([c.scales for c in m]), N, K)
    tokens = randn(R, K, seed=4)
    got = mx.linear_mxfp4_grouped(tokens, off.cuda(), w4, out_dtype=F32)
    for e in range(0, 512, 37):
        a, b = int(off[e]), int(off[e + 1])
        want = mx.linear_mxfp4(tokens[a:b], m[e], F32)
        most = tokens[a:b].double().abs() @ mx.dequantize_mxfp4(m[e], F32).double().abs().t()
        assert bool(((got[a:b].double() - want.double()).abs() <= 2 * (K + 8) * 2.0 ** -23 * 4 * most).all())


@pytest.mark.parametrize("T,H,dtype", [(700, 264, BF16), (310, 7168, F32), (90, 16384, BF16)])
def test_stream_in_place(T, H, dtype):
    y, h = randn(T, H, seed=1), randn(T, H, seed=2).to(dtype)
    w1, w2, gate = (1 + 0.3 * randn(H, seed=s).float() for s in (3, 4, 5))
    want = mx.block_norm(y, h, w2, w1, gate, 0.7)
    cfg = norm.BlockNormConfig(0, 0 if dtype is BF16 else 1, norm.GATE_CHANNEL, 0.7, 1e-6, w2.data_ptr(), w1.data_ptr(), gate.data_ptr())
    x = torch.empty(T, H, dtype=BF16, device="cuda")
    assert norm.block_norm_c(cfg, T, H, y, H, h, H, h, x) == 0
    assert ctypes.sizeof(cfg) > 0 and torch.equal(h, want.h) and torch.equal(x, want.x)


@pytest.mark.parametrize("T,H,kind", [(270000, 8192, "token"), (132000, 16384, "token"), (132000, 16384, "channel")])
def test_norm_gradients_past_2_to_31_elements(T, H, kind):
    """Those of y, of the gate and of the weight behind the block, by the formulas and bounds of the norms' own tests."""
    y, h, dh, dx = (randn(T, H, seed=s) for s in range(4))
    w1, w2 = 1 + 0.3 * randn(H, seed=5).float(), 1 + 0.3 * randn(H, seed=6).float()
    gate = 0.4 + 0.1 * (randn(T, 1, seed=7) if kind == "token" else randn(H, seed=7)).float()
    g = mx.block_norm_backward(dh, dx, y, h, w2, w1, gate, 0.7)
    assert mx.mxfp8_device_fault_word() == 0
    rows = torch.tensor(some(T)).cuda()
    part = gate[rows] if kind == "token" else gate
    want, mags = norms.formulas(dh[rows], dx[rows], y[rows], h[rows], w2, w1, part, 0.7, 1e-6)
    for name, got in (("y", g.y), ("h", g.h)):
        tol = 2.0 ** -17 * mags[name]
        norms.inside(got[rows], want[name], tol + 2.0 ** -8 * (want[name].abs() + tol), name)
    if kind == "token":
        norms.inside(g.gate.view(-1)[rows], want["gate"], 128 * 2.0 ** -23 * mags["gate"], "gate")
    sums = {n: [torch.zeros(H, dtype=torch.float64, device="cuda") for _ in range(2)] for n in ("pre", "post", "gate")}
    for a in range(0, T, 4096):
        s = slice(a, a + 4096)
        want, mags = norms.formulas(dh[s], dx[s], y[s], h[s], w2, w1, gate[s] if kind == "token" else gate, 0.7, 1e-6)
        for n, (total, most) in sums.items():
            if n != "gate" or kind == "channel":
                total += want[n]
                most += mags[n]
    path = T / 76 + 38 + 8 + 64  # additions of a sum over tokens, and its terms' own roundings
    for n, got in (("pre", g.pre_weight), ("post", g.post_weight), ("gate", g.gate)):
        if n != "gate" or kind == "channel":
            norms.inside(got, sums[n][0], (path + 64) * 2.0 ** -23 * sums[n][1], n)
