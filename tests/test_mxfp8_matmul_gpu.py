"""Experts' products in MXFP8 (forward, input gradient, weight gradient) against 64-bit products of the cast operands."""
import pytest
import torch

import mxfp8_ref as ref
import mxfp8_block_scaled_04_gb300 as mx

pytestmark = pytest.mark.gpu

BF16, F32 = torch.bfloat16, torch.float32


def draw(M, N, seed, spread=1.0):
    g = torch.Generator().manual_seed(seed)
    return (torch.randn(M, N, generator=g) * torch.exp(spread * torch.randn(M, 1, generator=g))).to(BF16)


def cast(x, offsets, fmt):
    return mx.quantize_grouped(x.cuda(), torch.tensor(offsets).cuda(), fmt, swizzled=True)


class Layer:
    """Casts of x [R, K], dy [R, N] and w [E * N, K], and their 64-bit values by expert."""

    def __init__(self, sizes, N, K, x_fmt="e4m3", w_fmt="e4m3", dy_fmt="e5m2", x=None, w=None, dy=None):
        E, R = len(sizes), sum(sizes)
        self.N, self.K, self.R, self.E = N, K, R, E
        self.fmts = (x_fmt, w_fmt, dy_fmt)
        self.off = torch.tensor([0] + sizes).cumsum(0).tolist()
        self.w_off = [e * N for e in range(E + 1)]
        self.x = cast(draw(R, K, 1) if x is None else x, self.off, x_fmt)
        self.dy = cast(draw(R, N, 2) if dy is None else dy, self.off, dy_fmt)
        self.w = cast(draw(E * N, K, 3, 0.2) if w is None else w, self.w_off, w_fmt)
        self.offsets = torch.tensor(self.off).cuda()

    def rows(self, which):
        t, off, fmt = {"x": (self.x, self.off, self.fmts[0]), "w": (self.w, self.w_off, self.fmts[1]),
                       "dy": (self.dy, self.off, self.fmts[2])}[which]
        return ref.groups(t.out_row, t.scale_row, off, fmt, True)

    def cols(self, which):
        t, off, fmt = {"x": (self.x, self.off, self.fmts[0]), "w": (self.w, self.w_off, self.fmts[1]),
                       "dy": (self.dy, self.off, self.fmts[2])}[which]
        return ref.groups(t.out_col, t.scale_col, off, fmt, False)

    def check(self, dtype=BF16):
        xf, wf, df = self.fmts
        err = torch.zeros(1, dtype=torch.int32, device="cuda")
        y = mx.matmul_mxfp8_grouped(self.x, self.offsets, self.w, dtype, xf, wf, err).cpu().double()
        dx = mx.matmul_mxfp8_grouped_dgrad(self.dy, self.offsets, self.w, dtype, df, wf, err).cpu().double()
        dw = mx.matmul_mxfp8_grouped_wgrad(self.dy, self.x, self.offsets, dtype, df, xf, err).cpu().double()
        assert int(err) == 0 and mx.mxfp8_device_fault_word() == 0
        worst = 0.0
        for got, pairs in ((y.split([b - a for a, b in zip(self.off, self.off[1:])]), zip(self.rows("x"), self.rows("w"))),
                           (dx.split([b - a for a, b in zip(self.off, self.off[1:])]), zip(self.rows("dy"), (w.t() for w in self.cols("w")))),
                           (dw, zip((d.t() for d in self.cols("dy")), (x.t() for x in self.cols("x"))))):
            for e, (g, (a, b)) in enumerate(zip(got, pairs)):
                want, tol = ref.product_bound(a, b, dtype == BF16)
                bad = ~((g - want).abs() <= tol)
                assert not bool(bad.any()), (e, int(bad.sum()), g.shape, float((g - want).abs().max()), float(want.abs().max()))
                if g.numel() and dtype == F32:
                    worst = max(worst, float((g - want).norm() / want.norm().clamp(min=1e-300)))
        return worst


SIZES = [[5], [0, 3, 0], [128, 0, 1, 127, 129], [1] * 40, [300, 2, 0, 0, 61], [0, 0, 257], [32, 64, 31, 33]]


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("N,K", [(48, 80), (256, 128), (272, 528), (16, 16)])
@pytest.mark.parametrize("sizes", SIZES)
def test_products(sizes, N, K, dtype):
    Layer(sizes, N, K).check(dtype)


@pytest.mark.parametrize("sizes,N,K", [([700, 0, 1025, 256, 3, 1700], 1424, 336), ([5120, 1], 1008, 256), ([40] * 30, 528, 1040)])
def test_products_of_many_tiles(sizes, N, K):
    """More tiles than pairs of CTAs: both accumulators and every stage are reused."""
    Layer(sizes, N, K).check(BF16)


@pytest.mark.parametrize("x_fmt", ["e4m3", "e5m2"])
@pytest.mark.parametrize("w_fmt", ["e4m3", "e5m2"])
@pytest.mark.parametrize("dy_fmt", ["e4m3", "e5m2"])
def test_formats(x_fmt, w_fmt, dy_fmt):
    Layer([100, 37], 144, 208, x_fmt, w_fmt, dy_fmt).check(F32)


def test_each_position_counts():
    """Small integers, equal scales: every sum is exact, whatever the order."""
    g = torch.Generator().manual_seed(4)
    sizes, N, K = [300, 77, 512], 272, 400
    x, dy, w = (torch.randint(-4, 5, s, generator=g).to(BF16) for s in ((889, K), (889, N), (3 * N, K)))
    layer = Layer(sizes, N, K, x=x, dy=dy, w=w)
    y = mx.matmul_mxfp8_grouped(layer.x, layer.offsets, layer.w, F32).cpu().double()
    dx = mx.matmul_mxfp8_grouped_dgrad(layer.dy, layer.offsets, layer.w, F32).cpu().double()
    dw = mx.matmul_mxfp8_grouped_wgrad(layer.dy, layer.x, layer.offsets, F32).cpu().double()
    for e in range(3):
        s = slice(layer.off[e], layer.off[e + 1])
        we = w[e * N:(e + 1) * N].double()
        assert torch.equal(y[s], x[s].double() @ we.t())
        assert torch.equal(dx[s], dy[s].double() @ we)
        assert torch.equal(dw[e], dy[s].double().t() @ x[s].double())


def test_sums_keep_fp32():
    """Norm-wise error of long sums of random signs: far below one rounding to 2^-14 per step."""
    assert Layer([4096, 100], 256, 4096).check(F32) < 2e-6


def test_ragged_rows_stay_out_of_their_neighbours():
    """An expert's last stage holds the next one's rows, 2^20 times as large or as small: exact sums of small integers show one that
    is added.  Both CTAs of a pair zero such rows; repeats take other interleavings."""
    g = torch.Generator().manual_seed(9)
    sizes = [1 + (37 * i) % 131 for i in range(60)]
    off = torch.tensor([0] + sizes).cumsum(0).tolist()
    R, N, K = off[-1], 528, 784
    x, dy = (torch.randint(-4, 5, (R, c), generator=g).double() for c in (K, N))
    for e in range(1, 60, 2):
        x[off[e]:off[e + 1]] *= 2.0 ** 20
    qx, qd = cast(x.to(BF16), off, "e4m3"), cast(dy.to(BF16), off, "e5m2")
    offsets = torch.tensor(off).cuda()
    first = mx.matmul_mxfp8_grouped_wgrad(qd, qx, offsets)
    for e in range(60):
        s = slice(off[e], off[e + 1])
        assert torch.equal(first[e].cpu().double(), dy[s].t() @ x[s]), e
    for _ in range(30):
        assert torch.equal(mx.matmul_mxfp8_grouped_wgrad(qd, qx, offsets), first)
    assert mx.mxfp8_device_fault_word() == 0


def in_pieces(total, piece):
    """(start, end) of the pieces that a sum to fp32 is made in."""
    return [(a, min(a + piece, total)) for a in range(0, total, piece)]


def added(parts):
    s = parts[0]
    for t in parts[1:]:
        s = s + t
    return s


@pytest.mark.parametrize("N,K", [(16, 16), (272, 528), (2064, 1040)])
def test_long_weight_gradients_are_sums_of_pieces(N, K):
    """To fp32 a sum over more than 2048 rows is the sum of its pieces, bit for bit, whatever the other experts have."""
    sizes = [9011, 5, 0, 4096, 2048, 2049, 40, 6000]
    off = torch.tensor([0] + sizes).cumsum(0).tolist()
    R = off[-1]
    x, dy = draw(R, K, 1), draw(R, N, 2)
    whole = mx.matmul_mxfp8_grouped_wgrad(cast(dy, off, "e5m2"), cast(x, off, "e4m3"), torch.tensor(off).cuda())
    cuts = [(e, off[e] + a, off[e] + b) for e in range(len(sizes)) for a, b in in_pieces(sizes[e], 2048)]
    ends = [0] + [b for _, _, b in cuts]  # a piece starts at a whole number of blocks: the same casts
    parts = mx.matmul_mxfp8_grouped_wgrad(cast(dy, ends, "e5m2"), cast(x, ends, "e4m3"), torch.tensor(ends).cuda())
    for e, n in enumerate(sizes):
        mine = [parts[i] for i, c in enumerate(cuts) if c[0] == e]
        assert torch.equal(whole[e], added(mine) if n else torch.zeros_like(whole[e])), e
    again = mx.matmul_mxfp8_grouped_wgrad(cast(dy, off, "e5m2"), cast(x, off, "e4m3"), torch.tensor(off).cuda())
    assert torch.equal(again, whole) and mx.mxfp8_device_fault_word() == 0


@pytest.mark.parametrize("sizes", [[40], [300, 0, 1, 257]])
def test_long_products_are_sums_of_pieces(sizes):
    """Forward over K and input gradient over N to fp32: of pieces of 8192."""
    off = torch.tensor([0] + sizes).cumsum(0).tolist()
    E, R, L, C = len(sizes), off[-1], 2 * 8192 + 3616, 272
    offsets = torch.tensor(off).cuda()

    def ends(n):
        return [n * e for e in range(E + 1)]
    x, w = draw(R, L, 3), draw(E * C, L, 4, 0.2)
    y = mx.matmul_mxfp8_grouped(cast(x, off, "e4m3"), offsets, cast(w, ends(C), "e4m3"), F32)
    parts = [mx.matmul_mxfp8_grouped(cast(x[:, a:b].contiguous(), off, "e4m3"), offsets, cast(w[:, a:b].contiguous(), ends(C), "e4m3"), F32)
             for a, b in in_pieces(L, 8192)]
    assert torch.equal(y, added(parts))
    dy, w = draw(R, L, 5), draw(E * L, C, 6, 0.2)
    dx = mx.matmul_mxfp8_grouped_dgrad(cast(dy, off, "e5m2"), offsets, cast(w, ends(L), "e4m3"), F32)
    parts = []
    for a, b in in_pieces(L, 8192):
        rows = w.view(E, L, C)[:, a:b].reshape(E * (b - a), C).contiguous()
        parts.append(mx.matmul_mxfp8_grouped_dgrad(cast(dy[:, a:b].contiguous(), off, "e5m2"), offsets, cast(rows, ends(b - a), "e4m3"), F32))
    assert torch.equal(dx, added(parts)) and mx.mxfp8_device_fault_word() == 0


def test_long_weight_gradients_keep_fp32():
    """65536 rows of very different scale: norm-wise within 1e-6 of the 64-bit product.  The truncation of a step is at most 2^-23 of the
    partial sum; 64 steps of a piece reach 2^-17 of it at worst, and the partial sums of random signs, far below the sum of the
    magnitudes, leave a twentieth of that (one sum of 2048 steps was 2.4e-5 off)."""
    layer = Layer([65536], 48, 80)
    got = mx.matmul_mxfp8_grouped_wgrad(layer.dy, layer.x, layer.offsets)[0].cpu().double()
    want = layer.cols("dy")[0].t() @ layer.cols("x")[0]
    assert float((got - want).norm() / want.norm()) < 1e-6
