"""Products of rows that are not cast with 4-bit weights (tests/mxfp4_ref.py's values of the weights), dense and per expert.

Allowed error: per block of 32 the operand differs from x by at most 2^-22 of the block's largest magnitude (2^-126 for
the smallest).  It is a sum of eight parts, octal digits between -4 and 4: a first digit d >= 1 of weight w stands for at
least (d - 4/7) w, so that it is at most 7/3 |x|, and the digits after it add up to at most 4/7 w <= 4/3 |x|: 11/3 |x| in all.
Each part is a product whose K additions may drop a unit of the last of 24 bits of a partial sum, and seven more
additions join them; bf16 adds half a unit of the last of its 8 bits.
"""
import pytest
import torch

import mxfp4_ref as ref
import mxfp8_block_scaled_04_gb300 as mx

pytestmark = pytest.mark.gpu

BF16, F32 = torch.bfloat16, torch.float32


def draw(M, N, dtype, seed, spread=1.0):
    g = torch.Generator().manual_seed(seed)
    return (torch.randn(M, N, generator=g) * torch.exp(spread * torch.randn(M, 1, generator=g))).to(dtype)


def bound(x, w, bf16):
    """(x @ w.T, allowed error) in float64."""
    x, w = x.double(), w.double()
    K = x.shape[1]
    blocks = torch.nn.functional.pad(x, (0, -K % 32)).unflatten(1, (-(-K // 32), 32))
    amax = blocks.abs().amax(2, keepdim=True)
    most = 4 * x.abs()  # what the parts' magnitudes add up to
    miss = (amax * 2.0 ** -22 + 2.0 ** -126).expand_as(blocks).flatten(1)[:, :K] * (x != 0)
    want = x @ w.t()
    tol = ((K + 8) * 2.0 ** -23 * most + miss) @ w.abs().t()
    return want, tol + (2.0 ** -8 * (want.abs() + tol) if bf16 else 0.0)


def weights(N, K, seed=2):
    w = draw(N, K, BF16, seed, 0.3)
    return mx.quantize_mxfp4(w.cuda()).row, ref.cast(w)


def check(x, w, wv, out_dtype):
    got = mx.linear_mxfp4(x.cuda(), w, out_dtype).cpu().double()
    want, tol = bound(x, wv, out_dtype == BF16)
    assert mx.mxfp8_device_fault_word() == 0
    err = (got - want).abs()
    assert bool((err <= tol).all()), (float((err - tol).max()), float(err.max()))
    return float((got - want).norm() / want.norm().clamp(min=1e-300))


@pytest.mark.parametrize("out_dtype", [BF16, F32])
@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("M,N,K", [(1, 1, 8), (1, 128, 256), (2, 40, 72), (3, 257, 1032), (4, 129, 4096), (5, 130, 40), (15, 300, 520),
                                   (16, 128, 2048), (17, 1000, 264), (33, 520, 136), (100, 264, 1000), (1, 5000, 8192)])
def test_linear(M, N, K, dtype, out_dtype):
    w, wv = weights(N, K)
    check(draw(M, K, dtype, M + K), w, wv, out_dtype)


@pytest.mark.parametrize("M,N,K", [(64, 20000, 264), (300, 4100, 136), (1030, 1000, 96)])
def test_linear_of_many_tiles(M, N, K):
    w, wv = weights(N, K)
    check(draw(M, K, BF16, 5), w, wv, BF16)


def test_keeps_fp32_accuracy():
    """Far below what one cast to 4 or 8 bits, or to bf16, would leave; fp32 x keeps its low bits."""
    w, wv = weights(512, 4096)
    assert check(draw(8, 4096, BF16, 3), w, wv, F32) < 1e-6
    assert check(draw(8, 4096, F32, 3), w, wv, F32) < 1e-6


def test_wide_ranges_within_a_block():
    """Elements far below their block's largest, powers of two apart, and outliers."""
    g = torch.Generator().manual_seed(6)
    x = torch.randn(24, 256, generator=g) * 2.0 ** -(torch.arange(256) % 32).float()
    x[::3, 7::32] *= 1e4
    w, wv = weights(96, 256)
    for dtype in (BF16, F32):
        check(x.to(dtype), w, wv, F32)


def test_every_bf16_value_alone_in_its_block():
    """The parts of each finite bf16 magnitude: against a weight of 1 the output is the value itself, to 2^-22 of it (2^-126)."""
    bits = torch.arange(0, 0x7F80, dtype=torch.int32).to(torch.int16)
    v = bits.view(BF16)
    x = torch.zeros(v.numel(), 32, dtype=BF16)
    x[:, 5] = v
    w = torch.zeros(8, 32, dtype=BF16)
    w[0, 5] = 6.0
    w[1] = 1.0
    got = mx.linear_mxfp4(x.cuda(), mx.quantize_mxfp4(w.cuda()).row, F32).cpu().double()
    top = v.double().abs() < 2.0 ** 124  # six times the largest values overflows
    err = (got[:, 0] - 6 * v.double()).abs()
    # eight parts of at most 4 |v| together, added in fp32
    tol = 6 * (v.double() * 2.0 ** -22 + 2.0 ** -126 + 9 * 2.0 ** -23 * 4 * v.double())
    assert bool((err <= tol)[top].all())
    err = (got[:, 1] - v.double()).abs()
    assert bool((err <= tol / 6)[v.double() < 2.0 ** 126].all())


def test_zeros_nan_and_infinity():
    x, (w, wv) = draw(20, 96, BF16, 1), weights(50, 96)
    x[3] = 0.0
    x[7, 40] = float("nan")
    x[9, 5] = float("inf")
    x[11, 95] = -float("inf")
    got = mx.linear_mxfp4(x.cuda(), w, F32).cpu()
    bad = torch.zeros(20, dtype=torch.bool)
    bad[[7, 9, 11]] = True
    assert torch.equal(torch.isnan(got).all(1), bad) and torch.equal(torch.isnan(got).any(1), bad)
    assert bool((got[3] == 0).all())


@pytest.mark.parametrize("dtype", [BF16, F32])
def test_pitches_and_guards(dtype):
    M, N, K, ld = 21, 70, 160, 96
    big = draw(M, K + 24, dtype, 9).cuda()
    w, _ = weights(N, K)
    x = big[:, 8:8 + K]
    want = mx.linear_mxfp4(x.contiguous(), w, dtype)
    buf = torch.full((M + 2, ld), 9.0, dtype=dtype, device="cuda")
    mx.linear_mxfp4(x, w, out=buf[1:M + 1, :N])
    assert torch.equal(buf[1:M + 1, :N], want)
    assert bool((buf[0] == 9).all() and (buf[-1] == 9).all() and (buf[:, N:] == 9).all())


def test_empty_sizes():
    w = weights(8, 64)[0]
    assert mx.linear_mxfp4(torch.ones(0, 64, dtype=BF16, device="cuda"), w).shape == (0, 8)
    none = mx.quantize_mxfp4(torch.ones(8, 0, dtype=BF16, device="cuda")).row
    assert bool((mx.linear_mxfp4(torch.ones(5, 0, dtype=BF16, device="cuda"), none) == 0).all())


# ---- experts -------------------------------------------------------------------------------------------

def experts(G, N, K, seed=2):
    w = draw(G * N, K, BF16, seed, 0.3)
    parts = [mx.quantize_mxfp4(w[g * N:(g + 1) * N].cuda()).row for g in range(G)]
    return (mx.MXFP4Matrix(torch.stack([p.codes for p in parts]), torch.stack([p.scales for p in parts]), N, K),
            [ref.cast(w[g * N:(g + 1) * N]) for g in range(G)])


SIZES = [[5], [0, 3, 0], [16, 0, 1, 17, 129], [1] * 40, [40, 2, 0, 0, 61], [0, 0, 33], [300, 7]]


@pytest.mark.parametrize("dtype,out_dtype", [(BF16, BF16), (BF16, F32), (F32, F32)])
@pytest.mark.parametrize("N,K", [(40, 72), (264, 520), (128, 256)])
@pytest.mark.parametrize("sizes", SIZES)
def test_experts(sizes, N, K, dtype, out_dtype):
    G, R = len(sizes), sum(sizes)
    T = max(1, R // 2)
    x = draw(T, K, dtype, 1)
    rows = torch.randint(0, T, (R,), generator=torch.Generator().manual_seed(3), dtype=torch.int32)
    off = torch.tensor([0] + sizes).cumsum(0)
    w, wv = experts(G, N, K)
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    got = mx.linear_mxfp4_grouped(x.cuda(), off.cuda(), w, rows=rows.cuda(), out_dtype=out_dtype, err_flag=err)
    ordered = mx.linear_mxfp4_grouped(x[rows.long()].cuda(), off.cuda(), w, out_dtype=out_dtype, err_flag=err)
    assert int(err) == 0 and mx.mxfp8_device_fault_word() == 0
    assert torch.equal(got, ordered)
    for g in range(G):
        s = slice(int(off[g]), int(off[g + 1]))
        want, tol = bound(x[rows[s].long()], wv[g], out_dtype == BF16)
        assert bool(((got[s].cpu().double() - want).abs() <= tol).all()), g


def test_experts_of_many_rows():
    """The kernel of CTA pairs, with experts whose rows fill several of its tiles."""
    test_experts([200, 0, 133, 3, 300], 3333, 328, BF16, BF16)


def test_experts_dropped_choices_and_bad_indices():
    G, N, K, R = 3, 72, 96, 40
    x, (w, wv) = draw(10, K, BF16, 4), experts(G, N, K)
    off = torch.tensor([0, 7, 7, 30])
    rows = torch.randint(0, 10, (R,), generator=torch.Generator().manual_seed(5), dtype=torch.int32)
    rows[30:] = -1
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    got = mx.linear_mxfp4_grouped(x.cuda(), off.cuda(), w, rows=rows.cuda(), out_dtype=F32, err_flag=err).cpu()
    assert int(err) == 0 and bool((got[30:] == 0).all())
    want, tol = bound(x[rows[7:30].long()], wv[2], False)
    assert bool(((got[7:30].double() - want).abs() <= tol).all())
    rows[2], rows[9] = 10, -1
    got2 = mx.linear_mxfp4_grouped(x.cuda(), off.cuda(), w, rows=rows.cuda(), out_dtype=F32, err_flag=err).cpu()
    assert int(err) == 1 and bool(torch.isnan(got2[[2, 9]]).all())
    keep = torch.ones(R, dtype=torch.bool)
    keep[[2, 9]] = False
    assert torch.equal(got2[keep], got[keep])
    for bad in ([0, 7, 5, 30], [1, 7, 7, 30], [0, 7, 7, 41], [0, 7, 7, 1 << 62], [0, -1, 7, 30]):
        err.zero_()
        out = torch.full((R, N), 9.0, device="cuda")
        ws = torch.empty(mx.mxfp4_linear_grouped_workspace_bytes(R, K, G), dtype=torch.uint8, device="cuda")
        assert mx.mxfp4_linear_grouped(x.cuda(), 0, 10, K, K, rows.cuda(), R, G, torch.tensor(bad).cuda(), w.codes, w.scales, N, out, 1,
                                       err, ws) == 0
        assert int(err) == 1 and bool((out == 9).all()), bad


# Few rows on many experts, each in a tile of its own: row counts per expert, the rest of 40 experts without any.
WEIGHTS = {}


def few_experts(G, N, K):
    """4-bit weights of G experts, and a function that gives the values of one."""
    if (G, N, K) not in WEIGHTS:
        w = torch.randn(G, N, K, generator=torch.Generator(device="cuda").manual_seed(2), device="cuda").to(BF16)
        parts = [mx.quantize_mxfp4(v).row for v in w]
        WEIGHTS[G, N, K] = (mx.MXFP4Matrix(torch.stack([p.codes for p in parts]), torch.stack([p.scales for p in parts]), N, K), w, {})
    m, w, known = WEIGHTS[G, N, K]

    def values(g):
        if g not in known:
            known[g] = ref.cast(w[g].cpu())
        return known[g]
    return m, values


FEW = [{0: 1}, {39: 2}, {3: 1, 4: 1, 20: 1, 39: 1}, {7: 16}, {0: 5, 1: 1, 38: 3}, {e: 1 for e in range(1, 33, 2)}]


@pytest.mark.parametrize("dtype,out_dtype", [(BF16, BF16), (BF16, F32), (F32, BF16), (F32, F32)])
@pytest.mark.parametrize("N,K", [(1, 8), (40, 72), (264, 520), (129, 4104), (1032, 2048), (2568, 264)])
@pytest.mark.parametrize("few", FEW)
def test_few_rows_on_many_experts(few, N, K, dtype, out_dtype):
    sizes = [few.get(e, 0) for e in range(40)]
    assert mx.mxfp4_linear_grouped_workspace_bytes(sum(sizes), K, 40) == 0
    R, T = sum(sizes), 3
    x, off = draw(T, K, dtype, 1), torch.tensor([0] + sizes).cumsum(0)
    rows = torch.randint(0, T, (R,), generator=torch.Generator().manual_seed(3), dtype=torch.int32)
    w, values = few_experts(40, N, K)
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    got = mx.linear_mxfp4_grouped(x.cuda(), off.cuda(), w, rows=rows.cuda(), out_dtype=out_dtype, err_flag=err)
    wide = torch.full((R, K + 24), float("nan"), dtype=dtype)
    wide[:, :K] = x[rows.long()]
    ordered = mx.linear_mxfp4_grouped(wide.cuda()[:, :K], off.cuda(), w, out_dtype=out_dtype, err_flag=err)
    assert int(err) == 0 and mx.mxfp8_device_fault_word() == 0
    assert torch.equal(got, ordered)
    for g in few:
        s = slice(int(off[g]), int(off[g + 1]))
        want, tol = bound(x[rows[s].long()], values(g), out_dtype == BF16)
        assert bool(((got[s].cpu().double() - want).abs() <= tol).all()), g


def test_few_rows_dropped_and_bad():
    G, N, K, R, T = 64, 200, 1096, 12, 5
    x, (w, values) = draw(T, K, BF16, 4).cuda(), few_experts(G, N, K)
    sizes = [0] * G
    sizes[2], sizes[33], sizes[63] = 1, 4, 3
    off = torch.tensor([0] + sizes).cumsum(0).cuda()
    rows = torch.tensor([4, 0, 1, 2, 2, 3, 4, 0, -1, -1, -1, -1], dtype=torch.int32, device="cuda")
    err = torch.zeros(1, dtype=torch.int32, device="cuda")

    def run(off, rows, x=x):
        out = torch.full((R + 2, N), 9.0, device="cuda")  # a guard behind the rows
        st = mx.mxfp4_linear_grouped(x, 0, x.shape[0], K, K, rows, R, G, off, w.codes, w.scales, N, out, 1, err, None)
        assert st == 0 and bool((out[R:] == 9).all()) and mx.mxfp8_device_fault_word() == 0
        return out[:R]
    good = run(off, rows)
    assert int(err) == 0 and bool((good[8:] == 0).all())
    for g, s in ((2, slice(0, 1)), (33, slice(1, 5)), (63, slice(5, 8))):
        want, tol = bound(x[rows[s].long()].cpu(), values(g), False)
        assert bool(((good[s].cpu().double() - want).abs() <= tol).all()), g
    lost = rows.clone()
    lost[9] = 2  # a row of no expert that is not marked
    assert torch.equal(run(off, lost), good) and int(err) == 1
    err.zero_()
    wrong = rows.clone()
    wrong[1], wrong[6] = T, -1
    got = run(off, wrong)
    keep = torch.ones(R, dtype=torch.bool)
    keep[[1, 6]] = False
    assert int(err) == 1 and bool(torch.isnan(got[[1, 6]]).all()) and torch.equal(got[keep], good[keep])
    for at, value in ((0, 1), (10, -1), (40, 2), (64, R + 1), (64, 1 << 62)):
        err.zero_()
        bad = off.clone()
        bad[at] = value
        assert bool((run(bad, rows) == 9).all()) and int(err) == 1, (at, value)
    err.zero_()
    bad_x = x.clone()
    bad_x[3, 77], bad_x[1, 5] = float("nan"), float("inf")
    got = run(off, rows, bad_x)
    assert bool(torch.isnan(got[[2, 5]]).all()) and int(err) == 0
    keep = torch.ones(R, dtype=torch.bool)
    keep[[2, 5]] = False
    assert torch.equal(got[keep], good[keep])
    none = torch.full((R,), -1, dtype=torch.int32, device="cuda")
    zero = mx.linear_mxfp4_grouped(x[:0], torch.zeros(G + 1, dtype=torch.int64, device="cuda"), w, rows=none, out_dtype=F32, err_flag=err)
    assert zero.shape == (R, N) and bool((zero == 0).all()) and int(err) == 0


def test_few_rows_repeat_and_follow_a_graph():
    G, N, K = 32, 520, 2048
    x, (w, _) = draw(8, K, BF16, 6).cuda(), few_experts(G, N, K)
    off = torch.zeros(G + 1, dtype=torch.int64, device="cuda")
    off[5:] = 3
    off[20:] = 8
    first = mx.linear_mxfp4_grouped(x, off, w, out_dtype=F32)
    for _ in range(5):
        assert torch.equal(mx.linear_mxfp4_grouped(x, off, w, out_dtype=F32), first)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = mx.linear_mxfp4_grouped(x, off, w, out_dtype=F32)
    moved = torch.zeros_like(off)
    moved[9:] = 8
    want = mx.linear_mxfp4_grouped(x, moved, w, out_dtype=F32)
    graph.replay()
    assert torch.equal(out, first)
    off.copy_(moved)
    graph.replay()
    assert torch.equal(out, want) and not torch.equal(out, first)


def test_the_largest_values():
    """What the parts add up to on the way is at most 7/3 of sum |x| |w|: below the end of fp32's range results are as accurate as
    anywhere, in one element and in sums that end far below their terms."""
    v = torch.arange(0x7E00, 0x7F80, dtype=torch.int32).to(torch.int16).view(BF16)  # from 2^125 on
    v = torch.cat((v, -v))
    x = torch.zeros(v.numel(), 64, dtype=BF16)
    x[:, 5] = v
    x[:, 6] = v / 2
    x[:, 40] = -v
    weight = torch.zeros(40, 64, dtype=BF16)
    weight[0, 5], weight[1, 6] = 1.0, 1.0
    weight[2, 5] = weight[2, 40] = 0.5  # the halves cancel
    weight[3, 5] = 0.25
    weight[39] = 0.0078125
    w, wv = mx.quantize_mxfp4(weight.cuda()).row, ref.cast(weight)
    for M in (2, 20, v.numel()):  # in the product's own kernel, by parts of a kernel before it, in pairs of CTAs
        for dtype in (BF16, F32):
            got = mx.linear_mxfp4(x[-M:].to(dtype).cuda(), w, F32).cpu().double()
            want, tol = bound(x[-M:], wv, False)
            inside = 7 / 3 * (x[-M:].double().abs() @ wv.double().abs().t()) < 2.0 ** 128
            assert bool(inside[:, [3, 39]].all()) and (M < v.numel() or bool(inside.any(0).all()))
            assert bool(((got - want).abs() <= tol)[inside].all()), (M, dtype)
    assert mx.mxfp8_device_fault_word() == 0
