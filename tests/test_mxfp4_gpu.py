"""MXFP4 cast and products against the 64-bit reference (tests/mxfp4_ref.py).

Codes, scale bytes and decoded values must be equal; a product's error is held to the bound that
mxfp4_ref.product_bound derives.
"""
import numpy as np
import pytest
import torch

import mxfp4_ref as ref
import mxfp8_block_scaled_04_gb300 as mx

pytestmark = pytest.mark.gpu

BF16, F32 = torch.bfloat16, torch.float32
GUARD = 4096


def draw(M, N, dtype, seed, spread=1.0):
    g = torch.Generator().manual_seed(seed)
    x = torch.randn(M, N, generator=g) * torch.exp(spread * torch.randn(M, 1, generator=g))
    return x.to(dtype)


def check_cast(x, rowwise=True, colwise=True):
    q = mx.quantize_mxfp4(x.cuda(), rowwise=rowwise, colwise=colwise)
    torch.cuda.synchronize()
    for m, src in ((q.row, x), (q.col, x.t())):
        if m is None:
            continue
        codes, scale = ref.quantize(src)
        assert (m.rows, m.cols) == tuple(src.shape)
        assert np.array_equal(m.codes.cpu().numpy(), codes)
        assert np.array_equal(m.scales.cpu().numpy(), ref.plane(scale))
        want = ref.values(codes, scale, src.shape[1])
        for dt in (BF16, F32):
            got = mx.dequantize_mxfp4(m, dt).cpu()
            assert torch.equal(torch.nan_to_num(got, nan=7e30), torch.nan_to_num(want.to(dt), nan=7e30))
    assert mx.mxfp8_device_fault_word() == 0


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("M,N", [(1, 8), (1, 32), (3, 40), (31, 72), (32, 128), (33, 136), (127, 248), (128, 256), (129, 264), (45, 80),
                                 (200, 1032), (1, 4096), (385, 8)])
def test_cast(M, N, dtype):
    check_cast(draw(M, N, dtype, M * 1000 + N))


@pytest.mark.parametrize("rowwise,colwise", [(True, False), (False, True)])
def test_cast_one_direction(rowwise, colwise):
    check_cast(draw(70, 168, BF16, 3), rowwise, colwise)


def test_cast_every_tie_and_boundary():
    """Every midpoint and level of the grid, one ulp to each side, at many scales; amax at and around 6 * 2^e."""
    mids = torch.tensor([0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0, 0.5, 1, 1.5, 2, 3, 4, 6])
    rows = []
    for e in (-126, -100, -3, 0, 1, 60, 120):
        for top in (6.0, float(np.nextafter(np.float32(6), np.float32(7))), 4.0, 3.0, float(np.nextafter(np.float32(3), np.float32(4)))):
            v = torch.cat((mids, torch.nextafter(mids, mids + 1), torch.tensor([top, 0.0, -0.0, -top])))
            v = torch.where(v.abs() > top, torch.full_like(v, top), v)
            rows.append((v * (-1.0) ** torch.arange(32)) * 2.0 ** e)
    check_cast(torch.stack(rows).repeat(1, 2))
    check_cast(torch.stack(rows).to(BF16))


def test_cast_extremes():
    """Zeros, subnormals of both types, the largest values, and blocks with NaN or infinities."""
    for dtype in (BF16, F32):
        x = draw(64, 64, F32, 5)
        x[0] = 0.0
        x[1] = -0.0
        x[2] *= 1e-39
        x[3] = 1e-45 if dtype == F32 else 1e-40
        x[4] *= 1e38
        x[5] = torch.finfo(dtype).max
        x[6, 3] = float("nan")
        x[7, 40] = float("inf")
        x[8, 63] = -float("inf")
        x[9] = torch.finfo(dtype).tiny
        check_cast(x.to(dtype))


@pytest.mark.parametrize("dtype", [BF16, F32])
def test_cast_strided_rows_and_guards(dtype):
    """Row pitch above N, outputs between canary bands that must stay untouched."""
    M, N = 77, 104
    big = draw(M, N + 24, dtype, 9).cuda()
    x = big[:, 8:8 + N]
    if dtype == BF16:
        assert x.data_ptr() % 16 == 0
    sizes = [M * mx.mxfp4_row_bytes(N), mx.mxfp4_scale_bytes(M, N), N * mx.mxfp4_row_bytes(M), mx.mxfp4_scale_bytes(N, M)]
    raw = [torch.full((n + 2 * GUARD,), 0xA5, dtype=torch.uint8, device="cuda") for n in sizes]
    view = [r[GUARD:GUARD + n] for r, n in zip(raw, sizes)]
    assert mx.mxfp4_quantize(x, 0 if dtype == BF16 else 1, M, N, N + 24, *view) == 0
    q = mx.quantize_mxfp4(x.contiguous(), colwise=True)
    for v, want in zip(view, (q.row.codes, q.row.scales, q.col.codes, q.col.scales)):
        assert torch.equal(v, want.flatten())
    for r in raw:
        assert bool((r[:GUARD] == 0xA5).all() and (r[-GUARD:] == 0xA5).all())
    assert torch.equal(mx.quantize_mxfp4(x).row.codes, q.row.codes)


def test_cast_noop_leaves_outputs():
    x = draw(40, 64, BF16, 1).cuda()
    codes = torch.full((40, 32), 0x33, dtype=torch.uint8, device="cuda")
    scales = torch.full((512,), 0x33, dtype=torch.uint8, device="cuda")
    assert mx.mxfp4_quantize(x, 0, 40, 64, 64, codes, scales, None, None, torch.ones(1, device="cuda")) == 0
    assert bool((codes == 0x33).all() and (scales == 0x33).all())
    assert mx.mxfp4_quantize(x, 0, 40, 64, 64, codes, scales, None, None, torch.zeros(1, device="cuda")) == 0
    assert torch.equal(codes, mx.quantize_mxfp4(x).row.codes)


# ---- products ------------------------------------------------------------------------------------------

def as_matrix(x):
    """x [R, C] as a 4-bit matrix; any C, through the transposed cast where C is no multiple of 8."""
    R, C = x.shape
    if C % 8 == 0:
        return mx.quantize_mxfp4(x.cuda()).row
    m = mx.quantize_mxfp4(torch.nn.functional.pad(x, (0, 0, 0, -R % 8)).t().contiguous().cuda(), False, True).col
    n = mx.mxfp4_scale_bytes(R, C)
    return mx.MXFP4Matrix(m.codes[:R].contiguous(), m.scales[:n].contiguous(), R, C)


def check_product(M, N, K, out_dtype, seed=0, a=None, b=None):
    a = draw(M, K, BF16, seed + 1) if a is None else a
    b = draw(N, K, BF16, seed + 2) if b is None else b
    qa, qb = as_matrix(a), as_matrix(b)
    got = mx.matmul_mxfp4(qa, qb, out_dtype).cpu().double()
    want, tol = ref.product_bound(ref.cast(a), ref.cast(b), out_dtype == BF16)
    assert mx.mxfp8_device_fault_word() == 0
    err = (got - want).abs()
    assert bool((err <= tol).all()), (float((err - tol).max()), float(err.max()))


@pytest.mark.parametrize("out_dtype", [BF16, F32])
@pytest.mark.parametrize("M,N,K", [(1, 1, 8), (2, 3, 1), (40, 50, 333), (1, 128, 256), (3, 5, 32), (16, 128, 64), (17, 130, 96), (33, 257, 136), (64, 64, 256),
                                   (128, 128, 512), (129, 383, 1000), (255, 256, 264), (300, 520, 2056), (1, 1000, 4096), (7, 3000, 8192)])
def test_product(M, N, K, out_dtype):
    check_product(M, N, K, out_dtype)


@pytest.mark.parametrize("M,N,K", [(1100, 1300, 512), (2049, 4100, 264)])
def test_product_many_tiles(M, N, K):
    """More tiles than CTAs: both accumulators and every stage are reused."""
    check_product(M, N, K, BF16)


def test_product_each_position_counts():
    """A one at each (row, k) in turn against weights that tell the positions apart: exact results."""
    K, N = 512, 64
    a = torch.zeros(K, K)
    a[torch.arange(K), torch.arange(K)] = 1.0
    b = torch.tensor([0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0, -6.0])[torch.randint(0, 8, (N, K), generator=torch.Generator().manual_seed(1))]
    b[:, ::32] = 6.0  # every block's scale is 1
    qa, qb = mx.quantize_mxfp4(a.to(BF16).cuda()).row, mx.quantize_mxfp4(b.to(BF16).cuda()).row
    got = mx.matmul_mxfp4(qa, qb, F32).cpu()
    want = ref.cast(a) @ ref.cast(b).t()
    assert torch.equal(got.double(), want)


def test_product_scales_of_every_block():
    """Constant codes, scales that differ by row and block of both operands."""
    M, N, K = 150, 200, 640
    g = torch.Generator().manual_seed(2)
    ea, eb = torch.randint(-6, 7, (M, K // 32), generator=g), torch.randint(-6, 7, (N, K // 32), generator=g)
    a, b = ((2.0 ** e.double()).repeat_interleave(32, 1) for e in (ea, eb))
    qa, qb = mx.quantize_mxfp4(a.float().cuda()).row, mx.quantize_mxfp4(b.float().cuda()).row
    got = mx.matmul_mxfp4(qa, qb, F32).cpu().double()
    want, tol = ref.product_bound(a, b, False)
    assert bool(((got - want).abs() <= tol).all())


def test_product_nan_block_reaches_its_rows_only():
    a, b = draw(40, 96, BF16, 1), draw(50, 96, BF16, 2)
    a[7, 40] = float("nan")
    b[9, 5] = float("inf")
    got = mx.matmul_mxfp4(mx.quantize_mxfp4(a.cuda()).row, mx.quantize_mxfp4(b.cuda()).row, F32).cpu()
    nan = torch.isnan(got)
    want = torch.zeros(40, 50, dtype=torch.bool)
    want[7] = True
    want[:, 9] = True
    assert torch.equal(nan, want)


@pytest.mark.parametrize("dtype", [BF16, F32])
def test_product_output_pitch_and_guards(dtype):
    M, N, K, ld = 37, 70, 160, 96
    qa, qb = mx.quantize_mxfp4(draw(M, K, BF16, 1).cuda()).row, mx.quantize_mxfp4(draw(N, K, BF16, 2).cuda()).row
    want = mx.matmul_mxfp4(qa, qb, dtype)
    buf = torch.full((M + 2, ld), 9.0, dtype=dtype, device="cuda")
    mx.matmul_mxfp4(qa, qb, out=buf[1:M + 1, :N])
    assert torch.equal(buf[1:M + 1, :N], want)
    assert bool((buf[0] == 9).all() and (buf[-1] == 9).all() and (buf[:, N:] == 9).all())


def test_product_empty_sizes():
    def m(r, c):
        return mx.quantize_mxfp4(torch.ones(r, c, dtype=BF16, device="cuda")).row
    assert mx.matmul_mxfp4(m(0, 64), m(8, 64)).shape == (0, 8)
    assert mx.matmul_mxfp4(m(8, 64), m(0, 64)).shape == (8, 0)
    assert bool((mx.matmul_mxfp4(m(5, 0), m(8, 0)) == 0).all())


@pytest.mark.parametrize("T,K,N", [(5, 64, 40), (67, 264, 136), (130, 512, 384)])
def test_linear_layer_gradients(T, K, N):
    """y = x W^T, dx = dy W, dw = dy^T x from the two forms of each cast, and against differences of the same
    quantized product: L = sum(dy * y) is linear in x's and W's quantized values, so steps of one level are exact."""
    x, w, dy = draw(T, K, BF16, 1), draw(N, K, BF16, 2, 0.0), draw(T, N, BF16, 3)
    qx, qw, qd = (mx.quantize_mxfp4(v.cuda(), colwise=True) for v in (x, w, dy))
    for got, a, b, dt in ((mx.matmul_mxfp4(qx.row, qw.row), ref.cast(x), ref.cast(w), BF16),
                          (mx.matmul_mxfp4(qd.row, qw.col), ref.cast(dy), ref.cast(w.t()), BF16),
                          (mx.matmul_mxfp4(qd.col, qx.col, F32), ref.cast(dy.t()), ref.cast(x.t()), F32)):
        want, tol = ref.product_bound(a, b, dt == BF16)
        assert bool(((got.cpu().double() - want).abs() <= tol).all())
    # differences: moving x[t, k]'s value by h moves y[t, :] by h * W[:, k], so dL/dx[t, k] = dy[t, :] . W[:, k]
    wv, dv, xv = ref.cast(w), ref.cast(dy), ref.cast(x)
    t, k, h = T // 2, K // 3, 0.25
    moved = xv.clone()
    moved[t, k] += h
    slope = ((moved @ wv.t() - xv @ wv.t()) * dv).sum() / h
    dx = (dv @ wv)[t, k]
    assert abs(slope - dx) <= 1e-9 * (dv[t].abs() @ wv[:, k].abs())


@pytest.mark.parametrize("out_dtype", [BF16, F32])
@pytest.mark.parametrize("M,N,K", [(2048, 2560, 256), (2300, 2433, 1064), (257, 20000, 320), (19500, 140, 96)])
def test_product_pair_tiles(M, N, K, out_dtype):
    """Sizes of the 256 x 256 tiles: whole, ragged in every dimension, several tiles per CTA pair."""
    check_product(M, N, K, out_dtype)


def test_product_pair_tiles_exact_positions():
    """Rows of P and Q that tell themselves apart (powers of two and small integers): exact results."""
    M, N, K = 2304, 2304, 512
    g = torch.Generator().manual_seed(4)
    lv = torch.tensor([0.0, 0.5, 1.0, -1.0, 2.0, 3.0, -4.0, 6.0])
    a, b = (lv[torch.randint(0, 8, (r, K), generator=g)] for r in (M, N))
    a[:, ::32] = 6.0
    b[:, ::32] = 6.0
    a *= 2.0 ** torch.randint(-2, 3, (M, 1), generator=g)
    b *= 2.0 ** torch.randint(-2, 3, (N, 1), generator=g)
    qa, qb = mx.quantize_mxfp4(a.cuda()).row, mx.quantize_mxfp4(b.cuda()).row
    got = mx.matmul_mxfp4(qa, qb, F32).cpu()
    assert torch.equal(got, a @ b.t())


# ---- experts' products -----------------------------------------------------------------------------------

def test_experts_product_pair_tiles():
    """Experts of several 256-row tiles, ragged, one of them empty."""
    test_experts_product([700, 0, 1025, 256, 3, 1700], 1416, 328, BF16)
    test_experts_product([5120, 1], 1000, 256, F32)


SIZES = [[5], [0, 3, 0], [128, 0, 1, 127, 129], [1] * 40, [300, 2, 0, 0, 61], [0, 0, 257]]


@pytest.mark.parametrize("out_dtype", [BF16, F32])
@pytest.mark.parametrize("N,K", [(40, 72), (264, 520), (128, 256)])
@pytest.mark.parametrize("sizes", SIZES)
def test_experts_product(sizes, N, K, out_dtype):
    G, R = len(sizes), sum(sizes)
    T = max(1, R // 2)
    x, w = draw(T, K, BF16, 1), draw(G * N, K, BF16, 2)
    g = torch.Generator().manual_seed(3)
    rows = torch.randint(0, T, (R,), generator=g, dtype=torch.int32)
    off = torch.tensor([0] + sizes).cumsum(0)
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    qa = mx.quantize_mxfp4_grouped(x.cuda(), off.cuda(), rows=rows.cuda(), err_flag=err)
    codes, scale = ref.quantize(x[rows.long()])
    assert np.array_equal(qa.codes.cpu().numpy(), codes)
    planes = np.concatenate([ref.plane(scale[off[g]:off[g + 1]]) for g in range(G)]) if R else np.zeros(0, np.uint8)
    assert np.array_equal(qa.scales.cpu().numpy()[:planes.size], planes)
    parts = [mx.quantize_mxfp4(w[g * N:(g + 1) * N].cuda()).row for g in range(G)]
    qb = mx.MXFP4Matrix(torch.stack([p.codes for p in parts]), torch.stack([p.scales for p in parts]), N, K)
    got = mx.matmul_mxfp4_grouped(qa, off.cuda(), qb, out_dtype, err_flag=err).cpu().double()
    assert int(err) == 0 and mx.mxfp8_device_fault_word() == 0
    xv = ref.cast(x)[rows.long()]
    for g in range(G):
        s = slice(int(off[g]), int(off[g + 1]))
        want, tol = ref.product_bound(xv[s], ref.cast(w[g * N:(g + 1) * N]), out_dtype == BF16)
        assert bool(((got[s] - want).abs() <= tol).all()), g


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("N", [8, 72, 1032])
@pytest.mark.parametrize("sizes", SIZES)
def test_grouped_cast_forms(sizes, N, dtype):
    """Gathered with and without a workspace (several rows per token and fewer rows than tokens), and in order: the
    same codes and planes; rows from a larger pitch."""
    G, R = len(sizes), sum(sizes)
    off = torch.tensor([0] + sizes).cumsum(0)
    for T in (max(1, R // 3), 2 * R + 1):
        big = draw(T, N + 16, dtype, T + N)
        x = big[:, 8:8 + N]
        rows = torch.randint(0, T, (R,), generator=torch.Generator().manual_seed(T), dtype=torch.int32)
        rows[R // 2] = T  # outside
        codes, scale = ref.quantize(x[rows.long().clamp(max=T - 1)])
        codes[R // 2] = 0
        scale[R // 2] = 255
        planes = np.concatenate([ref.plane(scale[off[g]:off[g + 1]]) for g in range(G)])
        nbytes = mx.mxfp4_grouped_scale_bytes(R, N, G)
        for ws in (False, True):
            err = torch.zeros(1, dtype=torch.int32, device="cuda")
            out = torch.full((R, mx.mxfp4_row_bytes(N)), 0x77, dtype=torch.uint8, device="cuda")
            plane = torch.full((nbytes,), 0x77, dtype=torch.uint8, device="cuda")
            need = mx.mxfp4_quantize_grouped_workspace_bytes(T, N, R)
            work = torch.empty(max(need, 16), dtype=torch.uint8, device="cuda") if ws else None
            xc = big.cuda()[:, 8:8 + N]
            assert mx.mxfp4_quantize_grouped(xc, 0 if dtype == BF16 else 1, T, N, N + 16, rows.cuda(), R, G, off.cuda(), out, plane,
                                             err, work) == 0
            assert int(err) == 1
            assert np.array_equal(out.cpu().numpy(), codes)
            assert np.array_equal(plane.cpu().numpy()[:planes.size], planes)
    ordered = draw(R, N, dtype, 1)
    q = mx.quantize_mxfp4_grouped(ordered.cuda(), off.cuda())
    codes, scale = ref.quantize(ordered)
    planes = np.concatenate([ref.plane(scale[off[g]:off[g + 1]]) for g in range(G)])
    assert np.array_equal(q.codes.cpu().numpy(), codes) and np.array_equal(q.scales.cpu().numpy()[:planes.size], planes)


@pytest.mark.parametrize("rows,cols", [(1, 1), (5, 7), (9, 31), (130, 33), (17, 65), (70, 1023), (3, 4093)])
def test_decode_any_width(rows, cols):
    """Rows of the output that start off a 16-byte boundary, and blocks that end inside a thread's elements."""
    x = draw(cols + (-cols % 8), rows + (-rows % 8), F32, rows + cols)[:, :rows + (-rows % 8)]
    x[cols:] = 0
    m = mx.quantize_mxfp4(x.cuda(), False, True).col      # [rows padded to 8, cols padded to 8]
    m = mx.MXFP4Matrix(m.codes[:rows].contiguous(), m.scales[:mx.mxfp4_scale_bytes(rows, cols)].contiguous(), rows, cols)
    want = ref.cast(x.t())[:rows, :cols]
    for dt in (BF16, F32):
        assert torch.equal(mx.dequantize_mxfp4(m, dt).cpu(), want.to(dt))


def test_experts_bad_offsets_and_rows_set_the_flag():
    x = draw(6, 64, BF16, 1).cuda()
    w = mx.quantize_mxfp4(draw(32, 64, BF16, 2).cuda()).row
    wb = mx.MXFP4Matrix(w.codes[None].repeat(2, 1, 1), w.scales[None].repeat(2, 1), 32, 64)
    good = torch.tensor([0, 2, 6], device="cuda")
    qa = mx.quantize_mxfp4_grouped(x, good)
    for bad in ([0, 7, 6], [1, 2, 6], [0, 2, 5]):
        err = torch.zeros(1, dtype=torch.int32, device="cuda")
        mx.quantize_mxfp4_grouped(x, torch.tensor(bad, device="cuda"), err_flag=err)
        assert int(err) == 1, bad
        err.zero_()
        mx.matmul_mxfp4_grouped(qa, torch.tensor(bad, device="cuda"), wb, err_flag=err)
        assert int(err) == 1, bad
    # a row index outside x: NaN in that row alone, and the flag
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    rows = torch.tensor([0, 6, 2, -1, 4, 5], dtype=torch.int32, device="cuda")
    y = mx.matmul_mxfp4_grouped(mx.quantize_mxfp4_grouped(x, good, rows=rows, err_flag=err), good, wb)
    assert int(err) == 1
    assert torch.isnan(y).all(1).tolist() == [False, True, False, True, False, False]
    assert torch.isnan(y).any(1).tolist() == [False, True, False, True, False, False]


def test_products_on_another_stream_and_in_a_graph():
    x, w = draw(50, 256, BF16, 1).cuda(), draw(96, 256, BF16, 2).cuda()
    want = mx.matmul_mxfp4(mx.quantize_mxfp4(x).row, mx.quantize_mxfp4(w).row)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    got = mx.matmul_mxfp4(mx.quantize_mxfp4(x, stream=side).row, mx.quantize_mxfp4(w, stream=side).row, stream=side)
    side.synchronize()
    assert torch.equal(got, want)
    qw = mx.quantize_mxfp4(w).row
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        y = mx.matmul_mxfp4(mx.quantize_mxfp4(x).row, qw)
    x.copy_(x.flip(0))
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(y, want.flip(0))


def test_past_2_32_elements():
    """Offsets beyond 32 bits: the ends of a cast, a decode and a product of more than 2^32 elements equal those of
    the same rows and columns on their own."""
    M, N = 66048, 65664
    assert M * N > 1 << 32
    x = torch.empty((M, N), dtype=BF16, device="cuda").normal_()
    q = mx.quantize_mxfp4(x, colwise=True)
    tail, right = x[-256:].clone(), x[:, -256:].contiguous()
    small = mx.quantize_mxfp4(tail, colwise=True)
    assert torch.equal(q.row.codes[-256:], small.row.codes) and torch.equal(q.row.scales[-small.row.scales.numel():], small.row.scales)
    assert torch.equal(q.col.codes[:, -128:], small.col.codes)
    small = mx.quantize_mxfp4(right, colwise=True)
    assert torch.equal(q.row.codes[:, -128:], small.row.codes)
    assert torch.equal(q.col.codes[-256:], small.col.codes) and torch.equal(q.col.scales[-small.col.scales.numel():], small.col.scales)
    del x, right, small
    v = mx.dequantize_mxfp4(q.row)
    assert torch.equal(v[-256:], mx.dequantize_mxfp4(mx.quantize_mxfp4(tail).row))
    del v, q, tail
    torch.cuda.empty_cache()
    K = 64
    a, b = torch.randn(M, K, device="cuda").to(BF16), torch.randn(N, K, device="cuda").to(BF16)
    y = mx.matmul_mxfp4(mx.quantize_mxfp4(a).row, mx.quantize_mxfp4(b).row)
    for rows, cols in ((slice(M - 300, M), slice(N - 300, N)), (slice(0, 300), slice(N - 300, N)), (slice(M - 300, M), slice(0, 300))):
        part = mx.matmul_mxfp4(mx.quantize_mxfp4(a[rows].contiguous()).row, mx.quantize_mxfp4(b[cols].contiguous()).row)
        assert torch.equal(y[rows, cols], part)
    del y
    torch.cuda.empty_cache()


def fuzz_shapes(seed, count):
    rng = np.random.default_rng(seed)
    for _ in range(count):
        M = int(np.exp(rng.uniform(0, np.log(3000))))
        N = int(np.exp(rng.uniform(0, np.log(9000))))
        K = 8 * int(np.exp(rng.uniform(0, np.log(900))))
        yield M, N, K, BF16 if rng.random() < 0.5 else F32


def bound_on_gpu(a, b, bf16):
    """ref.product_bound of decoded matrices, on the GPU in 64 bits."""
    return ref.product_bound(mx.dequantize_mxfp4(a, F32).double(), mx.dequantize_mxfp4(b, F32).double(), bf16)


@pytest.mark.parametrize("seed", range(3))
def test_product_fuzz(seed):
    """Random sizes over every kernel and split of K, against 64 bits of the decoded operands."""
    for M, N, K, dt in fuzz_shapes(seed, 25):
        g = torch.Generator(device="cuda").manual_seed(M + N + K)
        a, b = (mx.quantize_mxfp4(torch.randn(r, K, generator=g, device="cuda").to(BF16)).row for r in (M, N))
        want, tol = bound_on_gpu(a, b, dt == BF16)
        got = mx.matmul_mxfp4(a, b, dt).double()
        assert bool(((got - want).abs() <= tol).all()), (M, N, K, dt)
    assert mx.mxfp8_device_fault_word() == 0


@pytest.mark.parametrize("seed", range(3))
def test_experts_product_fuzz(seed):
    """Random experts, loads and sizes over both experts' kernels."""
    rng = np.random.default_rng(100 + seed)
    for _ in range(8):
        G, N, K = int(rng.integers(1, 33)), int(np.exp(rng.uniform(0, 7.3))), 8 * int(np.exp(rng.uniform(0, 5.5)))
        sizes = (rng.integers(0, 2, G) * np.exp(rng.uniform(0, rng.uniform(1, 6.5), G))).astype(int)
        off = torch.tensor(np.concatenate([[0], np.cumsum(sizes)]), device="cuda")
        R = int(off[-1])
        dt = BF16 if rng.random() < 0.5 else F32
        g = torch.Generator(device="cuda").manual_seed(seed)
        x = torch.randn(R, K, generator=g, device="cuda").to(BF16)
        w = [mx.quantize_mxfp4(torch.randn(N, K, generator=g, device="cuda").to(BF16)).row for _ in range(G)]
        qb = mx.MXFP4Matrix(torch.stack([m.codes for m in w]), torch.stack([m.scales for m in w]), N, K)
        got = mx.matmul_mxfp4_grouped(mx.quantize_mxfp4_grouped(x, off), off, qb, dt).double()
        xa = mx.quantize_mxfp4(x).row if R else None
        for e in range(G):
            s = slice(int(off[e]), int(off[e + 1]))
            if s.start == s.stop:
                continue
            rows = mx.dequantize_mxfp4(xa, F32).double()[s]
            want, tol = ref.product_bound(rows, mx.dequantize_mxfp4(w[e], F32).double(), dt == BF16)
            assert bool(((got[s] - want).abs() <= tol).all()), (G, N, K, e)
    assert mx.mxfp8_device_fault_word() == 0


def test_results_are_the_same_bits_every_time():
    """Casts, split and paired products and experts' products repeat exactly."""
    for M, N, K in ((1, 2048, 8192), (100, 512, 16384), (1024, 4096, 1024)):
        a, b = (mx.quantize_mxfp4(torch.randn(r, K, device="cuda").to(BF16)).row for r in (M, N))
        first = mx.matmul_mxfp4(a, b, F32)
        for _ in range(5):
            assert torch.equal(mx.matmul_mxfp4(a, b, F32), first)


def test_concurrent_streams():
    """Products of every kernel on four streams at once: each result equals the one computed alone."""
    jobs = []
    for M, N, K in ((1, 4096, 4096), (300, 1024, 2048), (2048, 2048, 512), (64, 8192, 1024)):
        a, b = (mx.quantize_mxfp4(torch.randn(r, K, device="cuda").to(BF16)).row for r in (M, N))
        jobs.append((a, b, mx.matmul_mxfp4(a, b)))
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in jobs]
    outs = []
    for _ in range(10):
        for st, (a, b, _) in zip(streams, jobs):
            outs.append(mx.matmul_mxfp4(a, b, stream=st))
    torch.cuda.synchronize()
    for i, out in enumerate(outs):
        assert torch.equal(out, jobs[i % len(jobs)][2])
    assert mx.mxfp8_device_fault_word() == 0
