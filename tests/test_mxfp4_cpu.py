"""Host-side checks of include/mxfp4.h and include/moe.h and of the 64-bit reference; no GPU needed.

Every rejection below is decided on the host before the library touches the device.
"""
import ctypes
import os
import re
import subprocess

import numpy as np
import pytest
import torch

import mxfp4_ref as ref
import mxfp8_block_scaled_04_gb300 as mx

INCLUDE = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "include")
OK, NULL, SHAPE, ALIGN, FORMAT, WORKSPACE, DEVICE, LAUNCH, GROUPS = range(9)
A = 1 << 20  # a fake, 16-byte aligned address: never dereferenced by these calls


def test_library_exports_every_declared_symbol(cuda_lib):
    for header in ("mxfp4.h", "moe.h"):
        text = re.sub(r"/\*.*?\*/", "", open(os.path.join(INCLUDE, header)).read(), flags=re.S)
        names = set(re.findall(r"\b((?:mxfp4|moe)_\w+)\s*\(", text))
        assert len(names) >= 6, names
        for n in names:
            assert ctypes.cast(getattr(cuda_lib, n), ctypes.c_void_p).value, n


def test_headers_compile_as_c_and_the_config_layout_matches(tmp_path):
    src = tmp_path / "probe.c"
    fields = [f for f, _ in mx.RouteConfig._fields_]
    src.write_text('#include <stdio.h>\n#include <stddef.h>\n#include "moe.h"\n'
                   '#define F(f) printf(" %zu", offsetof(moe_route_config_t, f));\n'
                   'int main(void){ printf("%zu", sizeof(moe_route_config_t)); ' + " ".join(f"F({f})" for f in fields) +
                   ' return 0; }\n')
    exe = tmp_path / "probe"
    subprocess.run(["gcc", "-std=c99", "-Wall", "-Werror", "-pedantic", "-I", INCLUDE, str(src), "-o", str(exe)], check=True)
    got = [int(v) for v in subprocess.run([str(exe)], capture_output=True, text=True, check=True).stdout.split()]
    assert got == [ctypes.sizeof(mx.RouteConfig)] + [getattr(mx.RouteConfig, f).offset for f in fields]


@pytest.mark.parametrize("rows,cols", [(0, 8), (1, 1), (1, 32), (127, 33), (128, 128), (129, 136), (4093, 7176)])
def test_sizes_agree_with_the_library(cuda_lib, rows, cols):
    assert mx.mxfp4_row_bytes(cols) == cuda_lib.mxfp4_row_bytes(cols) == -(-cols // 32) * 16
    assert mx.mxfp4_scale_bytes(rows, cols) == cuda_lib.mxfp4_scale_bytes(rows, cols)
    for g in (1, 3, 512):
        assert mx.mxfp4_grouped_scale_bytes(rows, cols, g) == cuda_lib.mxfp4_grouped_scale_bytes(rows, cols, g)
    for total in (rows, rows + 5):
        assert (mx.mxfp4_quantize_grouped_workspace_bytes(rows, cols, total) ==
                cuda_lib.mxfp4_quantize_grouped_workspace_bytes(rows, cols, total))


def test_grouped_scale_bytes_hold_any_offsets(cuda_lib):
    """The bound covers every split of the rows: sum over groups of ceil(rows_g / 128) row tiles."""
    rng = np.random.default_rng(0)
    for _ in range(300):
        total, groups = int(rng.integers(1, 700)), int(rng.integers(1, 40))
        cuts = np.sort(rng.integers(0, total + 1, groups - 1))
        sizes = np.diff(np.concatenate([[0], cuts, [total]]))
        need = int(np.sum(-(-sizes // 128))) * 512 * 2
        assert need <= mx.mxfp4_grouped_scale_bytes(total, 200, groups)


def quantize(x=A, t=0, M=64, N=64, ld=64, r=A, rs=A, c=A, cs=A, noop=None):
    return mx.mxfp4_quantize(x, t, M, N, ld, r, rs, c, cs, noop, 0)


@pytest.mark.parametrize("kw,status", [
    (dict(t=2), FORMAT), (dict(t=-1), FORMAT), (dict(M=-1), SHAPE), (dict(N=36), SHAPE), (dict(ld=56), SHAPE), (dict(ld=68), SHAPE),
    (dict(N=1 << 31, ld=1 << 31), SHAPE), (dict(x=None), NULL), (dict(r=None), NULL), (dict(cs=None), NULL),
    (dict(r=None, rs=None, c=None, cs=None), NULL), (dict(x=A + 8), ALIGN), (dict(r=A + 8), ALIGN), (dict(c=A + 4), ALIGN),
    (dict(rs=A + 2), ALIGN), (dict(cs=A + 1), ALIGN), (dict(noop=A + 2), ALIGN), (dict(), DEVICE), (dict(M=0, x=None), None),
])
def test_quantize_rejections(cuda_lib, kw, status):
    got = quantize(**kw)
    assert got == status if status is not None else got in (OK, DEVICE)


def grouped(x=A, t=0, T=10, N=64, ld=64, rows=A, total=20, G=2, off=A, out=A, sc=A, err=None, ws=None):
    return mx.mxfp4_quantize_grouped(x, t, T, N, ld, rows, total, G, off, out, sc, err, ws, 0)


@pytest.mark.parametrize("kw,status", [
    (dict(t=5), FORMAT), (dict(T=-1), SHAPE), (dict(total=-1), SHAPE), (dict(N=12), SHAPE), (dict(ld=32), SHAPE),
    (dict(rows=None), SHAPE), (dict(G=0), GROUPS), (dict(G=513), GROUPS), (dict(off=None), GROUPS), (dict(out=None), NULL),
    (dict(sc=None), NULL), (dict(x=None), NULL), (dict(rows=A + 2), ALIGN), (dict(off=A + 4), ALIGN), (dict(err=A + 1), ALIGN),
    (dict(ws=A + 8), ALIGN), (dict(), DEVICE), (dict(ws=A), DEVICE),
])
def test_quantize_grouped_rejections(cuda_lib, kw, status):
    assert grouped(**kw) == status


def matmul(a=A, sa=A, M=5, b=A, sb=A, N=7, K=64, out=A, t=0, ldo=7):
    return mx.mxfp4_matmul(a, sa, M, b, sb, N, K, out, t, ldo, 0)


@pytest.mark.parametrize("kw,status", [
    (dict(t=2), FORMAT), (dict(M=-1), SHAPE), (dict(N=-1), SHAPE), (dict(K=-8), SHAPE), (dict(ldo=6), SHAPE), (dict(M=1 << 31), SHAPE),
    (dict(a=None), NULL), (dict(sa=None), NULL), (dict(b=None), NULL), (dict(sb=None), NULL), (dict(out=None), NULL),
    (dict(a=A + 8), ALIGN), (dict(sa=A + 4), ALIGN), (dict(b=A + 8), ALIGN), (dict(sb=A + 8), ALIGN), (dict(out=A + 1), ALIGN),
    (dict(out=A + 2, t=1), ALIGN), (dict(), DEVICE), (dict(K=63), DEVICE), (dict(K=0, a=None, sa=None, b=None, sb=None), DEVICE),
])
def test_matmul_rejections(cuda_lib, kw, status):
    assert matmul(**kw) == status


def matmul_grouped(total=5, G=2, off=A, N=7, K=64, out=A, t=0, err=None, a=A, b=A):
    return mx.mxfp4_matmul_grouped(a, A, total, G, off, b, A, N, K, out, t, err, 0)


@pytest.mark.parametrize("kw,status", [
    (dict(t=3), FORMAT), (dict(total=-1), SHAPE), (dict(N=1 << 30, G=4), SHAPE), (dict(G=0), GROUPS), (dict(G=600), GROUPS),
    (dict(off=None), GROUPS), (dict(off=A + 4), ALIGN), (dict(err=A + 2), ALIGN), (dict(a=None), NULL), (dict(b=A + 8), ALIGN),
    (dict(), DEVICE),
])
def test_matmul_grouped_rejections(cuda_lib, kw, status):
    assert matmul_grouped(**kw) == status


def test_dequantize_rejections(cuda_lib):
    def d(c=A, s=A, R=4, C=40, out=A, t=0):
        return mx.mxfp4_dequantize(c, s, R, C, out, t, 0)
    assert d(t=2) == FORMAT and d(R=-1) == SHAPE and d(C=1 << 31) == SHAPE
    assert d(c=None) == NULL and d(s=None) == NULL and d(out=None) == NULL
    assert d(c=A + 8) == ALIGN and d(out=A + 8) == ALIGN and d(C=37) == DEVICE


def route(E=64, k=4, T=3, ld=None, t=0, logits=A, idx=A, w=A, cfg=None, **kw):
    cfg = mx.make_route_config(k, **kw) if cfg is None else cfg
    return mx.moe_route_c(logits, t, T, E, E if ld is None else ld, cfg, idx, w, 0)


@pytest.mark.parametrize("kw,status", [
    (dict(t=2), FORMAT), (dict(score=2), FORMAT), (dict(T=-1), SHAPE), (dict(E=0), SHAPE), (dict(E=513), GROUPS), (dict(ld=63), SHAPE),
    (dict(k=0), SHAPE), (dict(k=33), SHAPE), (dict(E=3, k=4), SHAPE), (dict(groups=0), GROUPS), (dict(groups=5), GROUPS),
    (dict(groups=8, topk_groups=9), GROUPS), (dict(groups=8, topk_groups=0), GROUPS), (dict(groups=32, topk_groups=1), SHAPE),
    (dict(logits=None), NULL), (dict(idx=None), NULL), (dict(w=None), NULL), (dict(logits=A + 1), ALIGN), (dict(idx=A + 2), ALIGN),
    (dict(w=A + 1), ALIGN), (dict(), DEVICE),
])
def test_route_rejections(cuda_lib, kw, status):
    assert route(**kw) == status


def test_route_config_rejections(cuda_lib):
    assert mx.moe_route_c(A, 0, 3, 64, 64, None, A, A, 0) == NULL
    cfg = mx.make_route_config(4)
    cfg.reserved[1] = 1
    assert route(cfg=cfg) == FORMAT
    cfg = mx.make_route_config(4)
    cfg.renormalize = 2
    assert route(cfg=cfg) == FORMAT
    back = mx.moe_route_backward_c
    cfg = mx.make_route_config(4)
    assert back(A, 0, 3, 64, 64, cfg, None, A, A, 0) == NULL and back(A, 0, 3, 64, 64, cfg, A, None, A, 0) == NULL
    assert back(A, 0, 3, 64, 64, cfg, A, A, A + 1, 0) == ALIGN and back(A, 0, 3, 64, 64, cfg, A, A, A, 0) == DEVICE
    assert back(A, 1, 3, 2, 2, cfg, A, A, A, 0) == SHAPE


def test_plan_and_combine_rejections(cuda_lib):
    def p(i=A, n=8, k=2, E=4, o=A, s=A, t=A, ws=A):
        return mx.moe_plan_c(i, n, k, E, o, s, t, ws, 0)
    assert p(n=-2) == SHAPE and p(n=7) == SHAPE and p(k=0) == SHAPE and p(k=33, n=33) == SHAPE
    assert p(E=0) == GROUPS and p(E=513) == GROUPS and p(o=None) == GROUPS
    assert p(i=None) == NULL and p(s=None) == NULL and p(t=None) == NULL
    assert p(o=A + 4) == ALIGN and p(s=A + 2) == ALIGN and p() == DEVICE
    assert p(n=1 << 20, ws=None) == WORKSPACE and mx.moe_plan_workspace_bytes(1 << 20, 4) > 0
    assert mx.moe_plan_workspace_bytes(8, 4) == 0 and mx.moe_plan_workspace_bytes(8, 0) == 0

    def c(y=A, R=8, H=16, s=A, w=A, T=4, k=2, out=A):
        return mx.moe_combine_c(y, R, H, s, w, T, k, out, 0)
    assert c(H=12) == SHAPE and c(R=-1) == SHAPE and c(k=33) == SHAPE and c(T=-1) == SHAPE
    assert c(y=None) == NULL and c(s=None) == NULL and c(out=None) == NULL
    assert c(y=A + 8) == ALIGN and c(out=A + 2) == ALIGN and c(w=A + 2) == ALIGN and c() == DEVICE and c(w=None) == DEVICE

    def b(d=A, y=A, R=8, H=16, s=A, w=A, T=4, k=2, dy=A, dw=A):
        return mx.moe_combine_backward_c(d, y, R, H, s, w, T, k, dy, dw, 0)
    assert b(dy=None, dw=None) == NULL and b(y=None) == NULL and b(d=None) == NULL
    assert b(y=None, dw=None) == DEVICE and b(dy=A + 8) == ALIGN and b() == DEVICE


def test_wrappers_refuse_bad_tensors(cuda_lib):
    bf, f32, i32 = torch.bfloat16, torch.float32, torch.int32
    m = mx.MXFP4Matrix(torch.zeros(4, 32, dtype=torch.uint8), torch.zeros(512, dtype=torch.uint8), 4, 64)
    x = torch.zeros(4, 64, dtype=bf)
    off = torch.tensor([0, 4])
    for call in (
            lambda: mx.quantize_mxfp4(torch.zeros(4, 64, dtype=torch.float16)),
            lambda: mx.quantize_mxfp4(torch.zeros(64, 4, dtype=bf).t()),
            lambda: mx.quantize_mxfp4(torch.zeros(4, dtype=bf)),
            lambda: mx.quantize_mxfp4_grouped(x, off.int()),
            lambda: mx.quantize_mxfp4_grouped(x, off, rows=torch.zeros(4, dtype=torch.int64)),
            lambda: mx.quantize_mxfp4_grouped(x, off, err_flag=torch.zeros(1)),
            lambda: mx.dequantize_mxfp4(m, torch.float16),
            lambda: mx.dequantize_mxfp4(m._replace(cols=96)),
            lambda: mx.dequantize_mxfp4(m._replace(scales=m.scales[:100])),
            lambda: mx.matmul_mxfp4(m, m._replace(cols=32, codes=m.codes[:, :16].contiguous())),
            lambda: mx.matmul_mxfp4(m, m, out_dtype=torch.float16),
            lambda: mx.matmul_mxfp4(m, m, out=torch.zeros(4, 5, dtype=bf)),
            lambda: mx.matmul_mxfp4_grouped(m, off, m),
            lambda: mx.matmul_mxfp4(m._replace(groups=1), m),
            lambda: mx.dequantize_mxfp4(m._replace(groups=2)),
            lambda: mx.matmul_mxfp4_grouped(m._replace(groups=2), off, m._replace(codes=m.codes[None], scales=m.scales[None])),
            lambda: mx.moe_route(torch.zeros(3, 8, dtype=torch.float64), 2),
            lambda: mx.moe_route(torch.zeros(3, 8), 2, bias=torch.zeros(7)),
            lambda: mx.moe_route_backward(torch.zeros(3, 8), torch.zeros(3, 2, dtype=i32), torch.zeros(3, 3)),
            lambda: mx.moe_route_backward(torch.zeros(3, 8), torch.zeros(4, 2, dtype=i32), torch.zeros(4, 2)),
            lambda: mx.moe_plan(torch.zeros(3, 2), 8),
            lambda: mx.moe_combine(torch.zeros(6, 8), torch.zeros(3, 2, dtype=i32)),
            lambda: mx.moe_combine(torch.zeros(6, 8, dtype=bf), torch.zeros(3, 2, dtype=i32), torch.zeros(3, 1)),
            lambda: mx.moe_combine_backward(torch.zeros(3, 16, dtype=bf), torch.zeros(6, 8, dtype=bf), torch.zeros(3, 2, dtype=i32))):
        with pytest.raises(ValueError):
            call()
    with pytest.raises(KeyError):
        mx.moe_route(torch.zeros(3, 8), 2, score="tanh")


# ---- the reference itself ------------------------------------------------------------------------------------

def test_reference_encodes_every_level_and_tie():
    want = {0.0: 0, 0.25: 0, 0.26: 1, 0.5: 1, 0.74: 1, 0.75: 2, 1.0: 2, 1.25: 2, 1.26: 3, 1.75: 4, 2.5: 4, 2.6: 5, 3.0: 5, 3.5: 6, 4.9: 6,
            5.0: 6, 5.01: 7, 6.0: 7}
    v = np.array(list(want))
    assert ref.encode(v).tolist() == list(want.values())
    assert ref.encode(-v).tolist() == [c + 8 for c in want.values()]


def test_reference_scale_is_the_smallest_that_fits():
    for amax in (6.0, 6.0001, 3.0, 3.1, 1e-30, 4e30, 2.0 ** -126):
        e = ref.block_exponent(amax)
        assert amax <= 6 * 2.0 ** e and (amax > 6 * 2.0 ** (e - 1) or e == -127)
    assert ref.block_exponent(0.0) == 0


def test_reference_layouts_round_trip():
    x = torch.randn(150, 200, generator=torch.Generator().manual_seed(0), dtype=torch.float64)
    codes, scale = ref.quantize(x)
    assert codes.shape == (150, 112) and scale.shape == (150, 7)
    plane = ref.plane(scale)
    assert plane.size == mx.mxfp4_scale_bytes(150, 200)
    # element (r, b) where include/mxfp4.h puts it, spot-checked by hand
    assert plane[(0 * 2 + 0) * 512 + 16 * 5 + 4 * 2 + 3] == scale[69, 3]
    assert plane[(1 * 2 + 1) * 512 + 16 * 21 + 4 * 0 + 2] == scale[149, 6]
    v = ref.values(codes, scale, 200)
    assert float((v - x).abs().max()) <= float(x.abs().max()) / 6  # half the widest gap over the largest level
    assert torch.equal(ref.cast(v), v)                             # a cast value casts to itself


def overlapping_rows(rows, cols, dtype):
    """[rows, cols] views whose rows share elements: one row repeated (the gradient of a sum over rows), and rows that
    start half a row apart."""
    yield torch.zeros(1, cols, dtype=dtype).expand(rows, cols)
    yield torch.zeros((rows + 1) * cols, dtype=dtype).as_strided((rows, cols), (cols // 2, 1))


@pytest.mark.parametrize("form", [0, 1])
def test_wrappers_refuse_rows_that_overlap(cuda_lib, form):
    """A row stride below the row's length is not a pitch: read as whole rows it runs past the tensor's storage."""
    bf, i32 = torch.bfloat16, torch.int32
    x = list(overlapping_rows(40, 64, bf))[form]
    assert x.stride(0) < 64 and x.stride(1) == 1
    logits = list(overlapping_rows(40, 8, torch.float32))[form]
    off = torch.tensor([0, 40])
    m = mx.MXFP4Matrix(torch.zeros(40, 32, dtype=torch.uint8), torch.zeros(512, dtype=torch.uint8), 40, 64)
    w = mx.MXFP4Matrix(torch.zeros(64, 32, dtype=torch.uint8), torch.zeros(512, dtype=torch.uint8), 64, 64)
    for call in (
            lambda: mx.quantize_mxfp4(x),
            lambda: mx.quantize_mxfp4(x.float().new_zeros(1, 64).expand(40, 64), colwise=True),
            lambda: mx.quantize_mxfp4_grouped(x, off),
            lambda: mx.quantize_mxfp4_grouped(x, off, rows=torch.zeros(40, dtype=i32)),
            lambda: mx.moe_route(logits, 2),
            lambda: mx.moe_route_backward(logits, torch.zeros(40, 2, dtype=i32), torch.zeros(40, 2)),
            lambda: mx.matmul_mxfp4(m, w, out=x)):
        with pytest.raises(ValueError, match="contiguous rows"):
            call()


def test_wrappers_take_rows_of_a_larger_pitch_and_single_rows(cuda_lib):
    """Row strides of at least a row stay accepted (the library then refuses these tensors for being off the GPU)."""
    x = torch.zeros(40, 96, dtype=torch.bfloat16)[:, 8:72]
    row = torch.zeros(64, dtype=torch.bfloat16).as_strided((1, 64), (3, 1))  # the stride of one row means nothing
    for t in (x, row, x.contiguous()):
        with pytest.raises(mx.MXFP8Error) as error:
            mx.quantize_mxfp4(t)
        assert error.value.status == DEVICE


def test_a_matrix_keeps_its_size(cuda_lib):
    """The scales' address follows from the size at the cast, so that the size cannot be changed under it."""
    cast = mx.MXFP4Matrix._in(torch.zeros(64 * 32 + 512, dtype=torch.uint8), 0, 64, 64, 512)
    held = mx.MXFP4Matrix(cast.codes, cast.scales, 64, 64)
    for m in (cast, held):
        for name in ("rows", "cols", "groups"):
            with pytest.raises(AttributeError):
                setattr(m, name, 10)
        assert (m.rows, m.cols, m.groups) == (64, 64, None)
    # a shorter matrix is another one, whose tensors are given
    short = cast._replace(rows=10, codes=cast.codes[:10])
    assert short.rows == 10 and short.scales.data_ptr() == cast.scales.data_ptr() and short.codes.data_ptr() == cast.codes.data_ptr()
