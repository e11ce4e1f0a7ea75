"""Refusals of the expert block's calls (MXFP8 products, uncast rows on 4-bit weights, norms around a block), without a GPU:
statuses of the C ABI, the wrappers' ValueErrors, workspace sizes and the config struct's layout."""
import ctypes
import os
import subprocess

import pytest
import torch

import mxfp8_block_scaled_04_gb300 as mx

OK, NULL, SHAPE, ALIGN, FORMAT, WORKSPACE, DEVICE, LAUNCH, GROUPS = range(9)
A = 1 << 20  # an aligned address that no device owns: a call that passes every other check ends with the device's
BF16, F32, U8 = torch.bfloat16, torch.float32, torch.uint8
ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


# ---- MXFP8 products ------------------------------------------------------------------------------------

def product(kind=0, a=A, asc=A, ab=1 << 20, af=0, b=A, bsc=A, bb=1 << 20, bf=0, R=64, N=128, K=256, G=4, off=A, out=A, ot=0, err=A):
    return mx.mxfp8_matmul_grouped(kind, a, asc, ab, af, b, bsc, bb, bf, R, N, K, G, off, out, ot, err, 0)


@pytest.mark.parametrize("kind", [0, 1, 2])
def test_product_statuses(cuda_lib, kind):
    p = lambda **how: product(kind, **how)  # noqa: E731
    assert p() == DEVICE
    assert p(af=2) == FORMAT and p(bf=-1) == FORMAT and p(ot=2) == FORMAT
    assert p(N=120) == SHAPE and p(K=8) == SHAPE and p(R=-1) == SHAPE and p(R=1 << 31) == SHAPE and p(K=1 << 31) == SHAPE
    assert p(N=1 << 30) == SHAPE  # four experts of that pass 2^31 rows
    assert p(G=0) == GROUPS and p(G=513) == GROUPS and p(off=None) == GROUPS
    for hole in ("a", "asc", "b", "bsc", "out"):
        assert p(**{hole: None}) == NULL, hole
        assert p(**{hole: A + 8}) == ALIGN, hole
    assert p(off=A + 4) == ALIGN and p(err=A + 2) == ALIGN and p(err=None) == DEVICE
    assert p(ab=511) in (WORKSPACE, DEVICE)  # too small for any plane (told after the pointers' device)
    if kind != 2:
        need = 4 * -(-(128 if kind == 0 else 256) // 128) * -(-(256 if kind == 0 else 128) // 128) * 512
        assert p(bb=need - 1) == WORKSPACE and p(bb=need) == DEVICE


def test_unknown_product(cuda_lib):
    assert product(3) == FORMAT and product(-1) == FORMAT


def cast8(rows, cols, **changed):
    t = dict(out_row=torch.zeros(rows, cols, dtype=U8), scale_row=torch.zeros(4096, dtype=U8), out_col=torch.zeros(rows, cols, dtype=U8),
             scale_col=torch.zeros(4096, dtype=U8), dbias=None)
    return mx.MXFP8Tensor(**{**t, **changed})


def test_product_wrappers_refuse(cuda_lib):
    off = torch.tensor([0, 3, 8])
    x, w, dy = cast8(8, 32), cast8(2 * 48, 32), cast8(8, 48)
    f, dg, wg = mx.matmul_mxfp8_grouped, mx.matmul_mxfp8_grouped_dgrad, mx.matmul_mxfp8_grouped_wgrad
    for call in (
            lambda: f(x, off.int(), w), lambda: f(x, off[None], w), lambda: f(x, off[:1], w),
            lambda: f(x, off, w, torch.float16), lambda: f(x, off, w, err_flag=torch.zeros(1)),
            lambda: f(cast8(8, 64), off, w), lambda: f(x, off, cast8(95, 32)),
            lambda: f(x._replace(out_row=None), off, w), lambda: f(x._replace(scale_row=torch.zeros(8, 1, dtype=U8)), off, w),
            lambda: f(x, off, w._replace(scale_row=None)), lambda: f(x._replace(out_row=torch.zeros(8, 32)), off, w),
            lambda: f(x._replace(out_row=torch.zeros(32, 8, dtype=U8).t()), off, w),
            lambda: f(x._replace(out_row=torch.zeros(1, 32, dtype=U8).expand(8, 32)), off, w),
            lambda: dg(x, off, w), lambda: dg(dy, off, w._replace(out_col=None)), lambda: dg(dy, off, w._replace(scale_col=torch.zeros(3, 32, dtype=U8))),
            lambda: dg(dy, off, w, torch.int8),
            lambda: wg(dy, cast8(9, 32), off), lambda: wg(dy._replace(scale_col=None), x, off), lambda: wg(dy, x, off, torch.float64)):
        with pytest.raises(ValueError):
            call()
    with pytest.raises(KeyError):
        f(x, off, w, a_fmt="e3m4")
    for call in (lambda: f(x, off, w), lambda: dg(dy, off, w), lambda: wg(dy, x, off)):  # off the GPU: the library's to refuse
        with pytest.raises(mx.MXFP8Error) as error:
            call()
        assert error.value.status == DEVICE
    with pytest.raises(mx.MXFP8Error) as error:
        f(cast8(8, 24), off, cast8(96, 24))  # no multiple of 16
    assert error.value.status == SHAPE


# ---- uncast rows on 4-bit weights ----------------------------------------------------------------------

def linear(x=A, xt=0, M=9, K=64, ldx=64, b=A, s=A, N=40, out=A, ot=0, ldo=40, ws=A):
    return mx.mxfp4_linear(x, xt, M, K, ldx, b, s, N, out, ot, ldo, ws, 0)


def test_linear_statuses(cuda_lib):
    assert linear() == DEVICE
    assert linear(xt=2) == FORMAT and linear(ot=5) == FORMAT
    assert linear(K=60) == SHAPE and linear(ldx=56) == SHAPE and linear(ldx=68) == SHAPE and linear(M=1 << 28) == SHAPE and linear(ldo=39) == SHAPE
    assert linear(M=-1) == SHAPE and linear(N=-1) == SHAPE
    for hole in ("x", "b", "s", "out"):
        assert linear(**{hole: None}) == NULL, hole
    assert linear(ws=None) == WORKSPACE and linear(M=2, ws=None) == DEVICE  # few rows need none
    assert linear(x=A + 8) == ALIGN and linear(ws=A + 8) == ALIGN and linear(b=A + 8) == ALIGN and linear(out=A + 1) == ALIGN


def linear_grouped(x=A, xt=0, T=4, K=64, ldx=64, rows=A, R=8, G=2, off=A, b=A, s=A, N=40, out=A, ot=0, err=A, ws=A):
    return mx.mxfp4_linear_grouped(x, xt, T, K, ldx, rows, R, G, off, b, s, N, out, ot, err, ws, 0)


def test_linear_grouped_statuses(cuda_lib):
    g = linear_grouped
    assert g() == DEVICE and g(err=None) == DEVICE and g(rows=None, R=4) == DEVICE
    assert g(rows=None) == SHAPE  # more rows than x has
    assert g(xt=3) == FORMAT and g(ot=2) == FORMAT and g(K=4) == SHAPE and g(R=1 << 28) == SHAPE and g(N=1 << 30) == SHAPE
    assert g(G=0) == GROUPS and g(G=513) == GROUPS and g(off=None) == GROUPS and g(ws=None) == WORKSPACE
    assert g(x=None) == NULL and g(out=None) == NULL and g(b=None) == NULL
    assert g(off=A + 4) == ALIGN and g(rows=A + 2) == ALIGN and g(err=A + 1) == ALIGN


def test_few_rows_on_many_experts_need_no_workspace(cuda_lib):
    g = linear_grouped
    assert mx.mxfp4_linear_grouped_workspace_bytes(16, 40, 32) == 0 and mx.mxfp4_linear_grouped_workspace_bytes(16, 40, 31) > 0
    assert mx.mxfp4_linear_grouped_workspace_bytes(17, 40, 512) > 0
    assert g(R=4, G=8, ws=None) == DEVICE and g(R=5, G=8, ws=None) == WORKSPACE
    assert g(R=4, G=8, ws=None, T=0, x=None) == DEVICE  # no tokens: rows of no expert, or of NaN
    assert g(R=4, G=8, ws=None, x=None) == NULL and g(R=4, G=8, ws=None, b=None) == NULL


def test_linear_workspaces(cuda_lib):
    assert mx.mxfp4_linear_workspace_bytes(9, 40, 40) == 72 * 32 + mx.mxfp4_scale_bytes(72, 40)
    assert mx.mxfp4_linear_grouped_workspace_bytes(3, 40, 2) == 24 * 32 + mx.mxfp4_grouped_scale_bytes(24, 40, 2)
    for none in (mx.mxfp4_linear_workspace_bytes(0, 40, 40), mx.mxfp4_linear_workspace_bytes(2, 8192, 28672), mx.mxfp4_linear_workspace_bytes(9, 0, 40), mx.mxfp4_linear_workspace_bytes(1 << 28, 8, 8),
                 mx.mxfp4_linear_grouped_workspace_bytes(3, 40, 0)):
        assert none == 0


def test_linear_wrappers_refuse(cuda_lib):
    x, off = torch.zeros(4, 64, dtype=BF16), torch.tensor([0, 4])
    m = mx.MXFP4Matrix(torch.zeros(40, 32, dtype=U8), torch.zeros(512, dtype=U8), 40, 64)
    e = m._replace(codes=m.codes[None], scales=m.scales[None])
    repeated = torch.zeros(1, 64, dtype=BF16).expand(4, 64)
    for call in (
            lambda: mx.linear_mxfp4(x.half(), m), lambda: mx.linear_mxfp4(x[0], m), lambda: mx.linear_mxfp4(torch.zeros(64, 4, dtype=BF16).t(), m),
            lambda: mx.linear_mxfp4(repeated, m), lambda: mx.linear_mxfp4(x[:, :32].contiguous(), m), lambda: mx.linear_mxfp4(x, m, torch.float16),
            lambda: mx.linear_mxfp4(x, m, out=torch.zeros(4, 41)), lambda: mx.linear_mxfp4(x, m._replace(scales=m.scales[:8])),
            lambda: mx.linear_mxfp4(x, e), lambda: mx.linear_mxfp4_grouped(x, off, m), lambda: mx.linear_mxfp4_grouped(x, off.int(), e),
            lambda: mx.linear_mxfp4_grouped(x, off, e, rows=torch.zeros(4, dtype=torch.int64)),
            lambda: mx.linear_mxfp4_grouped(x, off, e, out_dtype=torch.float16), lambda: mx.linear_mxfp4_grouped(repeated, off, e),
            lambda: mx.linear_mxfp4_grouped(x, off, e, err_flag=torch.zeros(1))):
        with pytest.raises(ValueError):
            call()
    for call in (lambda: mx.linear_mxfp4(x, m), lambda: mx.linear_mxfp4_grouped(x, off, e)):
        with pytest.raises(mx.MXFP8Error) as error:
            call()
        assert error.value.status == DEVICE


# ---- norms ---------------------------------------------------------------------------------------------

def config(yt=0, ht=0, kind=1, pre=A, post=A, gate=A, **reserved):
    c = mx.BlockNormConfig(yt, ht, kind, 1.0, 1e-6, pre, post, gate)
    if reserved:
        c.reserved[2] = 1
    return c


def forward(cfg=None, T=4, H=64, y=A, ldy=64, h=A, ldh=64, ho=A, x=A, **how):
    return mx.block_norm_c(config(**how) if cfg is None else cfg, T, H, y, ldy, h, ldh, ho, x, 0)


def backward(T=4, H=64, gh=A, ldgh=64, gx=A, ldgx=64, y=A, ldy=64, h=A, ldh=64, dh=A, dy=A, dpre=A, dpost=A, dgate=A, ws=A, **how):
    return mx.block_norm_backward_c(config(**how), T, H, gh, ldgh, gx, ldgx, y, ldy, h, ldh, dh, dy, dpre, dpost, dgate, ws, 0)


def test_norm_statuses(cuda_lib):
    assert mx.block_norm_c(None, 4, 64, A, 64, A, 64, A, A, 0) == NULL
    assert forward() == DEVICE and forward(ho=None) == DEVICE and forward(pre=None, x=None) == DEVICE
    assert forward(y=None, post=None, gate=None, kind=0) == DEVICE
    assert forward(yt=2) == FORMAT and forward(ht=-1) == FORMAT and forward(kind=3) == FORMAT and forward(reserved=1) == FORMAT
    assert forward(H=60, ldy=64) == SHAPE and forward(H=16392, ldy=16392, ldh=16392) == SHAPE and forward(T=-1) == SHAPE
    assert forward(ldy=56) == SHAPE and forward(ldh=68) == SHAPE
    assert forward(gate=None) == NULL and forward(kind=0) == NULL  # a gate and its kind belong together
    assert forward(h=None) == NULL and forward(y=None) == NULL and forward(x=None) == NULL and forward(pre=None) == NULL
    assert forward(ho=None, x=None, pre=None) == NULL
    assert forward(y=A + 8) == ALIGN and forward(pre=A + 4) == ALIGN and forward(gate=A + 4) == ALIGN and forward(kind=2, gate=A + 4) == DEVICE
    assert forward(kind=2, gate=A + 2) == ALIGN and forward(x=A + 2) == ALIGN


def test_norm_backward_statuses(cuda_lib):
    assert backward() == DEVICE and backward(gh=None) == DEVICE and backward(gx=None) == DEVICE
    assert backward(gh=None, gx=None) == NULL and backward(h=None) == NULL and backward(y=None) == NULL
    assert backward(pre=None) == NULL and backward(pre=None, dpre=None, gx=None) == DEVICE
    assert backward(post=None) == NULL and backward(post=None, dpost=None) == DEVICE
    assert backward(kind=0, gate=None) == NULL and backward(kind=0, gate=None, dgate=None) == DEVICE
    assert backward(dh=None, dy=None, dpre=None, dpost=None, dgate=None) == NULL
    assert backward(ws=None) == WORKSPACE and backward(ws=None, dpre=None, dpost=None, dgate=None) == DEVICE
    assert backward(ws=A + 8) == ALIGN and backward(dy=A + 8) == ALIGN and backward(dpre=A + 2) == ALIGN
    assert backward(ldgx=56) == SHAPE and backward(ldgh=68) == SHAPE and backward(H=12) == SHAPE
    assert backward(y=None, kind=0, gate=None, dgate=None, post=None, dpost=None) == DEVICE  # nothing needs y


def test_norm_workspace(cuda_lib):
    size = mx.block_norm_backward_workspace_bytes
    assert size(3, 64) == 3 * 2 * 64 * 4 and size(0, 64) == 0 and size(3, 0) == 0 and size(3, 16392) == 0
    assert size(1 << 20, 8192) == size(1 << 21, 8192) > 0  # bounded by the rows in work at once


def test_norm_config_layout_matches_the_c_header(tmp_path):
    src = tmp_path / "layout.c"
    names = [f for f, _ in mx.BlockNormConfig._fields_]
    src.write_text('#include <stdio.h>\n#include <stddef.h>\n#include "block_norm.h"\nint main(void){printf("%zu", sizeof(block_norm_config_t));' +
                   "".join(f'printf(" %zu", offsetof(block_norm_config_t, {n}));' for n in names) + "return 0;}\n")
    exe = tmp_path / "layout"
    subprocess.run(["gcc", "-std=c99", "-Wall", "-Werror", "-I", os.path.join(ROOT, "include"), "-o", str(exe), str(src)], check=True)
    got = [int(v) for v in subprocess.run([str(exe)], capture_output=True, check=True, text=True).stdout.split()]
    assert got == [ctypes.sizeof(mx.BlockNormConfig)] + [getattr(mx.BlockNormConfig, n).offset for n in names]


def test_headers_compile_as_c(tmp_path):
    for name in ("mxfp8_matmul.h", "mxfp4.h", "block_norm.h"):
        src = tmp_path / "one.c"
        src.write_text(f'#include "{name}"\nint main(void) {{ return 0; }}\n')
        subprocess.run(["gcc", "-std=c99", "-Wall", "-Werror", "-pedantic", "-I", os.path.join(ROOT, "include"), "-c", "-o", str(tmp_path / "one.o"), str(src)],
                       check=True)


def test_norm_wrappers_refuse(cuda_lib):
    h, y = torch.zeros(4, 64, dtype=BF16), torch.zeros(4, 64)
    w, t = torch.ones(64), torch.ones(4, 1)
    repeated = torch.zeros(1, 64, dtype=BF16).expand(4, 64)
    f, b = mx.block_norm, mx.block_norm_backward
    for call in (
            lambda: f(y.half(), h, w), lambda: f(y, h.half(), w), lambda: f(y[:3], h, w), lambda: f(y, h[:, :32], w), lambda: f(repeated, h, w),
            lambda: f(y, repeated, w), lambda: f(y, h, w.bfloat16()), lambda: f(y, h, w[:8]), lambda: f(y, h, w, w[None]),
            lambda: f(y, h, w, gate=torch.ones(4)), lambda: f(y, h, w, gate=t.bfloat16()), lambda: f(y, h, w, gate=torch.ones(3, 1)),
            lambda: f(y, h, w, gate=torch.ones(128)[::2]), lambda: f(None, h, w, w), lambda: f(None, h, w, gate=t),
            lambda: b(None, None, y, h, w), lambda: b(h, h, y, h, None), lambda: b(y, h, y, h, w), lambda: b(h, y, y, h, w),
            lambda: b(h, h[:3], y, h, w), lambda: b(h, h, None, h, w, w), lambda: b(h, h, y, h, w, gate=w[:5])):
        with pytest.raises(ValueError):
            call()
    for call in (lambda: f(y, h, w, w, t), lambda: b(h, h, y, h, w, w, w)):
        with pytest.raises(mx.MXFP8Error) as error:
            call()
        assert error.value.status == DEVICE
