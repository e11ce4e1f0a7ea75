"""Experts' products in MXFP8: binding of the C ABI in include/mxfp8_matmul.h.

``mxfp8_matmul_grouped`` mirrors the C entry point and returns the status code; ``matmul_mxfp8_grouped``,
``matmul_mxfp8_grouped_dgrad`` and ``matmul_mxfp8_grouped_wgrad`` take the outputs of ``quantize_grouped(...,
swizzled=True)`` (the weights' too: [E * N, K] rows in E groups of N), check them, allocate the result with torch and
raise :class:`MXFP8Error` on a non-OK status.
"""
from __future__ import annotations

from typing import Optional

import torch

from .binding import MXFP8Error, MXFP8Tensor, _addr, _fmt, lib
from .mxfp4 import _check_err, _check_offsets, _check_out_dtype, _lib, _on, _stream, _stream_of

FORWARD = 0
INPUT_GRADIENT = 1
WEIGHT_GRADIENT = 2


def mxfp8_matmul_grouped(product, a, a_scale, a_scale_bytes, a_fmt, b, b_scale, b_scale_bytes, b_fmt, total_rows, N, K,
                         num_groups, offsets, out, out_type, err_flag=None, stream=None) -> int:
    return lib().mxfp8_matmul_grouped(product, _addr(a), _addr(a_scale), a_scale_bytes, a_fmt, _addr(b), _addr(b_scale),
                                      b_scale_bytes, b_fmt, total_rows, N, K, num_groups, _addr(offsets), _addr(out),
                                      out_type, _addr(err_flag), _stream(stream))


def _direction(t: MXFP8Tensor, rows: bool, name: str):
    """(codes, scale plane) of one direction of a cast, checked."""
    codes, scale = (t.out_row, t.scale_row) if rows else (t.out_col, t.scale_col)
    which = "rowwise" if rows else "columnwise"
    if codes is None or scale is None:
        raise ValueError(f"{name} has no {which} cast")
    if codes.dtype is not torch.uint8 or codes.dim() != 2 or not codes.is_contiguous():
        raise ValueError(f"{name}'s {which} codes must be a contiguous 2-D uint8 tensor")
    if scale.dtype is not torch.uint8 or scale.dim() != 1 or not scale.is_contiguous():
        raise ValueError(f"{name}'s {which} scales must be a GEMM-ready plane (quantize_grouped with swizzled=True)")
    if scale.device != codes.device:
        raise ValueError(f"{name}'s {which} codes and scales are on different devices")
    return codes, scale


def _experts(rows: int, groups: int, name: str) -> int:
    if rows % groups:
        raise ValueError(f"{name} has {rows} rows, not a multiple of {groups} experts")
    return rows // groups


def _run(product, a, a_scale, a_fmt, b, b_scale, b_fmt, R, N, K, offsets, shape, out_dtype, err_flag):
    kind = _check_out_dtype(out_dtype)
    dev = a.device
    out = torch.empty(shape, dtype=out_dtype, device=dev)
    st = _lib().mxfp8_matmul_grouped(product, a.data_ptr(), a_scale.data_ptr(), a_scale.numel(), a_fmt, b.data_ptr(),
                                     b_scale.data_ptr(), b_scale.numel(), b_fmt, R, N, K, offsets.numel() - 1,
                                     offsets.data_ptr(), out.data_ptr(), kind, _addr(err_flag), _stream_of(dev))
    if st:
        raise MXFP8Error(st, "mxfp8_matmul_grouped")
    return out


def matmul_mxfp8_grouped(a: MXFP8Tensor, offsets: torch.Tensor, w: MXFP8Tensor, out_dtype: torch.dtype = torch.bfloat16,
                         a_fmt="e4m3", w_fmt="e4m3", err_flag: Optional[torch.Tensor] = None, stream=None) -> torch.Tensor:
    """Experts' forward products [R, N]: rows [offsets[g], offsets[g + 1]) of a [R, K] times expert g's w [N, K] transposed,
    from both rowwise casts.  N and K multiples of 16.  Rows past the last offset become zeros; ``err_flag`` (device int32) is
    set to 1 for bad offsets (nothing is written then) and where there are such rows."""
    if stream is not None:
        with _on(stream):
            return matmul_mxfp8_grouped(a, offsets, w, out_dtype, a_fmt, w_fmt, err_flag)
    groups = _check_offsets(offsets)
    _check_err(err_flag)
    ac, asc = _direction(a, True, "a")
    wc, wsc = _direction(w, True, "w")
    R, K = ac.shape
    N = _experts(wc.shape[0], groups, "w")
    if wc.shape[1] != K:
        raise ValueError(f"a has {K} columns, w has {wc.shape[1]}")
    return _run(FORWARD, ac, asc, _fmt(a_fmt), wc, wsc, _fmt(w_fmt), R, N, K, offsets, (R, N), out_dtype, err_flag)


def matmul_mxfp8_grouped_dgrad(grad: MXFP8Tensor, offsets: torch.Tensor, w: MXFP8Tensor,
                               out_dtype: torch.dtype = torch.bfloat16, grad_fmt="e5m2", w_fmt="e4m3",
                               err_flag: Optional[torch.Tensor] = None, stream=None) -> torch.Tensor:
    """Input gradient [R, K] of matmul_mxfp8_grouped: grad [R, N] (rowwise cast) times expert g's w [N, K] (columnwise
    cast).  ``offsets`` and ``err_flag`` as there."""
    if stream is not None:
        with _on(stream):
            return matmul_mxfp8_grouped_dgrad(grad, offsets, w, out_dtype, grad_fmt, w_fmt, err_flag)
    groups = _check_offsets(offsets)
    _check_err(err_flag)
    gc, gsc = _direction(grad, True, "grad")
    wc, wsc = _direction(w, False, "w")
    R, N = gc.shape
    K = wc.shape[1]
    if _experts(wc.shape[0], groups, "w") != N:
        raise ValueError(f"grad has {N} columns, w has {wc.shape[0] // groups} rows per expert")
    return _run(INPUT_GRADIENT, gc, gsc, _fmt(grad_fmt), wc, wsc, _fmt(w_fmt), R, N, K, offsets, (R, K), out_dtype, err_flag)


def matmul_mxfp8_grouped_wgrad(grad: MXFP8Tensor, a: MXFP8Tensor, offsets: torch.Tensor,
                               out_dtype: torch.dtype = torch.float32, grad_fmt="e5m2", a_fmt="e4m3",
                               err_flag: Optional[torch.Tensor] = None, stream=None) -> torch.Tensor:
    """Weight gradient [G, N, K] of matmul_mxfp8_grouped: expert g's grad [rows, N] transposed times its a [rows, K], from
    both columnwise casts; zeros for an expert without rows."""
    if stream is not None:
        with _on(stream):
            return matmul_mxfp8_grouped_wgrad(grad, a, offsets, out_dtype, grad_fmt, a_fmt, err_flag)
    groups = _check_offsets(offsets)
    _check_err(err_flag)
    gc, gsc = _direction(grad, False, "grad")
    ac, asc = _direction(a, False, "a")
    R, N = gc.shape
    K = ac.shape[1]
    if ac.shape[0] != R:
        raise ValueError(f"grad has {R} rows, a has {ac.shape[0]}")
    return _run(WEIGHT_GRADIENT, gc, gsc, _fmt(grad_fmt), ac, asc, _fmt(a_fmt), R, N, K, offsets, (groups, N, K), out_dtype,
                err_flag)
