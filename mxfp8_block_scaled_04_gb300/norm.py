"""The norms around a block fused with its gate and residual scale: binding of the C ABI in include/block_norm.h.

The C functions are mirrored one for one by ``block_norm_c`` and ``block_norm_backward_c`` (status codes);
``block_norm`` and ``block_norm_backward`` check their tensors, allocate the outputs with torch (on ``stream`` when one
is given) and raise :class:`MXFP8Error` on a non-OK status.
"""
from __future__ import annotations

import ctypes
from typing import NamedTuple, Optional

import torch

from .binding import MXFP8Error, _addr, lib
from .mxfp4 import _check_input, _lib, _on, _stream, _stream_of

GATE_NONE = 0
GATE_CHANNEL = 1
GATE_TOKEN = 2
MAX_H = 16384


class BlockNormConfig(ctypes.Structure):
    """Mirror of block_norm_config_t (include/block_norm.h)."""
    _fields_ = [("y_type", ctypes.c_int), ("h_type", ctypes.c_int), ("gate_kind", ctypes.c_int), ("scale", ctypes.c_float),
                ("eps", ctypes.c_float), ("pre_weight", ctypes.c_void_p), ("post_weight", ctypes.c_void_p),
                ("gate", ctypes.c_void_p), ("reserved", ctypes.c_int * 4)]


class BlockNorm(NamedTuple):
    h: torch.Tensor            # [T, H] of the stream's type: scale * h + gate * norm(y)
    x: Optional[torch.Tensor]  # bfloat16 [T, H]: its norm, what the next block reads (None without pre_weight)


class BlockNormGrads(NamedTuple):
    y: Optional[torch.Tensor]            # of y's type
    h: torch.Tensor                      # of the stream's type
    pre_weight: Optional[torch.Tensor]   # float32 [H]
    post_weight: Optional[torch.Tensor]  # float32 [H]
    gate: Optional[torch.Tensor]         # float32 [H] or [T, 1], as the gate


# ---- one-for-one C entry points --------------------------------------------------

def block_norm_c(cfg, T, H, y, ldy, h, ldh, h_out, x, stream=None) -> int:
    return lib().block_norm(None if cfg is None else ctypes.byref(cfg), T, H, _addr(y), ldy, _addr(h), ldh, _addr(h_out),
                            _addr(x), _stream(stream))


def block_norm_backward_workspace_bytes(T: int, H: int) -> int:
    return int(lib().block_norm_backward_workspace_bytes(T, H))


def block_norm_backward_c(cfg, T, H, dh_out, lddh, dx, lddx, y, ldy, h_out, ldh, dh, dy, dpre, dpost, dgate, workspace,
                          stream=None) -> int:
    return lib().block_norm_backward(None if cfg is None else ctypes.byref(cfg), T, H, _addr(dh_out), lddh, _addr(dx), lddx,
                                     _addr(y), ldy, _addr(h_out), ldh, _addr(dh), _addr(dy), _addr(dpre), _addr(dpost),
                                     _addr(dgate), _addr(workspace), _stream(stream))


# ---- torch conveniences ----------------------------------------------------------
# A given ``stream`` is made current around the whole call, so that outputs and workspace belong to it.  The outputs are
# empty_like an input where one has their type: between launches an allocation takes about 2.8 microseconds so, and half a
# microsecond more with its type and device spelled out (a view of a common buffer takes as long as an allocation).

def _vector(w: Optional[torch.Tensor], H: int, name: str) -> Optional[int]:
    if w is None:
        return None
    if w.dtype is not torch.float32 or w.shape != (H,) or not w.is_contiguous():
        raise ValueError(f"{name} must be a contiguous float32 tensor [{H}]")
    return w.data_ptr()


def _gate(gate: Optional[torch.Tensor], T: int, H: int):
    """(kind, address) of a gate: None, [H] (per channel) or [T, 1] (per token)."""
    if gate is None:
        return GATE_NONE, None
    if gate.dtype is torch.float32 and gate.is_contiguous():
        if gate.dim() == 1 and gate.shape == (H,):
            return GATE_CHANNEL, gate.data_ptr()
        if gate.dim() == 2 and gate.shape == (T, 1):
            return GATE_TOKEN, gate.data_ptr()
    raise ValueError(f"gate must be a contiguous float32 tensor [{H}] or [{T}, 1]")


def _rows(t: Optional[torch.Tensor], name: str, shape, kind: Optional[int] = None):
    """(type, address, pitch) of an input of the stream's shape; None: (given type or bf16, NULL, 0)."""
    if t is None:
        return kind or 0, None, 0
    k, rows, cols, ld = _check_input(t, name)
    if (rows, cols) != shape:
        raise ValueError(f"{name} must be [{shape[0]}, {shape[1]}]")
    if kind is not None and k != kind:
        raise ValueError(f"{name} has the wrong type ({t.dtype})")
    return k, t.data_ptr(), ld


def block_norm(y: Optional[torch.Tensor], h: torch.Tensor, pre_weight: Optional[torch.Tensor],
               post_weight: Optional[torch.Tensor] = None, gate: Optional[torch.Tensor] = None, scale: float = 1.0,
               eps: float = 1e-6, stream=None) -> BlockNorm:
    """A block's output y [T, H] joins the residual stream h [T, H] and the next block's input is normed:
    h' = scale * h + gate * rms_norm(y) * post_weight, x = rms_norm(h') * pre_weight.

    y and h CUDA bf16 or fp32 each (rows contiguous, H a multiple of 8 up to 16384); weights fp32 [H].  Without
    ``post_weight`` y joins as it is; ``gate`` is fp32 [H] (per channel) or [T, 1] (per token); without ``pre_weight`` there
    is no x; without y, h' is scale * h (the norm before the first block).  h' has h's type, and x is the norm of h' as kept.
    """
    if stream is not None:
        with _on(stream):
            return block_norm(y, h, pre_weight, post_weight, gate, scale, eps)
    h_type, T, H, ldh = _check_input(h, "h")
    y_type, ya, ldy = _rows(y, "y", (T, H))
    if y is None and (post_weight is not None or gate is not None):
        raise ValueError("post_weight and gate need y")
    kind, ga = _gate(gate, T, H)
    cfg = BlockNormConfig(y_type, h_type, kind, scale, eps, _vector(pre_weight, H, "pre_weight"),
                          _vector(post_weight, H, "post_weight"), ga)
    h_out = torch.empty_like(h)
    x = xa = None
    if pre_weight is not None:
        x = torch.empty_like(h) if h_type == 0 else h.new_empty((T, H), dtype=torch.bfloat16)
        xa = x.data_ptr()
    st = _lib().block_norm(ctypes.byref(cfg), T, H, ya, ldy, h.data_ptr(), ldh, h_out.data_ptr(), xa, _stream_of(h.device))
    if st:
        raise MXFP8Error(st, "block_norm")
    return BlockNorm(h_out, x)


def block_norm_backward(grad_h: Optional[torch.Tensor], grad_x: Optional[torch.Tensor], y: Optional[torch.Tensor],
                        h_out: torch.Tensor, pre_weight: Optional[torch.Tensor],
                        post_weight: Optional[torch.Tensor] = None, gate: Optional[torch.Tensor] = None,
                        scale: float = 1.0, eps: float = 1e-6, stream=None) -> BlockNormGrads:
    """Gradients of block_norm from those of its results (``grad_h`` of the stream's type, ``grad_x`` bf16; either may be
    None), the block's output y and the stream ``h_out`` that block_norm returned."""
    if stream is not None:
        with _on(stream):
            return block_norm_backward(grad_h, grad_x, y, h_out, pre_weight, post_weight, gate, scale, eps)
    h_type, T, H, ldh = _check_input(h_out, "h_out")
    if grad_h is None and grad_x is None:
        raise ValueError("grad_h or grad_x is needed")
    if grad_x is not None and pre_weight is None:
        raise ValueError("grad_x needs pre_weight")
    if y is None and (post_weight is not None or gate is not None):
        raise ValueError("post_weight and gate need y")
    y_type, ya, ldy = _rows(y, "y", (T, H))
    _, gh, lddh = _rows(grad_h, "grad_h", (T, H), h_type)
    _, gx, lddx = _rows(grad_x, "grad_x", (T, H), 0)
    kind, ga = _gate(gate, T, H)
    cfg = BlockNormConfig(y_type, h_type, kind, scale, eps, _vector(pre_weight, H, "pre_weight"),
                          _vector(post_weight, H, "post_weight"), ga)
    dh = torch.empty_like(h_out)
    dy = None if y is None else torch.empty_like(y)
    dpre = None if pre_weight is None else torch.empty_like(pre_weight)
    dpost = None if post_weight is None else torch.empty_like(post_weight)
    dgate = None if gate is None else torch.empty_like(gate)
    lib_ = _lib()
    workspace = None
    if dpre is not None or dpost is not None or dgate is not None:
        workspace = h_out.new_empty((lib_.block_norm_backward_workspace_bytes(T, H),), dtype=torch.uint8)
    st = lib_.block_norm_backward(ctypes.byref(cfg), T, H, gh, lddh, gx, lddx, ya, ldy, h_out.data_ptr(), ldh, dh.data_ptr(),
                                  _addr(dy), _addr(dpre), _addr(dpost), _addr(dgate), _addr(workspace),
                                  _stream_of(h_out.device))
    if st:
        raise MXFP8Error(st, "block_norm_backward")
    return BlockNormGrads(dy, dh, dpre, dpost, dgate)
