"""Expert routing, dispatch plan and combination: binding of the C ABI in include/moe.h.

The C functions are mirrored one for one by ``moe_*_c`` (status codes); ``moe_route``,
``moe_route_backward``, ``moe_plan``, ``moe_combine`` and ``moe_combine_backward`` allocate their outputs
and raise :class:`MXFP8Error` on a non-OK status.
"""
from __future__ import annotations

import ctypes
import functools
from typing import NamedTuple, Optional

import torch

from .binding import _addr, lib
from .mxfp4 import _check, _check_input, _lib, _on, _stream, _stream_of

SCORES = {"softmax": 0, "sigmoid": 1}
MAX_TOPK = 32


class RouteConfig(ctypes.Structure):
    """Mirror of moe_route_config_t (include/moe.h)."""
    _fields_ = [("score", ctypes.c_int), ("top_k", ctypes.c_int), ("num_groups", ctypes.c_int),
                ("topk_groups", ctypes.c_int), ("renormalize", ctypes.c_int), ("scale", ctypes.c_float),
                ("bias", ctypes.c_void_p), ("reserved", ctypes.c_int * 4)]


class MoERoute(NamedTuple):
    indices: torch.Tensor  # int32 [T, k], by falling key
    weights: torch.Tensor  # float32 [T, k]


class MoEPlan(NamedTuple):
    offsets: torch.Tensor  # int64 [E + 1]: expert e's rows
    slots: torch.Tensor    # int32 [T, k]: the row of each choice (-2 - r, r a row left over: dropped)
    tokens: torch.Tensor   # int32 [T * k]: the token of each row (-1: left over)


# ---- one-for-one C entry points --------------------------------------------------

def moe_route_c(logits, type_, T, E, ld, cfg, indices, weights, stream=None) -> int:
    return lib().moe_route(_addr(logits), type_, T, E, ld, None if cfg is None else ctypes.byref(cfg), _addr(indices),
                           _addr(weights), _stream(stream))


def moe_route_backward_c(logits, type_, T, E, ld, cfg, indices, dweights, dlogits, stream=None) -> int:
    return lib().moe_route_backward(_addr(logits), type_, T, E, ld, None if cfg is None else ctypes.byref(cfg),
                                    _addr(indices), _addr(dweights), _addr(dlogits), _stream(stream))


def moe_plan_workspace_bytes(n: int, E: int) -> int:
    return int(lib().moe_plan_workspace_bytes(n, E))


def moe_plan_c(indices, n, k, E, offsets, slots, tokens, workspace, stream=None) -> int:
    return lib().moe_plan(_addr(indices), n, k, E, _addr(offsets), _addr(slots), _addr(tokens), _addr(workspace),
                          _stream(stream))


def moe_combine_c(y, R, H, slots, weights, T, k, out, stream=None) -> int:
    return lib().moe_combine(_addr(y), R, H, _addr(slots), _addr(weights), T, k, _addr(out), _stream(stream))


def moe_combine_backward_c(dout, y, R, H, slots, weights, T, k, dy, dweights, stream=None) -> int:
    return lib().moe_combine_backward(_addr(dout), _addr(y), R, H, _addr(slots), _addr(weights), T, k, _addr(dy),
                                      _addr(dweights), _stream(stream))


# ---- torch conveniences ----------------------------------------------------------
# A given ``stream`` is made current around the whole call, so that outputs and workspace belong to it.

def _check_like(t: torch.Tensor, name: str, dtype: torch.dtype, shape=None):
    size = t.shape
    if t.dtype is not dtype or len(size) != 2 or not t.is_contiguous() or (shape is not None and size != shape):
        raise ValueError(f"{name} must be a contiguous {dtype} tensor" + (f" {list(shape)}" if shape else " [., .]"))
    return size


def make_route_config(top_k: int, score="softmax", bias: Optional[torch.Tensor] = None, groups: int = 1,
                      topk_groups: int = 1, renormalize: bool = True, scale: float = 1.0) -> RouteConfig:
    """A RouteConfig from tensors / names (marshalling only)."""
    score = SCORES[score.lower()] if isinstance(score, str) else int(score)
    return RouteConfig(score, top_k, groups, topk_groups, int(bool(renormalize)), scale, _addr(bias))


@functools.lru_cache(maxsize=64)
def _unbiased_config(*how) -> RouteConfig:
    """make_route_config without a bias, kept for the next call of the same options (the library only reads it)."""
    top_k, score, groups, topk_groups, renormalize, scale = how
    return make_route_config(top_k, score, None, groups, topk_groups, renormalize, scale)


def moe_route(logits: torch.Tensor, k: int, score="softmax", bias: Optional[torch.Tensor] = None, groups: int = 1,
              topk_groups: int = 1, renormalize: bool = True, scale: float = 1.0, stream=None) -> MoERoute:
    """Choose k of E experts for each row of ``logits`` [T, E] (CUDA bf16 or fp32, rows contiguous).

    ``score`` "softmax" or "sigmoid"; ``bias`` (fp32 [E]) enters the choice alone; with ``topk_groups`` <
    ``groups`` the choice is limited to the best groups of consecutive experts; ``renormalize`` divides the
    weights by their sum; ``scale`` multiplies them.
    """
    if stream is not None:
        with _on(stream):
            return moe_route(logits, k, score, bias, groups, topk_groups, renormalize, scale)
    kind, T, E, ld = _check_input(logits, "logits")
    if bias is not None and (bias.dtype != torch.float32 or bias.shape != (E,) or not bias.is_contiguous()):
        raise ValueError(f"bias must be a contiguous float32 tensor [{E}]")
    if bias is None:
        cfg = _unbiased_config(k, score, groups, topk_groups, renormalize, scale)
    else:
        cfg = make_route_config(k, score, bias, groups, topk_groups, renormalize, scale)
    dev = logits.device
    indices = torch.empty((T, k), dtype=torch.int32, device=dev)
    weights = torch.empty((T, k), dtype=torch.float32, device=dev)
    _check(_lib().moe_route(logits.data_ptr(), kind, T, E, ld, ctypes.byref(cfg), indices.data_ptr(), weights.data_ptr(),
                            _stream_of(dev)), "moe_route")
    return MoERoute(indices, weights)


def moe_route_backward(logits: torch.Tensor, indices: torch.Tensor, grad_weights: torch.Tensor, score="softmax",
                       renormalize: bool = True, scale: float = 1.0, stream=None) -> torch.Tensor:
    """Gradient of moe_route's weights with respect to the logits (the choice and the bias are constants)."""
    if stream is not None:
        with _on(stream):
            return moe_route_backward(logits, indices, grad_weights, score, renormalize, scale)
    kind, T, E, ld = _check_input(logits, "logits")
    rows, k = _check_like(indices, "indices", torch.int32)
    _check_like(grad_weights, "grad_weights", torch.float32, (rows, k))
    if rows != T:
        raise ValueError(f"indices must have {T} rows")
    cfg = _unbiased_config(k, score, 1, 1, renormalize, scale)
    dev = logits.device
    out = torch.empty((T, E), dtype=logits.dtype, device=dev)
    _check(_lib().moe_route_backward(logits.data_ptr(), kind, T, E, ld, ctypes.byref(cfg), indices.data_ptr(), grad_weights.data_ptr(),
                                     out.data_ptr(), _stream_of(dev)), "moe_route_backward")
    return out


def moe_plan(indices: torch.Tensor, num_experts: int, stream=None) -> MoEPlan:
    """Sort the choices ``indices`` (int32 [T, k]) by expert, in order within an expert."""
    if stream is not None:
        with _on(stream):
            return moe_plan(indices, num_experts)
    T, k = _check_like(indices, "indices", torch.int32)
    dev = indices.device
    offsets = torch.empty((num_experts + 1,), dtype=torch.int64, device=dev)
    slots = torch.empty((T, k), dtype=torch.int32, device=dev)
    tokens = torch.empty((T * k,), dtype=torch.int32, device=dev)
    # small plans need none; the library knows from where on
    nbytes = moe_plan_workspace_bytes(T * k, num_experts) if T * k > 1024 else 0
    workspace = torch.empty((nbytes,), dtype=torch.uint8, device=dev) if nbytes else None
    _check(_lib().moe_plan(indices.data_ptr(), T * k, k, num_experts, offsets.data_ptr(), slots.data_ptr(),
                           tokens.data_ptr(), _addr(workspace), _stream_of(dev)), "moe_plan")
    return MoEPlan(offsets, slots, tokens)


def moe_combine(y: torch.Tensor, slots: torch.Tensor, weights: Optional[torch.Tensor] = None, stream=None) -> torch.Tensor:
    """out[t] = sum_j weights[t, j] * y[slots[t, j]] (bf16 rows, fp32 sums; no ``weights``: all 1)."""
    if stream is not None:
        with _on(stream):
            return moe_combine(y, slots, weights)
    R, H = _check_like(y, "y", torch.bfloat16)
    T, k = _check_like(slots, "slots", torch.int32)
    if weights is not None:
        _check_like(weights, "weights", torch.float32, (T, k))
    dev = y.device
    out = torch.empty((T, H), dtype=torch.bfloat16, device=dev)
    _check(_lib().moe_combine(y.data_ptr(), R, H, slots.data_ptr(), _addr(weights), T, k, out.data_ptr(),
                              _stream_of(dev)), "moe_combine")
    return out


def moe_combine_backward(grad: torch.Tensor, y: torch.Tensor, slots: torch.Tensor, weights: Optional[torch.Tensor] = None,
                         stream=None):
    """(grad_y, grad_weights) of moe_combine.  The slots name every row of y (as moe_plan's do, dropped choices
    included); rows past T * k get zeros."""
    if stream is not None:
        with _on(stream):
            return moe_combine_backward(grad, y, slots, weights)
    R, H = _check_like(y, "y", torch.bfloat16)
    T, k = _check_like(slots, "slots", torch.int32)
    _check_like(grad, "grad", torch.bfloat16, (T, H))
    if weights is not None:
        _check_like(weights, "weights", torch.float32, (T, k))
    dev = y.device
    dy = (torch.zeros if R > T * k else torch.empty)((R, H), dtype=torch.bfloat16, device=dev)
    dweights = torch.empty((T, k), dtype=torch.float32, device=dev)
    _check(_lib().moe_combine_backward(grad.data_ptr(), y.data_ptr(), R, H, slots.data_ptr(), _addr(weights), T, k, dy.data_ptr(),
                                       dweights.data_ptr(), _stream_of(dev)), "moe_combine_backward")
    return dy, dweights
