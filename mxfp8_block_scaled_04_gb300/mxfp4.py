"""MXFP4 (4-bit microscaled) cast and products: binding of the C ABI in include/mxfp4.h.

The functions named ``mxfp4_*`` mirror the C entry points one for one and return the status code;
``quantize_mxfp4``, ``quantize_mxfp4_grouped``, ``dequantize_mxfp4``, ``matmul_mxfp4``, ``matmul_mxfp4_grouped``,
``linear_mxfp4`` and ``linear_mxfp4_grouped`` check their tensors, allocate the outputs with torch (on ``stream`` when one is
given) and raise :class:`MXFP8Error` on a non-OK status.
"""
from __future__ import annotations

import operator
from typing import NamedTuple, Optional

import torch

from .binding import MXFP8Error, _addr, lib
from .binding import _stream as _any_stream

TYPE_BF16 = 0
TYPE_F32 = 1
_TYPES = {torch.bfloat16: TYPE_BF16, torch.float32: TYPE_F32}


class MXFP4Matrix:
    """A 4-bit matrix [rows, cols]: blocks of 32 along the columns.  Experts' matrices of one shape are held
    together with a leading dimension on ``codes`` and ``scales``.

    ``codes``   uint8 [rows, 16 * ceil(cols / 32)]
    ``scales``  uint8, 1-D: the GEMM-ready E8M0 plane
    ``groups``  number of experts of a grouped cast, which has a plane per expert (None: one plane)

    The casts put both into one allocation and make the two tensors when they are asked for (an allocation or a
    view costs a call about two microseconds); the calls of this module use the addresses, which follow from the
    size: ``rows``, ``cols`` and ``groups`` are read-only.
    """
    __slots__ = ("_rows", "_cols", "_groups", "_codes", "_scales", "_buffer", "_offset", "_plane")

    def __init__(self, codes: torch.Tensor, scales: torch.Tensor, rows: int, cols: int, groups: Optional[int] = None):
        self._rows, self._cols, self._groups = rows, cols, groups
        self._codes, self._scales = codes, scales
        self._buffer, self._offset, self._plane = None, 0, 0

    @classmethod
    def _in(cls, buffer: torch.Tensor, offset: int, rows: int, cols: int, plane: int,
            groups: Optional[int] = None) -> "MXFP4Matrix":
        """A cast's matrix: codes at ``offset`` of the uint8 ``buffer``, ``plane`` bytes of scales after them."""
        m = cls.__new__(cls)
        m._rows, m._cols, m._groups = rows, cols, groups
        m._codes = m._scales = None
        m._buffer, m._offset, m._plane = buffer, offset, plane
        return m

    rows = property(operator.attrgetter("_rows"))
    cols = property(operator.attrgetter("_cols"))
    groups = property(operator.attrgetter("_groups"))

    @property
    def codes(self) -> torch.Tensor:
        if self._codes is None:
            n = self.rows * mxfp4_row_bytes(self.cols)
            self._codes = self._buffer[self._offset:self._offset + n].view(self.rows, mxfp4_row_bytes(self.cols))
        return self._codes

    @property
    def scales(self) -> torch.Tensor:
        if self._scales is None:
            at = self._offset + self.rows * mxfp4_row_bytes(self.cols)
            self._scales = self._buffer[at:at + self._plane]
        return self._scales

    def _replace(self, **changed) -> "MXFP4Matrix":
        return MXFP4Matrix(**{**dict(codes=self.codes, scales=self.scales, rows=self.rows, cols=self.cols,
                                       groups=self.groups), **changed})

    def __repr__(self) -> str:
        return f"MXFP4Matrix({self.rows} x {self.cols})"


class MXFP4Tensor(NamedTuple):
    """Outputs of quantize_mxfp4; a direction that was not requested is None."""
    row: Optional[MXFP4Matrix]  # x [M, N]
    col: Optional[MXFP4Matrix]  # x transposed [N, M]


_raw_stream = torch._C._cuda_getCurrentRawStream if hasattr(torch._C, "_cuda_getCurrentRawStream") else None


def _stream(stream) -> Optional[int]:
    """The cudaStream_t of ``stream``, or of the current device's current stream."""
    if stream is None and torch.cuda.is_initialized():
        return _raw_stream(torch._C._cuda_getDevice())
    return _any_stream(stream)


def _stream_of(device: torch.device) -> Optional[int]:
    """The current stream of a tensor's device, by torch's raw getter (a tenth of a microsecond, where
    torch.cuda.current_stream() costs three).  A tensor off the GPU is the library's to refuse."""
    return None if device.index is None else _raw_stream(device.index)


_library = None


def _lib():
    """The loaded library, without binding.lib()'s lock once it is there."""
    global _library
    if _library is None:
        _library = lib()
    return _library


# ---- one-for-one C entry points --------------------------------------------------

def mxfp4_row_bytes(cols: int) -> int:
    return -(-cols // 32) * 16 if cols > 0 else 0


def mxfp4_scale_bytes(rows: int, cols: int) -> int:
    return -(-rows // 128) * -(-cols // 128) * 512 if rows > 0 and cols > 0 else 0


def mxfp4_grouped_scale_bytes(total_rows: int, cols: int, num_groups: int) -> int:
    if total_rows <= 0 or cols <= 0 or num_groups < 1:
        return 0
    return (total_rows // 128 + min(num_groups, total_rows)) * -(-cols // 128) * 512


def mxfp4_quantize(x, x_type, M, N, ldx, out_row, scale_row, out_col, scale_col, noop=None, stream=None) -> int:
    return lib().mxfp4_quantize(_addr(x), x_type, M, N, ldx, _addr(out_row), _addr(scale_row), _addr(out_col),
                                _addr(scale_col), _addr(noop), _stream(stream))


def mxfp4_quantize_grouped_workspace_bytes(T: int, N: int, total_rows: int) -> int:
    if T <= 0 or N <= 0 or total_rows <= T:
        return 0
    return T * mxfp4_row_bytes(N) + mxfp4_scale_bytes(T, N)


def mxfp4_quantize_grouped(x, x_type, T, N, ldx, rows, total_rows, num_groups, offsets, out, scale, err_flag=None,
                           workspace=None, stream=None) -> int:
    return lib().mxfp4_quantize_grouped(_addr(x), x_type, T, N, ldx, _addr(rows), total_rows, num_groups,
                                        _addr(offsets), _addr(out), _addr(scale), _addr(err_flag), _addr(workspace),
                                        _stream(stream))


def mxfp4_dequantize(codes, scale, rows, cols, out, out_type, stream=None) -> int:
    return lib().mxfp4_dequantize(_addr(codes), _addr(scale), rows, cols, _addr(out), out_type, _stream(stream))


def mxfp4_matmul(a_codes, a_scale, M, b_codes, b_scale, N, K, out, out_type, ldo, stream=None) -> int:
    return lib().mxfp4_matmul(_addr(a_codes), _addr(a_scale), M, _addr(b_codes), _addr(b_scale), N, K, _addr(out),
                              out_type, ldo, _stream(stream))


def mxfp4_matmul_grouped(a_codes, a_scale, total_rows, num_groups, offsets, b_codes, b_scale, N, K, out, out_type,
                         err_flag=None, stream=None) -> int:
    return lib().mxfp4_matmul_grouped(_addr(a_codes), _addr(a_scale), total_rows, num_groups, _addr(offsets),
                                      _addr(b_codes), _addr(b_scale), N, K, _addr(out), out_type, _addr(err_flag),
                                      _stream(stream))


def mxfp4_linear_workspace_bytes(M: int, K: int, N: int) -> int:
    return int(lib().mxfp4_linear_workspace_bytes(M, K, N))


def mxfp4_linear(x, x_type, M, K, ldx, b_codes, b_scale, N, out, out_type, ldo, workspace, stream=None) -> int:
    return lib().mxfp4_linear(_addr(x), x_type, M, K, ldx, _addr(b_codes), _addr(b_scale), N, _addr(out), out_type, ldo,
                              _addr(workspace), _stream(stream))


def mxfp4_linear_grouped_workspace_bytes(total_rows: int, K: int, num_groups: int) -> int:
    return int(lib().mxfp4_linear_grouped_workspace_bytes(total_rows, K, num_groups))


def mxfp4_linear_grouped(x, x_type, T, K, ldx, rows, total_rows, num_groups, offsets, b_codes, b_scale, N, out, out_type,
                         err_flag=None, workspace=None, stream=None) -> int:
    return lib().mxfp4_linear_grouped(_addr(x), x_type, T, K, ldx, _addr(rows), total_rows, num_groups, _addr(offsets),
                                      _addr(b_codes), _addr(b_scale), N, _addr(out), out_type, _addr(err_flag),
                                      _addr(workspace), _stream(stream))


# ---- torch conveniences ----------------------------------------------------------
# A given ``stream`` is made current around the whole call, so that the outputs belong to it.

def _on(stream):
    """The context of ``stream`` (a torch stream or a cudaStream_t address)."""
    return torch.cuda.stream(stream if isinstance(stream, torch.cuda.Stream) else torch.cuda.ExternalStream(int(stream)))


def _check(status: int, what: str) -> None:
    if status != 0:
        raise MXFP8Error(status, what)


def _check_input(x: torch.Tensor, name: str = "x"):
    """(type, rows, columns, row pitch) of a 2-D bf16 / fp32 tensor whose rows are contiguous and do not overlap (an
    expanded row, as the gradient of a sum over rows is, has a stride of 0: no pitch)."""
    kind = _TYPES.get(x.dtype)
    if kind is None or x.dim() != 2:
        raise ValueError(f"{name} must be a 2-D bfloat16 or float32 tensor with contiguous rows")
    rows, cols = x.shape
    pitch, step = x.stride()
    if step != 1 and cols > 1:
        raise ValueError(f"{name} must be a 2-D bfloat16 or float32 tensor with contiguous rows")
    if rows < 2 or cols == 0:
        return kind, rows, cols, cols
    if pitch < cols:
        raise ValueError(f"{name} must have contiguous rows that do not overlap (row stride {pitch}, {cols} columns)")
    return kind, rows, cols, pitch


def _check_offsets(offsets: torch.Tensor) -> int:
    if offsets.dtype != torch.int64 or offsets.dim() != 1 or offsets.numel() < 2 or not offsets.is_contiguous():
        raise ValueError("offsets must be a contiguous 1-D int64 tensor of num_groups + 1 entries")
    return offsets.numel() - 1


def _check_err(err_flag) -> None:
    if err_flag is not None and (err_flag.dtype != torch.int32 or err_flag.numel() < 1):
        raise ValueError("err_flag must be an int32 tensor")


def _laid_out(m: MXFP4Matrix, codes: int, plane: int) -> bool:
    """Whether a cast made m with that many bytes of codes and at least that many of scales."""
    return m._buffer is not None and m._plane >= plane and m._buffer.numel() - m._offset >= codes + m._plane


def _check_matrix(m: MXFP4Matrix, name: str, groups: Optional[int] = None):
    """(address of the codes, address of the scales) of a matrix whose tensors have the right types and shapes."""
    rows, cols = m.rows, m.cols
    if m.groups is not None:
        raise ValueError(f"{name} is a grouped cast (a scale plane per expert)")
    pitch = -(-cols // 32) * 16
    plane = -(-rows // 128) * -(-cols // 128) * 512
    if _laid_out(m, rows * pitch, plane) and groups is None:
        at = m._buffer.data_ptr() + m._offset
        return at, at + rows * pitch
    codes, scales = m.codes, m.scales
    shape = (rows, pitch) if groups is None else (groups, rows, pitch)
    if codes.dtype is not torch.uint8 or codes.shape != shape or not codes.is_contiguous():
        raise ValueError(f"{name}.codes must be a contiguous uint8 tensor {list(shape)}")
    if scales.dtype is not torch.uint8 or not scales.is_contiguous() or (
            scales.numel() < plane if groups is None else scales.shape != (groups, plane)):
        raise ValueError(f"{name}.scales must be a contiguous uint8 tensor of {plane} bytes per matrix")
    return codes.data_ptr(), scales.data_ptr()


def _device(m: MXFP4Matrix) -> torch.device:
    return (m._codes if m._buffer is None else m._buffer).device


def _check_out_dtype(dtype: torch.dtype) -> int:
    kind = _TYPES.get(dtype)
    if kind is None:
        raise ValueError("the output type must be torch.bfloat16 or torch.float32")
    return kind


# Both matrices of a cast share an allocation up to this size; a larger one keeps each alive on its own.
_SHARED_BYTES = 1 << 20


def quantize_mxfp4(x: torch.Tensor, rowwise: bool = True, colwise: bool = False, noop: Optional[torch.Tensor] = None,
                   stream=None) -> MXFP4Tensor:
    """MXFP4-quantize a CUDA bf16 or fp32 tensor [M, N] (any M, N a multiple of 8, rows contiguous).

    ``row`` is x with blocks along its rows; ``col`` is x transposed with blocks along M, the operand of
    the products that sum over M (input and weight gradients).
    """
    if stream is not None:
        with _on(stream):
            return quantize_mxfp4(x, rowwise, colwise, noop)
    kind, M, N, ld = _check_input(x)
    dev = x.device
    row = col = rc = rs = cc = cs = None
    codes = M * (-(-N // 32) * 16)
    codes_t = N * (-(-M // 32) * 16)
    plane = plane_t = -(-M // 128) * -(-N // 128) * 512
    first = codes + plane if rowwise else 0
    second = codes_t + plane_t if colwise else 0
    buffer = torch.empty((first + second if first + second <= _SHARED_BYTES else first or second,), dtype=torch.uint8, device=dev)
    if rowwise:
        rc = buffer.data_ptr()
        rs = rc + codes
        row = MXFP4Matrix._in(buffer, 0, M, N, plane)
    if colwise:
        at = first
        if rowwise and first + second > _SHARED_BYTES:
            buffer, at = torch.empty((second,), dtype=torch.uint8, device=dev), 0
        cc = buffer.data_ptr() + at
        cs = cc + codes_t
        col = MXFP4Matrix._in(buffer, at, N, M, plane_t)
    st = _lib().mxfp4_quantize(x.data_ptr(), kind, M, N, ld, rc, rs, cc, cs, _addr(noop), _stream_of(dev))
    if st:
        raise MXFP8Error(st, "mxfp4_quantize")
    return MXFP4Tensor(row, col)


def quantize_mxfp4_grouped(x: torch.Tensor, offsets: torch.Tensor, rows: Optional[torch.Tensor] = None,
                           err_flag: Optional[torch.Tensor] = None, stream=None) -> MXFP4Matrix:
    """The rowwise cast of x's rows gathered for experts: output row i is x[rows[i]] (x[i] without ``rows``),
    expert g owns rows [offsets[g], offsets[g + 1]) (device int64) and has a scale plane of its own.

    Rows past the last offset belong to no expert (a plan's dropped choices, whose ``rows`` are negative): zero codes.
    ``err_flag`` (device int32) is set to 1 for bad offsets, an index outside x, or such rows without a negative index.
    """
    if stream is not None:
        with _on(stream):
            return quantize_mxfp4_grouped(x, offsets, rows, err_flag)
    kind, T, N, ld = _check_input(x)
    groups = _check_offsets(offsets)
    _check_err(err_flag)
    if rows is not None and (rows.dtype != torch.int32 or rows.dim() != 1 or not rows.is_contiguous()):
        raise ValueError("rows must be a contiguous 1-D int32 tensor")
    total = T if rows is None else rows.numel()
    dev = x.device
    codes, plane = total * mxfp4_row_bytes(N), mxfp4_grouped_scale_bytes(total, N, groups)
    buffer = torch.empty((codes + plane,), dtype=torch.uint8, device=dev)
    nbytes = 0 if rows is None else mxfp4_quantize_grouped_workspace_bytes(T, N, total)
    workspace = torch.empty((nbytes,), dtype=torch.uint8, device=dev) if nbytes else None
    at = buffer.data_ptr()
    st = _lib().mxfp4_quantize_grouped(x.data_ptr(), kind, T, N, ld, _addr(rows), total, groups, offsets.data_ptr(), at,
                                       at + codes, _addr(err_flag), _addr(workspace), _stream_of(dev))
    if st:
        raise MXFP8Error(st, "mxfp4_quantize_grouped")
    return MXFP4Matrix._in(buffer, 0, total, N, plane, groups)


def dequantize_mxfp4(m: MXFP4Matrix, dtype: torch.dtype = torch.bfloat16, stream=None) -> torch.Tensor:
    """The values [rows, cols] of a 4-bit matrix (exact in bf16 and fp32)."""
    if stream is not None:
        with _on(stream):
            return dequantize_mxfp4(m, dtype)
    kind = _check_out_dtype(dtype)
    codes, scales = _check_matrix(m, "m")
    dev = _device(m)
    out = torch.empty((m.rows, m.cols), dtype=dtype, device=dev)
    st = _lib().mxfp4_dequantize(codes, scales, m.rows, m.cols, out.data_ptr(), kind, _stream_of(dev))
    if st:
        raise MXFP8Error(st, "mxfp4_dequantize")
    return out


def matmul_mxfp4(a: MXFP4Matrix, b: MXFP4Matrix, out_dtype: torch.dtype = torch.bfloat16,
                 out: Optional[torch.Tensor] = None, stream=None) -> torch.Tensor:
    """a [M, K] times b [N, K] transposed: [M, N] in ``out_dtype``, or into ``out`` (rows contiguous)."""
    if stream is not None:
        with _on(stream):
            return matmul_mxfp4(a, b, out_dtype, out)
    ac, asc = _check_matrix(a, "a")
    bc, bsc = _check_matrix(b, "b")
    dev = _device(a)
    M, N, K = a.rows, b.rows, a.cols
    if K != b.cols:
        raise ValueError(f"a has {K} columns, b has {b.cols}")
    if out is None:
        kind, ldo = _check_out_dtype(out_dtype), N
        out = torch.empty((M, N), dtype=out_dtype, device=dev)
    else:
        kind, rows, cols, ldo = _check_input(out, "out")
        if (rows, cols) != (M, N):
            raise ValueError(f"out must be [{M}, {N}]")
    st = _lib().mxfp4_matmul(ac, asc, M, bc, bsc, N, K, out.data_ptr(), kind, ldo, _stream_of(dev))
    if st:
        raise MXFP8Error(st, "mxfp4_matmul")
    return out


def matmul_mxfp4_grouped(a: MXFP4Matrix, offsets: torch.Tensor, b: MXFP4Matrix, out_dtype: torch.dtype = torch.bfloat16,
                         err_flag: Optional[torch.Tensor] = None, stream=None) -> torch.Tensor:
    """Experts' products: rows [offsets[g], offsets[g + 1]) of a (from quantize_mxfp4_grouped) times expert g's
    b [N, K] transposed; b.codes [G, N, .], b.scales [G, .].  Returns [total_rows, N], zeros in the rows past the
    last offset; ``err_flag`` is set to 1 for bad offsets and where there are such rows."""
    if stream is not None:
        with _on(stream):
            return matmul_mxfp4_grouped(a, offsets, b, out_dtype, err_flag)
    groups = _check_offsets(offsets)
    _check_err(err_flag)
    bc, bsc = _check_matrix(b, "b", groups)
    kind = _check_out_dtype(out_dtype)
    R, K = a.rows, a.cols
    if K != b.cols:
        raise ValueError(f"a has {K} columns, b has {b.cols}")
    if a.groups is not None and a.groups != groups:
        raise ValueError(f"a was cast for {a.groups} experts, offsets name {groups}")
    need = mxfp4_grouped_scale_bytes(R, K, groups)
    if _laid_out(a, R * mxfp4_row_bytes(K), need):
        ac = a._buffer.data_ptr() + a._offset
        asc = ac + R * mxfp4_row_bytes(K)
    else:
        codes, scales = a.codes, a.scales
        if codes.dtype is not torch.uint8 or codes.shape != (R, mxfp4_row_bytes(K)) or not codes.is_contiguous():
            raise ValueError("a.codes must be a contiguous uint8 tensor [rows, 16 * ceil(cols / 32)]")
        if scales.dtype is not torch.uint8 or scales.numel() < need or not scales.is_contiguous():
            raise ValueError("a.scales must hold mxfp4_grouped_scale_bytes(rows, cols, groups) bytes")
        ac, asc = codes.data_ptr(), scales.data_ptr()
    dev = _device(a)
    out = torch.empty((R, b.rows), dtype=out_dtype, device=dev)
    st = _lib().mxfp4_matmul_grouped(ac, asc, R, groups, offsets.data_ptr(), bc, bsc, b.rows, K, out.data_ptr(), kind,
                                     _addr(err_flag), _stream_of(dev))
    if st:
        raise MXFP8Error(st, "mxfp4_matmul_grouped")
    return out


def linear_mxfp4(x: torch.Tensor, w: MXFP4Matrix, out_dtype: torch.dtype = torch.bfloat16,
                 out: Optional[torch.Tensor] = None, stream=None) -> torch.Tensor:
    """x [M, K] (CUDA bf16 or fp32, not cast; K a multiple of 8, rows contiguous) times 4-bit weights w [N, K] transposed:
    [M, N] in ``out_dtype``, or into ``out`` (rows contiguous).  For few rows, as a serving step has (for many, cast them and use
    ``matmul_mxfp4``).

    x enters as 24-bit fixed point under the scale of each block of 32 columns: an element is off by at most 2^-22 of its block's
    largest magnitude, which is fp32 accuracy where a block's magnitudes are alike and less for elements far below an outlier.
    A NaN or an infinity in a row of x makes that output row NaN, and results may overflow from 3/7 of fp32's range on."""
    if stream is not None:
        with _on(stream):
            return linear_mxfp4(x, w, out_dtype, out)
    kind, M, K, ld = _check_input(x)
    wc, wsc = _check_matrix(w, "w")
    dev, N = x.device, w.rows
    if K != w.cols:
        raise ValueError(f"x has {K} columns, w has {w.cols}")
    if out is None:
        out_kind, ldo = _check_out_dtype(out_dtype), N
        out = torch.empty((M, N), dtype=out_dtype, device=dev)
    else:
        out_kind, rows, cols, ldo = _check_input(out, "out")
        if (rows, cols) != (M, N):
            raise ValueError(f"out must be [{M}, {N}]")
    lib_ = _lib()
    # few rows need none; the library knows up to how many
    nbytes = lib_.mxfp4_linear_workspace_bytes(M, K, N) if M > 1 else 0
    workspace = torch.empty((nbytes,), dtype=torch.uint8, device=dev) if nbytes else None
    st = lib_.mxfp4_linear(x.data_ptr(), kind, M, K, ld, wc, wsc, N, out.data_ptr(), out_kind, ldo, _addr(workspace),
                           _stream_of(dev))
    if st:
        raise MXFP8Error(st, "mxfp4_linear")
    return out


def linear_mxfp4_grouped(x: torch.Tensor, offsets: torch.Tensor, w: MXFP4Matrix, rows: Optional[torch.Tensor] = None,
                         out_dtype: torch.dtype = torch.bfloat16, err_flag: Optional[torch.Tensor] = None,
                         stream=None) -> torch.Tensor:
    """linear_mxfp4 for experts: output row i is x[rows[i]] (x[i] without ``rows``) times expert g's w [N, K] transposed,
    for i in [offsets[g], offsets[g + 1]); w.codes [G, N, .], w.scales [G, .].  Rows past the last offset become zeros.
    ``err_flag`` (device int32) is set to 1 for bad offsets (nothing is written then), an index outside x, or rows past the
    last offset without a negative index."""
    if stream is not None:
        with _on(stream):
            return linear_mxfp4_grouped(x, offsets, w, rows, out_dtype, err_flag)
    kind, T, K, ld = _check_input(x)
    groups = _check_offsets(offsets)
    _check_err(err_flag)
    if rows is not None and (rows.dtype != torch.int32 or rows.dim() != 1 or not rows.is_contiguous()):
        raise ValueError("rows must be a contiguous 1-D int32 tensor")
    wc, wsc = _check_matrix(w, "w", groups)
    out_kind = _check_out_dtype(out_dtype)
    if K != w.cols:
        raise ValueError(f"x has {K} columns, w has {w.cols}")
    R, dev, lib_ = T if rows is None else rows.numel(), x.device, _lib()
    out = torch.empty((R, w.rows), dtype=out_dtype, device=dev)
    nbytes = lib_.mxfp4_linear_grouped_workspace_bytes(R, K, groups)
    workspace = torch.empty((nbytes,), dtype=torch.uint8, device=dev) if nbytes else None
    st = lib_.mxfp4_linear_grouped(x.data_ptr(), kind, T, K, ld, _addr(rows), R, groups, offsets.data_ptr(), wc, wsc, w.rows,
                                   out.data_ptr(), out_kind, _addr(err_flag), _addr(workspace), _stream_of(dev))
    if st:
        raise MXFP8Error(st, "mxfp4_linear_grouped")
    return out
