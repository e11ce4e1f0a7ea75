"""Plain 64-bit values of grouped MXFP8 casts, from their codes and GEMM-ready planes (torch CPU), and the products' bound."""
import torch


def elements(codes: torch.Tensor, fmt: str) -> torch.Tensor:
    """float64 values of FP8 codes from their fields (E4M3: no infinities, one NaN; E5M2: as IEEE)."""
    c = codes.cpu().long()
    mbits, bias = (3, 7) if fmt == "e4m3" else (2, 15)
    e, m = (c & 127) >> mbits, (c & ((1 << mbits) - 1)).double()
    one = float(1 << mbits)
    mag = torch.where(e == 0, m / one * 2.0 ** (1 - bias), (1 + m / one) * 2.0 ** (e - bias).double())
    if fmt == "e4m3":
        mag = torch.where((c & 127) == 127, torch.full_like(mag, float("nan")), mag)
    else:
        mag = torch.where(e == 31, torch.where(m == 0, float("inf"), float("nan")).double(), mag)
    return torch.where(c >= 128, -mag, mag)


def scales(plane: torch.Tensor, rows: int, blocks: int) -> torch.Tensor:
    """float64 scales [rows, blocks] of one plane."""
    r, b = torch.arange(rows)[:, None], torch.arange(blocks)[None]
    at = ((r // 128) * -(-blocks // 4) + b // 4) * 512 + 16 * (r % 32) + 4 * (r % 128 // 32) + b % 4
    byte = plane.cpu().long()[at]
    return torch.where(byte == 255, float("nan"), 2.0 ** (byte - 127).double())


def groups(codes, plane, offsets, fmt: str, rowwise: bool):
    """Each group's values [rows_g, C], float64."""
    v, C, at, out = elements(codes, fmt), codes.shape[1], 0, []
    for a, b in zip(offsets[:-1], offsets[1:]):
        n = b - a
        shape = (n, -(-C // 32)) if rowwise else (C, -(-n // 32))
        size = -(-shape[0] // 128) * -(-shape[1] // 4) * 512 if n else 0
        if n:
            s = scales(plane[at:at + size], *shape)
            s = s.repeat_interleave(32, 1)[:, :C] if rowwise else s.t().repeat_interleave(32, 0)[:n]
            out.append(v[a:b] * s)
        else:
            out.append(torch.zeros(0, C, dtype=torch.float64))
        at += size
    return out


def product_bound(a: torch.Tensor, b: torch.Tensor, bf16: bool):
    """(a @ b.T, allowed error).  Products are exact; each of the K additions may drop up to one unit of the last of 24 bits
    of a partial sum, which is at most sum |a||b|; bf16 adds half a unit of the last of its 8 bits."""
    want = a @ b.t()
    tol = a.shape[1] * 2.0 ** -23 * (a.abs() @ b.abs().t())
    return want, tol + (2.0 ** -8 * (want.abs() + tol) if bf16 else 0.0)
