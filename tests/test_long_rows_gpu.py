"""Columns and summed dimensions past 2^29, where the bytes of a row's scales (16 per 128 columns and row) pass 2^31.

Expected values are exact: powers of two times E2M1 levels, and sums of a few of them.
"""
import pytest
import torch

import mxfp8_block_scaled_04_gb300 as mx

pytestmark = pytest.mark.gpu

BF16, F32 = torch.bfloat16, torch.float32
LEVELS = [0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0]
GUARD = 4096


@pytest.fixture(autouse=True)
def free_memory():
    yield
    torch.cuda.empty_cache()


def scale_bytes(cols, exponent_of_block):
    """The plane of a one-row matrix, block b's exponent from a function of the block numbers (a tensor)."""
    tiles = -(-cols // 128)
    plane = torch.zeros(tiles, 32, 4, 4, dtype=torch.uint8, device="cuda")
    block = torch.arange(4 * tiles, device="cuda").view(tiles, 4)
    plane[:, 0, 0, :] = torch.where(block < -(-cols // 32), exponent_of_block(block) + 127, 0).to(torch.uint8)
    return plane.view(-1)


@pytest.mark.parametrize("cols,dtype", [((1 << 29) + 264, BF16), ((1 << 29) + 260, F32), ((1 << 29) + 259, BF16), ((1 << 30) + 1, F32),
                                        ((1 << 31) - 8, BF16), ((1 << 31) - 1, BF16), ((1 << 31) - 3, F32), ((1 << 31) - 7, BF16)])
def test_decode_of_a_long_row(cols, dtype):
    """Whole vectors and rows off vector boundaries, up to the last column that an int64 below 2^31 allows."""
    pitch = mx.mxfp4_row_bytes(cols)
    at = torch.arange(pitch, device="cuda", dtype=torch.int64)
    codes = ((at * 37 + at // 251) & 0xFF).to(torch.uint8)
    del at
    plane = scale_bytes(cols, lambda b: b % 11 - 5)
    out = torch.full((cols + GUARD,), 77.0, dtype=dtype, device="cuda")
    assert mx.mxfp4_dequantize(codes, plane, 1, cols, out, 0 if dtype == BF16 else 1) == 0
    levels = torch.tensor(LEVELS + [-v for v in LEVELS], device="cuda")
    width = 1 << 20
    for lo in {0, (1 << 29) - width // 2, (1 << 29) + 96, cols // 2, cols - width}:
        hi = min(lo + width, cols)
        c = torch.arange(lo, hi, device="cuda")
        code = (codes[c // 2].int() >> (4 * (c % 2))) & 15
        want = levels[code] * torch.exp2((c // 32 % 11 - 5).float())
        assert torch.equal(out[lo:hi].float(), want), lo
    assert bool((out[cols:] == 77.0).all())


def long_row(K, blocks, values):
    """A one-row 4-bit matrix: ones in the first element of the given blocks times the given powers of two, else zeros."""
    codes = torch.zeros(1, mx.mxfp4_row_bytes(K), dtype=torch.uint8, device="cuda")
    plane = torch.zeros(-(-K // 128), 32, 4, 4, dtype=torch.uint8, device="cuda")
    for b, e in zip(blocks, values):
        codes[0, 16 * b] = 2
        plane[b // 4, 0, 0, b % 4] = 127 + e
    return codes, plane.view(-1)


@pytest.mark.parametrize("K", [(1 << 29) + 512, (1 << 29) + 360])
def test_products_of_long_rows(K):
    """Terms at the start, around K = 2^29 and at the end: exact sums, dense and per expert."""
    blocks = [0, 5, (1 << 24) - 1, 1 << 24, (1 << 24) + 5, -(-K // 32) - 1]
    ea, eb = [0, 3, -2, 4, 1, -4], [1, -1, 2, 3, 5, 2]
    want = sum(2.0 ** (x + y) for x, y in zip(ea, eb))
    a, b = mx.MXFP4Matrix(*long_row(K, blocks, ea), 1, K), mx.MXFP4Matrix(*long_row(K, blocks, eb), 1, K)
    for dtype in (BF16, F32):
        got = mx.matmul_mxfp4(a, b, dtype)
        assert float(got) == float(torch.tensor(want).to(dtype))
    off = torch.tensor([0, 1], device="cuda")
    experts = mx.MXFP4Matrix(b.codes[None], b.scales[None], 1, K)
    assert float(mx.matmul_mxfp4_grouped(a, off, experts, F32)) == want
    assert mx.mxfp8_device_fault_word() == 0
