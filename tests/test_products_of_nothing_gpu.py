"""Experts' products whose sum or output is empty keep the contract of the others: bad offsets write nothing and are told, rows of no
expert become zeros and are told, good offsets give zeros.  All results are exact."""
import pytest
import torch

import mxfp8_block_scaled_04_gb300 as mx

pytestmark = pytest.mark.gpu

BF16, F32, U8 = torch.bfloat16, torch.float32, torch.uint8
GOOD, SHORT = [0, 4, 4, 10], [0, 4, 4, 7]
BAD = [[0, 7, 5, 10], [1, 4, 4, 10], [0, 4, 4, 11], [0, -1, 4, 10], [0, 4, 4, 1 << 62], [-3, 0, 4, 10]]
NONE = [0, 0, 0, 0]
BAD_NONE = [[0, 0, 0, 1], [0, 3, 0, 0], [1, 1, 1, 1], [-1, 0, 0, 0], [0, 0, -2, 0]]


def flag():
    return torch.zeros(1, dtype=torch.int32, device="cuda")


def outputs(call, shape, dtype):
    """call(out, err_flag) on a guarded output: (rows, flag); without a flag the rows are the same."""
    seen = []
    for err in (flag(), None):
        n = 1
        for s in shape:
            n *= s
        buffer = torch.full((n + 64,), 9.0, dtype=dtype, device="cuda")
        assert call(buffer[32:], err) == 0
        assert bool((buffer[:32] == 9).all()) and bool((buffer[n + 32:] == 9).all())
        seen.append(buffer[32:n + 32].view(shape))
        told = int(err) if err is not None else told
    assert torch.equal(seen[0].nan_to_num(5), seen[1].nan_to_num(5))
    assert mx.mxfp8_device_fault_word() == 0
    return seen[0], told


# ---- MXFP8 ---------------------------------------------------------------------------------------------

def product8(kind, R, N, K, off, dtype):
    codes, plane = torch.zeros(4096, dtype=U8, device="cuda"), torch.zeros(4096, dtype=U8, device="cuda")
    shape = {0: (R, N), 1: (R, K), 2: (len(off) - 1, N, K)}[kind]
    offsets = torch.tensor(off, device="cuda")
    return outputs(lambda out, err: mx.mxfp8_matmul_grouped(kind, codes, plane, plane.numel(), 0, codes, plane, plane.numel(), 0, R, N, K, len(off) - 1,
                                                            offsets, out, 0 if dtype is BF16 else 1, err), shape, dtype)


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("kind,N,K", [(0, 48, 0), (1, 0, 48)])
def test_mxfp8_rows_of_an_empty_sum(kind, N, K, dtype):
    out, told = product8(kind, 10, N, K, GOOD, dtype)
    assert bool((out == 0).all()) and told == 0
    out, told = product8(kind, 10, N, K, SHORT, dtype)
    assert bool((out == 0).all()) and told == 1
    for bad in BAD:
        out, told = product8(kind, 10, N, K, bad, dtype)
        assert bool((out == 9).all()) and told == 1, bad


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("N,K", [(16, 16), (48, 1040)])
def test_mxfp8_weight_gradient_of_no_rows(N, K, dtype):
    out, told = product8(2, 0, N, K, NONE, dtype)
    assert bool((out == 0).all()) and told == 0
    out, told = product8(2, 0, N, K, [0] * 513, dtype)
    assert bool((out == 0).all()) and told == 0
    for bad in BAD_NONE + [[0] * 512 + [1], [0] * 300 + [1] + [0] * 212]:
        out, told = product8(2, 0, N, K, bad, dtype)
        assert bool((out == 9).all()) and told == 1, bad


def test_mxfp8_empty_outputs():
    for kind, N, K in ((0, 32, 64), (1, 32, 64)):  # no rows
        assert product8(kind, 0, N, K, NONE, F32)[1] == 0
        for bad in BAD_NONE:
            assert product8(kind, 0, N, K, bad, F32)[1] == 1, (kind, bad)
    for kind, N, K in ((0, 0, 64), (1, 64, 0), (2, 0, 64), (2, 64, 0), (0, 0, 0), (1, 0, 0), (2, 0, 0)):  # no columns
        assert product8(kind, 10, N, K, GOOD, F32)[1] == 0 and product8(kind, 10, N, K, SHORT, F32)[1] == 1
        for bad in BAD:
            assert product8(kind, 10, N, K, bad, F32)[1] == 1, (kind, bad)


def test_mxfp8_wrappers_tell_of_bad_offsets():
    E, N, K = 3, 32, 64
    empty, plane = (lambda cols: torch.empty(0, cols, dtype=U8, device="cuda")), torch.zeros(512, dtype=U8, device="cuda")
    x, dy = (mx.MXFP8Tensor(empty(c), plane, empty(c), plane, None) for c in (K, N))
    w = mx.quantize_grouped(torch.ones(E * N, K, dtype=BF16, device="cuda"), (torch.arange(E + 1) * N).cuda(), swizzled=True)
    for off, told in ((NONE, 0), ([0, 0, 2, 2], 1)):
        for call in (lambda o, e: mx.matmul_mxfp8_grouped(x, o, w, err_flag=e), lambda o, e: mx.matmul_mxfp8_grouped_dgrad(dy, o, w, err_flag=e),
                     lambda o, e: mx.matmul_mxfp8_grouped_wgrad(dy, x, o, err_flag=e)):
            err = flag()
            call(torch.tensor(off, device="cuda"), err)
            assert int(err) == told


# ---- MXFP4 ---------------------------------------------------------------------------------------------

def product4(R, N, K, off, dtype):
    codes, plane = torch.zeros(4096, dtype=U8, device="cuda"), torch.zeros(4096, dtype=U8, device="cuda")
    offsets = torch.tensor(off, device="cuda")
    return outputs(lambda out, err: mx.mxfp4_matmul_grouped(codes, plane, R, len(off) - 1, offsets, codes, plane, N, K, out, 0 if dtype is BF16 else 1, err),
                   (R, N), dtype)


def linear4(R, N, K, off, dtype, rows=None, T=10, workspace=True):
    x = torch.ones(T, max(K, 8), dtype=dtype, device="cuda")
    codes, plane = torch.zeros(1 << 16, dtype=U8, device="cuda"), torch.zeros(1 << 16, dtype=U8, device="cuda")
    offsets = torch.tensor(off, device="cuda")
    rows = None if rows is None else torch.tensor(rows, dtype=torch.int32, device="cuda")
    ws = torch.empty(1 << 16, dtype=U8, device="cuda") if workspace else None
    kind = 0 if dtype is BF16 else 1
    return outputs(lambda out, err: mx.mxfp4_linear_grouped(x, kind, T, K, max(K, 8), rows, R, len(off) - 1, offsets, codes, plane, N, out, kind, err, ws),
                   (R, N), dtype)


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("N", [1, 40, 513])
def test_mxfp4_rows_of_an_empty_sum(N, dtype):
    for call in (product4, linear4):
        out, told = call(10, N, 0, GOOD, dtype)
        assert bool((out == 0).all()) and told == 0
        out, told = call(10, N, 0, SHORT, dtype)
        assert bool((out == 0).all()) and told == 1
        for bad in BAD:
            out, told = call(10, N, 0, bad, dtype)
            assert bool((out == 9).all()) and told == 1, bad


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("groups", [3, 40])  # few rows on many experts take a kernel of their own
def test_uncast_rows_of_an_empty_sum_follow_their_indices(groups, dtype):
    grow = lambda off: off + [off[-1]] * (groups - 3)  # noqa: E731
    rows = [0, 1, 2, 3, 2, 1, 0, -1, -1, -1]
    out, told = linear4(10, 40, 0, grow(SHORT), dtype, rows, T=4, workspace=groups == 3)
    assert bool((out == 0).all()) and told == 0  # a plan marks the rows of no expert
    rows[8] = 2
    out, told = linear4(10, 40, 0, grow(SHORT), dtype, rows, T=4, workspace=groups == 3)
    assert bool((out == 0).all()) and told == 1  # a lost one
    rows[8], rows[1], rows[5] = -1, 4, -1
    out, told = linear4(10, 40, 0, grow(SHORT), dtype, rows, T=4, workspace=groups == 3)
    lost = torch.zeros(10, dtype=torch.bool, device="cuda")
    lost[[1, 5]] = True  # rows that x does not have
    assert bool(out[lost].isnan().all()) and bool((out[~lost] == 0).all()) and told == 1
    for bad in BAD:
        out, told = linear4(10, 40, 0, grow(bad), dtype, rows, T=4, workspace=groups == 3)
        assert bool((out == 9).all()) and told == 1, bad


def test_mxfp4_empty_outputs():
    for K in (0, 64):
        for call in (product4, linear4):
            assert call(0, 40, K, NONE, F32)[1] == 0
            for bad in BAD_NONE:
                assert call(0, 40, K, bad, F32)[1] == 1, bad
            assert call(10, 0, K, GOOD, F32)[1] == 0 and call(10, 0, K, SHORT, F32)[1] == 1
            for bad in BAD:
                assert call(10, 0, K, bad, F32)[1] == 1, bad
        marked = [0, 1, 2, 3, 2, 1, 0, -1, -1, -1]
        assert linear4(10, 0, K, SHORT, F32, marked, T=4)[1] == 0
        assert linear4(10, 0, K, SHORT, F32, marked[:9] + [1], T=4)[1] == 1
        assert linear4(10, 0, K, SHORT, F32, [7] + marked[1:], T=4)[1] == 1


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("plane_bytes", [0, 1, 511, 512])
def test_mxfp8_rows_of_no_expert_need_no_planes(plane_bytes, dtype):
    """Offsets that give no expert a row need none of the ragged planes' bytes; others need more than there are."""
    R, N, K = 10, 48, 80
    codes, plane = torch.full((4096,), 0x7F, dtype=U8, device="cuda"), torch.full((4096,), 127, dtype=U8, device="cuda")
    kind_of = 0 if dtype is BF16 else 1
    for kind, shape in ((0, (R, N)), (1, (R, K)), (2, (3, N, K))):
        w = plane.numel() if kind != 2 else plane_bytes
        for off, value in (([0, 0, 0, 0], 0), ([0, 0, 4, 4], 9), ([0, 0, 0, -1], 9)):
            if plane_bytes == 512 and off[2] == 4:
                continue  # one tile is there
            offsets = torch.tensor(off, device="cuda")
            out, told = outputs(lambda out, err: mx.mxfp8_matmul_grouped(kind, codes, plane, plane_bytes, 0, codes, plane, w, 0, R, N, K, 3, offsets, out, kind_of,
                                                                         err), shape, dtype)
            assert bool((out == value).all()) and told == 1, (kind, off)
