"""Choices outside the experts through the whole chain: plan, gathered cast, experts' products, combination, gradients.

A plan gives such choices the rows past the last expert's (tokens -1).  Those rows hold zero codes and zero products,
and every other row is what its expert makes of its token, against the 64-bit reference (tests/mxfp4_ref.py).
"""
import numpy as np
import pytest
import torch

import mxfp4_ref as ref
import mxfp8_block_scaled_04_gb300 as mx

pytestmark = pytest.mark.gpu

BF16, F32 = torch.bfloat16, torch.float32


def draw(M, N, dtype, seed):
    return torch.randn(M, N, generator=torch.Generator().manual_seed(seed)).to(dtype)


def cast_experts(w):
    parts = [mx.quantize_mxfp4(m.cuda()).row for m in w]
    return mx.MXFP4Matrix(torch.stack([p.codes for p in parts]), torch.stack([p.scales for p in parts]), w.shape[1], w.shape[2])


def poison(nbytes):
    """Leave memory of odd values where the next allocations come from."""
    for n in (nbytes, nbytes // 2, nbytes // 4, 1 << 20, 1 << 18):
        torch.full((max(n, 512),), 0x7B, dtype=torch.uint8, device="cuda")


def choices(T, k, E, kept, seed):
    """Indices [T, k], each inside [0, E) with probability ``kept`` (a boolean mask of them too)."""
    g = torch.Generator().manual_seed(seed)
    idx = torch.randint(0, E, (T, k), generator=g, dtype=torch.int32)
    out = torch.rand(T, k, generator=g) >= kept
    idx[out] = torch.where(torch.rand(int(out.sum()), generator=g) < 0.5, -1, E + 3).to(torch.int32)
    return idx


def check_rows(got, a, w, offsets, bf16):
    """Rows [offsets[g], offsets[g + 1]) of got are a times w[g] transposed (float64), the rows past the last zeros."""
    for g in range(w.shape[0]):
        s = slice(int(offsets[g]), int(offsets[g + 1]))
        want, tol = ref.product_bound(a[s], w[g], bf16)
        assert bool(((got[s].cpu().double() - want).abs() <= tol).all()), g
    assert bool((got[int(offsets[-1]):] == 0).all())


CHAINS = [  # T, k, E, K, N, kept: gathers of more and of fewer rows than tokens, both products' kernels, odd widths
    (40, 3, 5, 72, 40, 0.6), (40, 3, 5, 72, 41, 0.6), (1, 1, 4, 64, 24, 0.0), (7, 8, 3, 40, 9, 0.1), (300, 1, 2, 264, 136, 0.5),
    (64, 2, 512, 32, 8, 0.9), (4100, 2, 2, 64, 512, 0.7), (4100, 2, 2, 96, 515, 0.02), (4100, 2, 2, 64, 512, 0.0)]


@pytest.mark.parametrize("out_dtype", [BF16, F32])
@pytest.mark.parametrize("T,k,E,K,N,kept", CHAINS)
def test_layer_of_a_plan_with_dropped_choices(T, k, E, K, N, kept, out_dtype):
    idx = choices(T, k, E, kept, T + N)
    off, slots, tokens = ref.plan(idx, E)
    used = int(off[-1])
    assert used < T * k
    x, w = draw(T, K, BF16, 1), draw(E * N, K, BF16, 2).view(E, N, K)
    plan = mx.moe_plan(idx.cuda(), E)
    poison(4 * T * k * N)
    gathered = mx.quantize_mxfp4_grouped(x.cuda(), plan.offsets, rows=plan.tokens)
    y = mx.matmul_mxfp4_grouped(gathered, plan.offsets, cast_experts(w), out_dtype)
    codes, _ = ref.quantize(x)
    assert np.array_equal(gathered.codes.cpu().numpy()[:used], codes[tokens[:used].long()])
    assert bool((gathered.codes[used:] == 0).all())
    xv, wv = ref.cast(x), torch.stack([ref.cast(m) for m in w])
    check_rows(y, xv[tokens.long().clamp(min=0)], wv, off, out_dtype == BF16)
    if out_dtype == F32:
        return
    # the combination, and back: the gradient's rows of dropped choices are zeros, their casts and products too
    weights = torch.rand(T, k, generator=torch.Generator().manual_seed(3))
    N8 = N // 8 * 8  # the combination takes rows of whole 16-byte vectors
    y8 = y[:, :N8].contiguous()
    out = mx.moe_combine(y8, plan.slots, weights.cuda())
    live = (slots >= 0).double() * weights.double()
    rows = y8.cpu().double()[slots.long().clamp(min=0)]
    want, mag = (live[:, :, None] * rows).sum(1), (live[:, :, None] * rows.abs()).sum(1)
    assert bool(((out.cpu().double() - want).abs() <= k * 2.0 ** -23 * mag + 2.0 ** -8 * (want.abs() + k * 2.0 ** -23 * mag)).all())
    d = draw(T, N8, BF16, 4)
    dy, dw = mx.moe_combine_backward(d.cuda(), y8, plan.slots, weights.cuda())
    assert bool((dy[used:] == 0).all()) and bool((dw.cpu()[slots < 0] == 0).all())
    poison(4 * T * k * K)
    wt = w[:, :N8].transpose(1, 2).contiguous()
    dq = mx.quantize_mxfp4_grouped(dy, plan.offsets)
    assert bool((dq.codes[used:] == 0).all())
    dx = mx.matmul_mxfp4_grouped(dq, plan.offsets, cast_experts(wt))
    check_rows(dx, ref.cast(dy.cpu()), torch.stack([ref.cast(m) for m in wt]), off, True)
    assert mx.mxfp8_device_fault_word() == 0


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("workspace", [True, False])
def test_left_over_rows_and_the_flag(dtype, workspace):
    """Left over rows marked by a negative index raise no flag; others do, and are still written as zeros.  Nothing
    outside the outputs is touched."""
    T, K, R, G, guard = 5, 72, 12, 3, 1024
    x = draw(T, K, dtype, 1)
    off = torch.tensor([0, 4, 4, 7])
    rows = torch.randint(0, T, (R,), generator=torch.Generator().manual_seed(2), dtype=torch.int32)
    rows[7:] = torch.tensor([-1, -1, -2, -2 ** 31, -1], dtype=torch.int32)
    codes, scale = ref.quantize(x[rows[:7].long()])
    planes = np.concatenate([ref.plane(scale[a:b]) for a, b in ((0, 4), (4, 7))])
    pitch = mx.mxfp4_row_bytes(K)
    work = torch.empty(mx.mxfp4_quantize_grouped_workspace_bytes(T, K, R), dtype=torch.uint8, device="cuda") if workspace else None
    for last, flag in ((-1, 0), (0, 1), (T + 7, 1)):
        rows[R - 1] = last
        buf = torch.full((2 * guard + R * pitch,), 0x5A, dtype=torch.uint8, device="cuda")
        plane = torch.full((mx.mxfp4_grouped_scale_bytes(R, K, G),), 0x5A, dtype=torch.uint8, device="cuda")
        err = torch.zeros(1, dtype=torch.int32, device="cuda")
        out = buf[guard:guard + R * pitch]
        assert mx.mxfp4_quantize_grouped(x.cuda(), 0 if dtype == BF16 else 1, T, K, K, rows.cuda(), R, G, off.cuda(), out, plane, err,
                                         work) == 0
        got = out.view(R, pitch).cpu().numpy()
        assert np.array_equal(got[:7], codes) and not got[7:].any()
        assert np.array_equal(plane.cpu().numpy()[:planes.size], planes)
        assert bool((buf[:guard] == 0x5A).all() and (buf[guard + R * pitch:] == 0x5A).all())
        assert int(err) == flag


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("N", [24, 21])
def test_product_writes_its_rows_and_nothing_past_them(dtype, N):
    """Rows of no expert become zeros between guards; the flag tells of them."""
    R, K, guard = 9, 64, 256
    x, w = draw(R, K, BF16, 1).cuda(), draw(2 * N, K, BF16, 2).view(2, N, K)
    off = torch.tensor([0, 2, 5], device="cuda")
    qa, qb = mx.quantize_mxfp4_grouped(x, off), cast_experts(w)
    buf = torch.full((R * N + 2 * guard,), 3.0, dtype=dtype, device="cuda")
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    assert mx.mxfp4_matmul_grouped(qa.codes, qa.scales, R, 2, off, qb.codes, qb.scales, N, K, buf[guard:], 0 if dtype == BF16 else 1, err) == 0
    check_rows(buf[guard:guard + R * N].view(R, N), ref.cast(x.cpu()), torch.stack([ref.cast(m) for m in w]), off.cpu(), dtype == BF16)
    assert bool((buf[:guard] == 3).all() and (buf[guard + R * N:] == 3).all())
    assert int(err) == 1


def test_offsets_past_the_rows_write_nothing():
    x = draw(6, 64, BF16, 1).cuda()
    for bad in ([0, 2, 7], [0, 7, 6], [1, 2, 6], [0, -1, 6]):
        out = torch.full((6, 32), 0x5A, dtype=torch.uint8, device="cuda")
        plane = torch.full((mx.mxfp4_grouped_scale_bytes(6, 64, 2),), 0x5A, dtype=torch.uint8, device="cuda")
        err = torch.zeros(1, dtype=torch.int32, device="cuda")
        assert mx.mxfp4_quantize_grouped(x, 0, 6, 64, 64, None, 6, 2, torch.tensor(bad, device="cuda"), out, plane, err) == 0
        assert int(err) == 1 and bool((out == 0x5A).all() and (plane == 0x5A).all()), bad
