"""Gradients of the 4-bit linear layer against differences of its own output, repeats of every kernel, and every product
kernel on streams at once.
"""
import pytest
import torch

import mxfp8_block_scaled_04_gb300 as mx

pytestmark = pytest.mark.gpu

BF16, F32 = torch.bfloat16, torch.float32
LEVELS = torch.tensor([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0])


def levels(rows, cols, seed):
    """A matrix of E2M1 levels and their negatives: both casts hold it exactly (a block whose largest element is below 4
    is scaled by a power of two that keeps its levels on the grid)."""
    g = torch.Generator().manual_seed(seed)
    v = LEVELS[torch.randint(0, 8, (rows, cols), generator=g)]
    return torch.where(torch.rand(rows, cols, generator=g) < 0.5, -v, v)


@pytest.mark.parametrize("T,K,N", [(1, 64, 40), (5, 72, 264), (67, 264, 136), (130, 512, 384), (1030, 64, 4104)])
def test_gradients_against_differences_of_the_products(T, K, N):
    """L = sum(dy * (x w^T)).  Moving one element of x or w from a level to another moves L by the gradient times the step;
    every operand is exact in four bits and every sum a multiple of 1/4 below 2^22, so the differences of the
    package's own outputs equal the package's own gradients."""
    x, w, dy = levels(T, K, 1).cuda(), levels(N, K, 2).cuda(), levels(T, N, 3).cuda()
    qx, qw, qd = (mx.quantize_mxfp4(v, colwise=True) for v in (x, w, dy))
    for q, v in ((qx, x), (qw, w), (qd, dy)):
        assert torch.equal(mx.dequantize_mxfp4(q.row, F32), v) and torch.equal(mx.dequantize_mxfp4(q.col, F32), v.t())
    y = mx.matmul_mxfp4(qx.row, qw.row, F32).double()
    dx, dw = mx.matmul_mxfp4(qd.row, qw.col, F32), mx.matmul_mxfp4(qd.col, qx.col, F32)
    assert dx.shape == x.shape and dw.shape == w.shape
    g = torch.Generator().manual_seed(4)
    for first, grad in ((x, dx), (w, dw)):
        rows, cols = first.shape
        for _ in range(6):
            r, c = int(torch.randint(0, rows, (1,), generator=g)), int(torch.randint(0, cols, (1,), generator=g))
            moved = first.clone()
            moved[r, c] = 6.0 if float(first[r, c]) < 2 else -1.5
            step = float(moved[r, c] - first[r, c])
            q = mx.quantize_mxfp4(moved).row
            out = mx.matmul_mxfp4(q, qw.row, F32) if first is x else mx.matmul_mxfp4(qx.row, q, F32)
            slope = ((out.double() - y) * dy.double()).sum() / step
            assert float(slope) == float(grad[r, c]), (r, c)


def experts(E, N, K, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    parts = [mx.quantize_mxfp4(torch.randn(N, K, generator=g, device="cuda").to(BF16)).row for _ in range(E)]
    return mx.MXFP4Matrix(torch.stack([p.codes for p in parts]), torch.stack([p.scales for p in parts]), N, K)


def routed(T, k, E, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return mx.moe_plan(torch.rand(T, E, generator=g, device="cuda").topk(k, 1).indices.int(), E)


def bits(v):
    """The tensors of a result, as bytes."""
    if isinstance(v, torch.Tensor):
        return [v.contiguous().view(torch.uint8)]
    if isinstance(v, mx.MXFP4Matrix):
        return [v.codes, v.scales]
    return [b for part in v if part is not None for b in bits(part)]


def jobs():
    """A call of every kernel of the casts and products: (name, call)."""
    g = torch.Generator(device="cuda").manual_seed(0)

    def rnd(*s):
        return torch.randn(*s, generator=g, device="cuda")
    out = []
    for name, x in (("bf16", rnd(1000, 2056).to(BF16)), ("fp32", rnd(777, 1032))):
        out += [(f"cast {name}", lambda x=x: mx.quantize_mxfp4(x)),
                (f"cast both ways {name}", lambda x=x: mx.quantize_mxfp4(x, colwise=True))]
        q = mx.quantize_mxfp4(x, colwise=True).col
        out += [(f"decode {name}", lambda q=q: mx.dequantize_mxfp4(q)), (f"decode to fp32 {name}", lambda q=q: mx.dequantize_mxfp4(q, F32))]
    for M, N, K in ((1, 4096, 4096), (300, 1024, 2048), (100, 512, 16384), (2048, 2048, 512)):
        a, b = (mx.quantize_mxfp4(rnd(r, K).to(BF16)).row for r in (M, N))
        out += [(f"product {M}x{N}x{K} {dt}", lambda a=a, b=b, dt=dt: mx.matmul_mxfp4(a, b, dt)) for dt in (BF16, F32)]
    for T, E, N, K in ((40, 16, 520, 256), (2100, 4, 1024, 264)):  # the kernel for few rows per expert, and the pairs'
        x, plan, w = rnd(T, K).to(BF16), routed(T, 2, E, T), experts(E, N, K, T)
        q = mx.quantize_mxfp4_grouped(x, plan.offsets, rows=plan.tokens)
        rows = x[plan.tokens.long()]
        out += [(f"gathered cast {T}", lambda x=x, p=plan: mx.quantize_mxfp4_grouped(x, p.offsets, rows=p.tokens).codes),
                (f"cast in order {T}", lambda x=rows, p=plan: mx.quantize_mxfp4_grouped(x, p.offsets).codes)]
        out += [(f"experts' product {T} {dt}", lambda q=q, p=plan, w=w, dt=dt: mx.matmul_mxfp4_grouped(q, p.offsets, w, dt)) for dt in (BF16, F32)]
    return out


def test_every_cast_and_product_repeats_its_bits():
    for name, call in jobs():
        first = bits(call())
        for _ in range(5):
            again = bits(call())
            assert len(again) == len(first) and all(torch.equal(a, b) for a, b in zip(again, first)), name
    assert mx.mxfp8_device_fault_word() == 0


def test_every_cast_and_product_on_streams_at_once():
    """Each job on a stream of its own, ten times over: the results are those of the job alone."""
    work = jobs()
    alone = [bits(call()) for _, call in work]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(6)]
    results = []
    for turn in range(10):
        for i, (_, call) in enumerate(work):
            with torch.cuda.stream(streams[(i + turn) % len(streams)]):
                results.append((i, call()))
    torch.cuda.synchronize()
    for i, r in results:
        assert all(torch.equal(a, b) for a, b in zip(bits(r), alone[i])), work[i][0]
    assert mx.mxfp8_device_fault_word() == 0
