"""examples/expert_block.py: norms, routing, MXFP8 products with every gradient, and serving from 4-bit weights, together.

Each step is recomputed in 64 bits from the block's own intermediate results, with the single operators' tolerances; then
the block as a whole against one that casts nothing; then repeats, streams at once and CUDA graphs.
"""
import importlib.util
import os

import pytest
import torch

import mxfp4_ref as ref4
import mxfp8_ref as ref8

pytestmark = pytest.mark.gpu

PATH = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples", "expert_block.py")
spec = importlib.util.spec_from_file_location("expert_block", PATH)
example = importlib.util.module_from_spec(spec)
spec.loader.exec_module(example)
mx = example.mx
BF16, F32 = torch.bfloat16, torch.float32


def draw(T, H, seed):
    return torch.randn(T, H, generator=torch.Generator(device="cuda").manual_seed(seed), device="cuda").to(BF16)


def inside(got, want, tol, what):
    bad = ~((got.cpu().double() - want).abs() <= tol)
    assert not bool(bad.any()), (what, int(bad.sum()))


def check_experts(got, pairs, off, bf16, what):
    """Rows of each expert (or its matrix) are a @ b.T of the 64-bit values."""
    for e, (a, b) in enumerate(pairs):
        want, tol = ref8.product_bound(a, b, bf16)
        inside(got[e] if off is None else got[off[e]:off[e + 1]], want, tol, (what, e))


def rows(t, off, fmt):
    return ref8.groups(t.out_row, t.scale_row, off, fmt, True)


def cols(t, off, fmt):
    return ref8.groups(t.out_col, t.scale_col, off, fmt, False)


SIZES = [(1, 256, 128, 8, 2), (37, 272, 144, 8, 3), (700, 512, 272, 4, 2)]


@pytest.mark.parametrize("tokens,hidden,ffn,experts,k", SIZES)
def test_training_step_by_step(tokens, hidden, ffn, experts, k):
    block = example.ExpertBlock(hidden, ffn, experts, k, scale=0.9)
    h, gx, gh = (draw(tokens, hidden, s) for s in (1, 2, 3))
    x = mx.block_norm(None, h, block.pre).x
    nx, nh, s = block.forward(x, h)
    off = s.plan.offsets.tolist()
    w1_off, w2_off = [e * 2 * ffn for e in range(experts + 1)], [e * hidden for e in range(experts + 1)]
    check_experts(s.ab, zip(rows(s.rows, off, "e4m3"), rows(block.q1, w1_off, "e4m3")), off, True, "ab")
    check_experts(s.y, zip(rows(s.inner, off, "e4m3"), rows(block.q2, w2_off, "e4m3")), off, True, "y")
    # the norm behind the block: 64 bits from the block's output, then of the stream as it is kept
    out, hd = s.out.double(), h.double()
    rms = lambda v: v / torch.sqrt((v * v).mean(1, keepdim=True) + 1e-6)  # noqa: E731
    v = block.gate.double() * rms(out) * block.post.double()
    mag = (0.9 * hd).abs() + v.abs()
    inside(nh, (0.9 * hd + v).cpu(), (2.0 ** -18 * mag + 2.0 ** -8 * (1 + 2.0 ** -18) * mag).cpu(), "h")
    want = rms(nh.double()) * block.pre.double()
    inside(nx, want.cpu(), (2.0 ** -8 + 2.0 ** -17) * want.abs().cpu(), "x")
    # backward, from the same casts that it makes
    g = block.backward(gx, gh, s)
    n = mx.block_norm_backward(gh, gx, s.out, s.h, block.pre, block.post, block.gate, 0.9)
    dy, _ = mx.moe_combine_backward(n.y, s.y, s.plan.slots, s.route.weights)
    qdy = mx.quantize_grouped(dy, s.plan.offsets, mx.E5M2, swizzled=True)
    check_experts(g["w2"], zip((d.t() for d in cols(qdy, off, "e5m2")), (i.t() for i in cols(s.inner, off, "e4m3"))), None, False, "w2")
    dinner = mx.matmul_mxfp8_grouped_dgrad(qdy, s.plan.offsets, block.q2)
    check_experts(dinner, zip(rows(qdy, off, "e5m2"), (w.t() for w in cols(block.q2, w2_off, "e4m3"))), off, True, "dinner")
    qdab = mx.quantize_grouped(example.swiglu_backward(s.ab, dinner), s.plan.offsets, mx.E5M2, swizzled=True)
    check_experts(g["w1"], zip((d.t() for d in cols(qdab, off, "e5m2")), (r.t() for r in cols(s.rows, off, "e4m3"))), None, False, "w1")
    drows = mx.matmul_mxfp8_grouped_dgrad(qdab, s.plan.offsets, block.q1)
    check_experts(drows, zip(rows(qdab, off, "e5m2"), (w.t() for w in cols(block.q1, w1_off, "e4m3"))), off, True, "drows")
    for name, t in (("h", n.h), ("pre", n.pre_weight), ("post", n.post_weight), ("gate", n.gate)):
        assert torch.equal(g[name], t)
    assert all(bool(torch.isfinite(t).all()) for t in g.values())
    assert mx.mxfp8_device_fault_word() == 0


@pytest.mark.parametrize("tokens,hidden,ffn,experts,k", SIZES)
def test_serving_step_by_step(tokens, hidden, ffn, experts, k):
    block = example.ExpertBlock(hidden, ffn, experts, k)
    h = draw(tokens, hidden, 4)
    x = mx.block_norm(None, h, block.pre).x
    served = block.serve(x, h)
    route = mx.moe_route(x.float() @ block.router.float().t(), k, **block.how)
    plan = mx.moe_plan(route.indices, experts)
    off = plan.offsets.tolist()
    ab = mx.linear_mxfp4_grouped(x, plan.offsets, block.s1, rows=plan.tokens)
    inner = example.swiglu(ab)
    y = mx.linear_mxfp4_grouped(inner, plan.offsets, block.s2)
    for got, a, w in ((ab, x[plan.tokens.long()], block.w1), (y, inner, block.w2)):
        a = a.cpu().double()
        for e in range(experts):
            s, b = slice(off[e], off[e + 1]), ref4.cast(w[e].cpu())
            want = a[s] @ b.t()
            # eight parts of at most 4 |a| together, which miss 2^-22 of the block's largest
            top = a[s].abs().amax(1, keepdim=True) if off[e + 1] > off[e] else a[s].abs().sum(1, keepdim=True)
            tol = ((a.shape[1] + 8) * 2.0 ** -23 * 4 * a[s].abs() + 2.0 ** -22 * top) @ b.abs().t()
            inside(got[s], want, tol + 2.0 ** -8 * (want.abs() + tol), e)
    want = block.norm(mx.moe_combine(y, plan.slots, route.weights), h)
    assert torch.equal(served.x, want.x) and torch.equal(served.h, want.h)


def test_block_against_the_one_that_casts_nothing():
    """A cast to E4M3 errs by 2^-5 rms of an element at most (E5M2 2^-4), one to 4 bits by about 0.12 of a normal block's rms.
    Four 8-bit casts on the way to a result make at most 0.1 of its rms, eight casts of a gradient 0.35: cosines of 0.99 and
    0.94.  Held to 0.98 and 0.9 (serving, four 4-bit casts of weights alone: 0.9); an operand in the wrong place gives 0."""
    block = example.ExpertBlock(512, 256, 8, 2)
    h, gx, gh = (draw(600, 512, s) for s in (5, 6, 7))
    got = example.compare(block, mx.block_norm(None, h, block.pre).x, h, gx, gh)
    for name, cosine in got.items():
        assert cosine >= (0.9 if name.startswith(("grad", "served")) else 0.98), got


def calls():
    """Every new call, at sizes of each of its kernels: (name, call), tensors out."""
    out = []
    for tokens, hidden, ffn, experts, k in SIZES + [(3000, 512, 528, 2, 1)]:
        block = example.ExpertBlock(hidden, ffn, experts, k)
        h, gx, gh = (draw(tokens, hidden, 8 + s) for s in range(3))
        x = mx.block_norm(None, h, block.pre).x
        nx, nh, s = block.forward(x, h)
        qdab = mx.quantize_grouped(draw(s.ab.shape[0], s.ab.shape[1], 11), s.plan.offsets, mx.E5M2, swizzled=True)
        w4 = mx.quantize_mxfp4(block.w1[0]).row

        def add(name, call):
            out.append((f"{name} {tokens}x{hidden}", call))
        add("forward", lambda s=s, b=block: [mx.matmul_mxfp8_grouped(s.rows, s.plan.offsets, b.q1, dt) for dt in (BF16, F32)])
        add("dgrad", lambda s=s, b=block, q=qdab: [mx.matmul_mxfp8_grouped_dgrad(q, s.plan.offsets, b.q1, dt) for dt in (BF16, F32)])
        add("wgrad", lambda s=s, q=qdab: [mx.matmul_mxfp8_grouped_wgrad(q, s.rows, s.plan.offsets, dt) for dt in (BF16, F32)])
        add("linear", lambda x=x, w=w4: [mx.linear_mxfp4(x, w, dt) for dt in (BF16, F32)])
        add("experts' linear", lambda x=x, s=s, b=block: [mx.linear_mxfp4_grouped(x, s.plan.offsets, b.s1, rows=s.plan.tokens)])
        add("norm", lambda s=s, b=block, h=h: list(b.norm(s.out, h)))
        add("norm's gradient", lambda s=s, b=block, gx=gx, gh=gh: list(mx.block_norm_backward(gh, gx, s.out, s.h, b.pre, b.post, b.gate, 0.5)))
    for H in (9000, 16384):
        y, h = draw(50, H, 12), draw(50, H, 13)
        w = torch.ones(H, device="cuda")
        out.append((f"norm {H}", lambda y=y, h=h, w=w: list(mx.block_norm(y, h, w, w, w))))
        out.append((f"norm's gradient {H}", lambda y=y, h=h, w=w: list(mx.block_norm_backward(h, y, y, h, w, w, w))))
    return out


def test_every_call_repeats_its_bits():
    for name, call in calls():
        first = call()
        for _ in range(4):
            assert all(torch.equal(a, b) for a, b in zip(call(), first)), name
    assert mx.mxfp8_device_fault_word() == 0


def test_every_call_on_streams_at_once():
    work = calls()
    alone = [call() for _, call in work]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(5)]
    results = []
    for turn in range(6):
        for i, (_, call) in enumerate(work):
            with torch.cuda.stream(streams[(i + turn) % len(streams)]):
                results.append((i, call()))
    torch.cuda.synchronize()
    for i, r in results:
        assert all(torch.equal(a, b) for a, b in zip(r, alone[i])), work[i][0]
    assert mx.mxfp8_device_fault_word() == 0


def test_a_given_stream_owns_the_outputs():
    block = example.ExpertBlock(256, 128, 4, 2)
    h = draw(30, 256, 1)
    x = mx.block_norm(None, h, block.pre).x
    w4 = mx.quantize_mxfp4(block.w1[0]).row
    want = mx.linear_mxfp4(x, w4)
    stream = torch.cuda.Stream()
    stream.wait_stream(torch.cuda.current_stream())
    got = [mx.linear_mxfp4(x, w4, stream=stream), mx.linear_mxfp4(x, w4, stream=stream.cuda_stream)]
    norm = mx.block_norm(x, h, block.pre, stream=stream)
    stream.synchronize()
    assert all(torch.equal(g, want) for g in got) and torch.equal(norm.x, mx.block_norm(x, h, block.pre).x)


def test_captured_graphs_follow_their_inputs():
    """Two graphs of every call, captured one after the other and replayed in turn on changed inputs: each replay gives
    what the calls give."""
    block = example.ExpertBlock(512, 272, 4, 2)
    graphs = []
    for seed in (1, 2):
        h, gx = draw(64, 512, seed), draw(64, 512, seed + 10)
        x = mx.block_norm(None, h, block.pre).x
        _, _, s = block.forward(x, h)
        qdab = mx.quantize_grouped(draw(s.ab.shape[0], s.ab.shape[1], seed + 20), s.plan.offsets, mx.E5M2, swizzled=True)

        def run(x=x, h=h, gx=gx, s=s, q=qdab):
            y = mx.linear_mxfp4_grouped(x, s.plan.offsets, block.s1, rows=s.plan.tokens)
            n = block.norm(x, h)
            g = mx.block_norm_backward(gx, n.x, x, n.h, block.pre, block.post, block.gate)
            return [y, n.x, n.h, *g, mx.matmul_mxfp8_grouped(s.rows, s.plan.offsets, block.q1),
                    mx.matmul_mxfp8_grouped_dgrad(q, s.plan.offsets, block.q1), mx.matmul_mxfp8_grouped_wgrad(q, s.rows, s.plan.offsets)]
        run()
        torch.cuda.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            out = run()
        graphs.append((graph, out, run, (x, h, gx)))
    for turn in range(3):
        for graph, out, run, inputs in graphs:
            for t in inputs:
                t.mul_(0.75).add_(0.125)
            graph.replay()
        torch.cuda.synchronize()
        for graph, out, run, inputs in graphs:
            assert all(torch.equal(a, b) for a, b in zip(out, run())), turn
    assert mx.mxfp8_device_fault_word() == 0


def test_rows_of_no_expert_and_bad_offsets():
    """MXFP8 products: rows past the last offset become zeros (the weight gradient leaves them out), bad offsets write nothing."""
    E, R, N, K = 3, 100, 144, 272
    off = torch.tensor([0, 30, 30, 77])
    x, dy, w = draw(R, K, 1), draw(R, N, 2), draw(E * N, K, 3)
    inner = slice(0, 77)
    qx, qdy = (mx.quantize_grouped(t[inner].contiguous(), off.cuda(), swizzled=True) for t in (x, dy))
    qw = mx.quantize_grouped(w, (torch.arange(E + 1) * N).cuda(), swizzled=True)

    def longer(t):  # the same casts with rows of no expert behind them
        pad = lambda c: torch.cat((c, torch.full((R - 77, c.shape[1]), 0x7F, dtype=torch.uint8, device="cuda")))  # noqa: E731
        return t._replace(out_row=pad(t.out_row), out_col=pad(t.out_col))
    lx, ldy = longer(qx), longer(qdy)
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    for call, short in ((lambda a, b, o, **k: mx.matmul_mxfp8_grouped(a, o, qw, **k), False),
                        (lambda a, b, o, **k: mx.matmul_mxfp8_grouped_dgrad(b, o, qw, grad_fmt="e4m3", **k), False),
                        (lambda a, b, o, **k: mx.matmul_mxfp8_grouped_wgrad(b, a, o, grad_fmt="e4m3", **k), True)):
        want = call(qx, qdy, off.cuda(), err_flag=err)
        assert int(err) == 0
        got = call(lx, ldy, off.cuda(), err_flag=err)
        assert int(err) == 1
        err.zero_()
        if short:
            assert torch.equal(got, want)
        else:
            assert torch.equal(got[:77], want) and bool((got[77:] == 0).all())
    for bad in ([0, 30, 20, 77], [1, 30, 30, 77], [0, 30, 30, 101], [0, -5, 30, 77], [0, 30, 30, 1 << 60]):
        for kind, a, b, shape in ((0, (qx.out_row, qx.scale_row), (qw.out_row, qw.scale_row), (R, N)),
                                  (1, (qdy.out_row, qdy.scale_row), (qw.out_col, qw.scale_col), (R, K)),
                                  (2, (qdy.out_col, qdy.scale_col), (qx.out_col, qx.scale_col), (E, N, K))):
            err.zero_()
            out = torch.full(shape, 9.0, device="cuda")
            assert mx.mxfp8_matmul_grouped(kind, a[0], a[1], a[1].numel(), 0, b[0], b[1], b[1].numel(), 0, 77, N, K, E,
                                           torch.tensor(bad).cuda(), out, 1, err) == 0
            assert int(err) == 1 and bool((out == 9).all()), (bad, kind)
    # planes too small for the offsets are bad offsets too
    err.zero_()
    out = torch.full((R, N), 9.0, device="cuda")
    assert mx.mxfp8_matmul_grouped(0, qx.out_row, qx.scale_row, qx.scale_row.numel() // 2, 0, qw.out_row, qw.scale_row, qw.scale_row.numel(), 0, 77, N, K, E,
                                   off.cuda(), out, 1, err) == 0
    assert int(err) == 1 and bool((out == 9).all())


def test_products_of_nothing():
    off = torch.zeros(4, dtype=torch.int64, device="cuda")
    empty, plane = (lambda cols: torch.empty(0, cols, dtype=torch.uint8, device="cuda")), torch.zeros(1, dtype=torch.uint8, device="cuda")
    none, dy = (mx.MXFP8Tensor(empty(c), plane, empty(c), plane, None) for c in (64, 32))
    w = mx.quantize_grouped(draw(3 * 32, 64, 1), (torch.arange(4) * 32).cuda(), swizzled=True)
    assert mx.matmul_mxfp8_grouped(none, off, w).shape == (0, 32)
    assert mx.matmul_mxfp8_grouped_dgrad(dy, off, w).shape == (0, 64)
    dw = mx.matmul_mxfp8_grouped_wgrad(dy, none, off)
    assert dw.shape == (3, 32, 64) and bool((dw == 0).all())
