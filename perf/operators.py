"""Cases of the 4-bit and expert-layer operators: MXFP4 cast, product, experts' product, routing, combination.

``run`` computes each operator in a plain form (elementary torch operations in fp32) or, with ``own``
set, through the package's public calls.  Data layout shared by both: a 4-bit matrix [R, C] is held as
uint8 codes [R, ceil(C/32)*16] (element 2i in the low half of byte i, the tail zero) and one 1-D plane
of E8M0 bytes in 128x4 tiles (entry (r, c) of a tile at 16*(r % 32) + 4*(r // 32) + c).
"""
import math

import torch

own = False

SCORES = ("softmax", "sigmoid")


# ---- cases -----------------------------------------------------------------------------------------

def listed():
    return [
        # An MLP's activations in training, cast both ways (the second for the weight gradient).
        {"name": "cast_both_8192x28672", "op": "cast", "M": 8192, "N": 28672, "dtype": "bf16", "cols": True},
        # An fp32 gradient of an odd number of rows whose last blocks are partial, both ways.
        {"name": "cast_both_fp32_4093x7176", "op": "cast", "M": 4093, "N": 7176, "dtype": "fp32", "cols": True},
        # One token through an MLP's first layer: the weights' bytes are the work.
        {"name": "linear_1x8192x28672", "op": "linear", "M": 1, "K": 8192, "N": 28672, "out": "bf16"},
        # A ragged mid-size batch through a square layer.
        {"name": "linear_333x4096x4096", "op": "linear", "M": 333, "K": 4096, "N": 4096, "out": "bf16"},
        # A training forward at full size.
        {"name": "linear_8192x8192x28672", "op": "linear", "M": 8192, "K": 8192, "N": 28672, "out": "bf16"},
        # A training step of one layer (output, input gradient, fp32 weight gradient), an odd number of tokens.
        {"name": "train_4099x8192x8192", "op": "train", "M": 4099, "K": 8192, "N": 8192},
        # Sixteen tokens of a serving step, eight experts each, through 64 experts.
        {"name": "experts_64x128x7168x2048", "op": "experts", "T": 16, "k": 8, "E": 64, "K": 7168, "N": 2048,
         "skew": 0.5},
        # A long prefill through 64 experts of unequal load.
        {"name": "experts_64x65536x7168x2048", "op": "experts", "T": 8192, "k": 8, "E": 64, "K": 7168, "N": 2048,
         "skew": 0.3},
        # Routing of a serving step: bf16 logits, softmax, no bias.
        {"name": "route_16x64", "op": "route", "T": 16, "E": 64, "k": 8, "score": "softmax", "bias": False,
         "groups": 1, "topk_groups": 1, "renorm": True, "dtype": "bf16", "grad": False},
        # Routing of a training batch and its gradient: sigmoid scores, a bias for balance, groups.
        {"name": "route_train_65536x256", "op": "route", "T": 65536, "E": 256, "k": 8, "score": "sigmoid",
         "bias": True, "groups": 8, "topk_groups": 4, "renorm": True, "dtype": "fp32", "grad": True},
        # Combination of the experts' rows of a training batch, with its gradients (the plan included).
        {"name": "combine_train_8192x8x7168", "op": "combine", "T": 8192, "k": 8, "E": 64, "H": 7168, "grad": True},
        # The same of a serving step's sixteen tokens, forward only.
        {"name": "combine_16x8x7168", "op": "combine", "T": 16, "k": 8, "E": 64, "H": 7168, "grad": False},
    ]


def _log(rng, lo, hi, step=1):
    v = int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))
    return max(step, v // step * step)


def draw(rng):
    op = rng.choice(["cast", "linear", "train", "experts", "route", "combine"])
    if op == "cast":
        while True:
            c = {"op": op, "M": _log(rng, 1, 16384), "N": _log(rng, 64, 28672, 8),
                 "dtype": rng.choice(["bf16", "fp32"]), "cols": rng.random() < 0.6}
            if c["M"] * c["N"] <= (8192 * 28672 if c["dtype"] == "bf16" else 4096 * 28672):
                return c
    if op == "linear":
        return {"op": op, "M": _log(rng, 1, 8192), "K": _log(rng, 256, 8192, 8), "N": _log(rng, 128, 28672, 8),
                "out": rng.choice(["bf16", "fp32"])}
    if op == "train":
        return {"op": op, "M": _log(rng, 16, 4099), "K": _log(rng, 256, 8192, 8), "N": _log(rng, 256, 8192, 8)}
    if op == "experts":
        E = rng.choice([4, 8, 16, 64])
        return {"op": op, "T": _log(rng, 1, 8192), "k": rng.randint(1, min(E, 8)), "E": E,
                "K": _log(rng, 512, 7168, 8), "N": _log(rng, 256, 2048, 8), "skew": rng.choice([0.0, 0.3, 0.5])}
    if op == "route":
        E = rng.choice([8, 64, 96, 128, 160, 256])
        groups = rng.choice([1, 4, 8])
        topk_groups = rng.randint(max(1, groups // 2), groups)
        return {"op": op, "T": _log(rng, 1, 65536), "E": E, "k": rng.randint(1, min(8, E // groups * topk_groups)),
                "score": rng.choice(SCORES), "bias": rng.random() < 0.5, "groups": groups,
                "topk_groups": topk_groups, "renorm": rng.random() < 0.7, "dtype": rng.choice(["bf16", "fp32"]),
                "grad": rng.random() < 0.6}
    return {"op": op, "T": _log(rng, 1, 8192), "k": rng.randint(1, 8), "E": rng.choice([8, 64, 160, 256]),
            "H": _log(rng, 512, 7168, 8), "grad": rng.random() < 0.6}


# ---- inputs ----------------------------------------------------------------------------------------

def _gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(int(seed) * 1000003 + 17)
    return g


def _randn(g, *shape):
    return torch.randn(shape, generator=g, device="cuda", dtype=torch.float32)


def _rand(g, *shape):
    return torch.rand(shape, generator=g, device="cuda", dtype=torch.float32)


def _activation(g, M, N, dtype):
    """Normal values under a spread of row scales, one in a thousand an outlier, one row in fifty zero."""
    x = _randn(g, M, N)
    x *= torch.exp(_randn(g, M, 1))
    x *= torch.where(_rand(g, M, N) < 1e-3, 40.0, 1.0)
    if M > 1:
        x *= (_rand(g, M, 1) >= 0.02).float()
    return x.to(dtype)


def _weight(g, R, C):
    return (_randn(g, R, C) * 0.02).to(torch.bfloat16)


def _pack(w):
    """A layer's weights as a user keeps them: codes and GEMM-ready scale planes of w [B, R, C] (C % 32 == 0)."""
    B, R, C = w.shape
    values, e = _blocks(w.float())
    a = values.abs()
    code = (2.0 * a.clamp(max=2.0) + (a - 2.0).clamp(0.0, 2.0) + 0.5 * (a - 4.0).clamp(min=0.0)).to(torch.uint8)
    code = (code + 8 * (values < 0).to(torch.uint8)).view(B, R, -1)
    codes = code[..., 0::2] + 16 * code[..., 1::2]
    byte = (e + 127).to(torch.uint8)
    byte = torch.nn.functional.pad(byte, (0, -byte.shape[2] % 4, 0, -R % 128))
    tiles = byte.view(B, byte.shape[1] // 128, 4, 32, byte.shape[2] // 4, 4)
    return codes.contiguous(), tiles.permute(0, 1, 4, 3, 2, 5).reshape(B, -1).contiguous()


def _dtype(name):
    return {"bf16": torch.bfloat16, "fp32": torch.float32}[name]


def _pad32(w):
    return torch.nn.functional.pad(w, (0, -w.shape[-1] % 32))


def _sizes(case, seed):
    """Chosen experts [T, k] of a batch whose experts are loaded unequally (distinct within a token)."""
    g = _gen(seed + 7)
    popularity = _randn(g, 1, case["E"]) * case.get("skew", 0.3)
    noise = -torch.log(-torch.log(_rand(g, case["T"], case["E"]).clamp(1e-7, 1 - 1e-7)))
    return (popularity + noise).topk(case["k"], dim=1).indices.to(torch.int32)


def prepare(case, seed):
    g = _gen(seed)
    op = case["op"]
    s = dict(case)
    if op == "cast":
        s["x"] = _activation(g, case["M"], case["N"], _dtype(case["dtype"]))
    elif op == "linear":
        s["x"] = _activation(g, case["M"], case["K"], torch.bfloat16)
        codes, scales = _pack(_pad32(_weight(g, case["N"], case["K"]))[None])
        s["w"] = (codes[0], scales[0])
    elif op == "train":
        s["x"] = _activation(g, case["M"], case["K"], torch.bfloat16)
        s["dy"] = (_randn(g, case["M"], case["N"]) * 1e-3).to(torch.bfloat16)
        w = _weight(g, case["N"], case["K"])
        codes, scales = _pack(_pad32(w)[None])
        s["w"] = (codes[0], scales[0])
        codes, scales = _pack(_pad32(w.t())[None])  # blocks along the layer's outputs, for the input gradient
        s["wt"] = (codes[0], scales[0])
    elif op == "experts":
        T, E, K, N = case["T"], case["E"], case["K"], case["N"]
        s["x"] = _activation(g, T, K, torch.bfloat16)
        chosen = _sizes(case, seed).flatten().long()
        order = torch.sort(chosen, stable=True).indices
        s["tokens"] = (order // case["k"]).to(torch.int32)
        s["expert_of"] = chosen[order]
        counts = torch.bincount(chosen, minlength=E)
        s["offsets"] = torch.nn.functional.pad(counts.cumsum(0), (1, 0))
        s["most"] = int(counts.max())
        s["w"] = _pack(_pad32(_weight(g, E * N, K)).view(E, N, -1))
    elif op == "route":
        s["logits"] = (_randn(g, case["T"], case["E"]) * 1.5).to(_dtype(case["dtype"]))
        s["b"] = _randn(g, case["E"]) * 0.05 if case["bias"] else None
        s["dw"] = _randn(g, case["T"], case["k"])
    else:
        T, k, H = case["T"], case["k"], case["H"]
        s["indices"] = _sizes(case, seed)
        s["y"] = _randn(g, T * k, H).to(torch.bfloat16)
        s["weights"] = torch.softmax(_randn(g, T, k), 1)
        s["dout"] = (_randn(g, T, H) * 1e-2).to(torch.bfloat16)
    return s


# ---- plain forms -----------------------------------------------------------------------------------

def _pow2(e):
    """2**e in fp32 for integers -127 <= e <= 127, from the bits (e = -127 is subnormal)."""
    bits = torch.where(e > -127, (e + 127) << 23, torch.full_like(e, 1 << 22))
    return bits.to(torch.int32).view(torch.float32)


def _blocks(x):
    """x [..., C] fp32 (C % 32 == 0): its E2M1 values [..., C/32, 32] before scaling, and exponents [..., C/32]."""
    b = x.unflatten(-1, (-1, 32))
    amax = b.abs().amax(-1)
    m, ex = torch.frexp(amax)
    e = (ex.to(torch.int32) - 3 + (m > 0.75).to(torch.int32)).clamp(-127, 127)
    e = torch.where(amax == 0, torch.zeros_like(e), e)
    v = b * _pow2(-e)[..., None]
    a = v.abs()
    q = torch.where(a < 2, torch.round(2 * a) / 2, torch.where(a < 4, torch.round(a), 2 * torch.round(a / 2)))
    return torch.copysign(q.clamp(max=6.0), v), e


def _values(x):
    """What the 4-bit cast of x [..., C] stands for, in fp32."""
    C = x.shape[-1]
    q, e = _blocks(_pad32(x.float()))
    return (q * _pow2(e)[..., None]).flatten(-2)[..., :C]


def _unpack(codes, plane, R, C):
    """The fp32 values [..., R, C] of a 4-bit matrix held as codes and scale plane."""
    levels = torch.tensor([0, .5, 1, 1.5, 2, 3, 4, 6, -0., -.5, -1, -1.5, -2, -3, -4, -6], device=codes.device)
    q = levels[torch.stack((codes & 15, codes >> 4), -1).flatten(-2).int()]
    nb = q.shape[-1] // 32
    lead = plane.shape[:-1]
    byte = plane.view(-1, -(-R // 128), -(-nb // 4), 32, 4, 4).permute(0, 1, 4, 3, 2, 5)
    byte = byte.reshape(*lead, -(-R // 128) * 128, -(-nb // 4) * 4)[..., :R, :nb]
    return (q.unflatten(-1, (nb, 32)) * _pow2(byte.int() - 127)[..., None]).flatten(-2)[..., :C]


def _key(s, logits):
    """Scores (fp32), and the keys that experts are chosen by."""
    l = logits.float()
    if s["score"] == "softmax":
        e = torch.exp(l - l.amax(1, keepdim=True))
        e2 = torch.nn.functional.pad(e, (0, 512 - s["E"]))
        e2 = e2[:, :256] + e2[:, 256:]  # the sum is formed by halves, so that it has one value
        e2 = e2[:, :128] + e2[:, 128:]
        e2 = e2[:, :64] + e2[:, 64:]
        e2 = e2[:, :32] + e2[:, 32:]
        e2 = e2[:, :16] + e2[:, 16:]
        e2 = e2[:, :8] + e2[:, 8:]
        e2 = e2[:, :4] + e2[:, 4:]
        e2 = e2[:, :2] + e2[:, 2:]
        score = e / (e2[:, :1] + e2[:, 1:])
    else:
        score = 1.0 / (1.0 + torch.exp(-l))
    return score, (l if s["b"] is None else score + s["b"])


def _choose(s, key):
    """Indices [T, k] of the largest keys among the chosen groups' experts, ties to the lowest index."""
    G = s["groups"]
    if s["topk_groups"] < G:
        by_group = key.unflatten(1, (G, -1))
        if s["b"] is None:
            rank = by_group.amax(2)
        else:
            rank = by_group.sort(dim=2, descending=True).values[:, :, :2].sum(2)
        first = rank.sort(dim=1, descending=True, stable=True).indices[:, :s["topk_groups"]]
        keep = torch.zeros_like(rank).scatter(1, first, 1.0) > 0
        key = torch.where(keep[:, :, None], by_group, float("-inf")).flatten(1)
    return key.sort(dim=1, descending=True, stable=True).indices[:, :s["k"]]


def _route(s):
    score, key = _key(s, s["logits"])
    idx = _choose(s, key)
    p = score.gather(1, idx)
    total = p.sum(1, keepdim=True)
    w = 2.5 * (p / total if s["renorm"] else p)
    out = {"indices": idx.to(torch.int32), "weights": w}
    if s["grad"]:
        d = 2.5 * s["dw"]
        if s["renorm"]:
            d = (d - (d * p).sum(1, keepdim=True) / total) / total
        if s["score"] == "sigmoid":
            dl = torch.zeros_like(score).scatter(1, idx, d * p * (1 - p))
        else:
            ds = torch.zeros_like(score).scatter(1, idx, d)
            dl = score * (ds - (d * p).sum(1, keepdim=True))
        out["dlogits"] = dl.to(s["logits"].dtype)
    return out


def _combine(s):
    T, k = s["indices"].shape
    flat = s["indices"].flatten().long()
    order = torch.sort(flat, stable=True).indices
    slots = torch.empty_like(order).scatter(0, order, torch.arange(T * k, device=order.device)).view(T, k)
    counts = (flat[:, None] == torch.arange(s["E"], device=flat.device)).sum(0)
    rows = s["y"].float()[slots]
    out = {"offsets": torch.nn.functional.pad(counts.cumsum(0), (1, 0)), "slots": slots.to(torch.int32),
           "tokens": (order // k).to(torch.int32),
           "out": (rows * s["weights"][:, :, None]).sum(1).to(torch.bfloat16)}
    if s["grad"]:
        d = s["dout"].float()
        out["dweights"] = (rows * d[:, None]).sum(2)
        out["dy"] = (d[order // k] * s["weights"].flatten()[order][:, None]).to(torch.bfloat16)
    return out


def _experts(s):
    E, N = s["E"], s["N"]
    x = _values(s["x"])
    at = s["offsets"][:-1, None] + torch.arange(s["most"], device=x.device)
    live = at < s["offsets"][1:, None]
    padded = x[s["tokens"][at.clamp(max=s["tokens"].numel() - 1)]] * live[:, :, None]
    y = torch.bmm(padded, _unpack(*s["w"], N, s["K"]).transpose(1, 2))
    row = torch.arange(s["tokens"].numel(), device=x.device)
    return y[s["expert_of"], row - s["offsets"][s["expert_of"]]].to(torch.bfloat16)


def _run_plain(s):
    op = s["op"]
    if op == "cast":
        out = {"rows": _values(s["x"]).to(torch.bfloat16)}
        if s["cols"]:
            out["cols"] = _values(s["x"].t()).to(torch.bfloat16)
        return out
    if op == "linear":
        return (_values(s["x"]) @ _unpack(*s["w"], s["N"], s["K"]).t()).to(_dtype(s["out"]))
    if op == "train":
        y = _values(s["x"]) @ _unpack(*s["w"], s["N"], s["K"]).t()
        dx = _values(s["dy"]) @ _unpack(*s["wt"], s["K"], s["N"]).t()
        dw = _values(s["dy"].t()) @ _values(s["x"].t()).t()
        return {"y": y.to(torch.bfloat16), "dx": dx.to(torch.bfloat16), "dw": dw}
    if op == "experts":
        return _experts(s)
    return _route(s) if op == "route" else _combine(s)


# ---- the package's calls ---------------------------------------------------------------------------

def _run_own(s):
    import mxfp8_block_scaled_04_gb300 as mx

    op = s["op"]
    if op == "cast":
        q = mx.quantize_mxfp4(s["x"], colwise=s["cols"])
        out = {"rows": mx.dequantize_mxfp4(q.row)}
        if s["cols"]:
            out["cols"] = mx.dequantize_mxfp4(q.col)
        return out
    if op == "linear":
        q = mx.quantize_mxfp4(s["x"])
        return mx.matmul_mxfp4(q.row, mx.MXFP4Matrix(*s["w"], s["N"], s["K"]), out_dtype=_dtype(s["out"]))
    if op == "train":
        x = mx.quantize_mxfp4(s["x"], colwise=True)
        dy = mx.quantize_mxfp4(s["dy"], colwise=True)
        return {"y": mx.matmul_mxfp4(x.row, mx.MXFP4Matrix(*s["w"], s["N"], s["K"])),
                "dx": mx.matmul_mxfp4(dy.row, mx.MXFP4Matrix(*s["wt"], s["K"], s["N"])),
                "dw": mx.matmul_mxfp4(dy.col, x.col, out_dtype=torch.float32)}
    if op == "experts":
        q = mx.quantize_mxfp4_grouped(s["x"], s["offsets"], rows=s["tokens"])
        return mx.matmul_mxfp4_grouped(q, s["offsets"], mx.MXFP4Matrix(*s["w"], s["N"], s["K"]))
    if op == "route":
        how = dict(score=s["score"], bias=s["b"], groups=s["groups"], topk_groups=s["topk_groups"],
                   renormalize=s["renorm"], scale=2.5)
        r = mx.moe_route(s["logits"], s["k"], **how)
        out = {"indices": r.indices, "weights": r.weights}
        if s["grad"]:
            how = dict(score=s["score"], renormalize=s["renorm"], scale=2.5)
            out["dlogits"] = mx.moe_route_backward(s["logits"], r.indices, s["dw"], **how)
        return out
    plan = mx.moe_plan(s["indices"], s["E"])
    out = {"offsets": plan.offsets, "slots": plan.slots, "tokens": plan.tokens,
           "out": mx.moe_combine(s["y"], plan.slots, s["weights"])}
    if s["grad"]:
        out["dy"], out["dweights"] = mx.moe_combine_backward(s["dout"], s["y"], plan.slots, s["weights"])
    return out


def run(state):
    return _run_own(state) if own else _run_plain(state)


# ---- what a pass cannot do without -----------------------------------------------------------------

def _fp4(r, c):
    """Bytes of a 4-bit matrix [r, c] with its scales."""
    return r * c * 17 / 32


def work(case):
    op = case["op"]
    if op == "cast":  # x in; codes and scales out and in again; the values out
        n = case["M"] * case["N"]
        ways = 2 if case["cols"] else 1
        size = 2 if case["dtype"] == "bf16" else 4
        return {"bytes": n * size + ways * (2 * _fp4(1, n) + 2 * n), "flops": 2 * ways * n}
    if op == "linear":
        M, K, N = case["M"], case["K"], case["N"]
        return {"bytes": 2 * M * K + _fp4(N, K) + M * N * (2 if case["out"] == "bf16" else 4), "flops": 2 * M * K * N}
    if op == "train":
        M, K, N = case["M"], case["K"], case["N"]
        return {"bytes": 2 * M * (K + N) + 2 * _fp4(N, K) + 2 * M * (N + K) + 4 * N * K, "flops": 6 * M * K * N}
    if op == "experts":
        R, K, N, E = case["T"] * case["k"], case["K"], case["N"], case["E"]
        used = E * (1 - (1 - case["k"] / E) ** case["T"])  # experts that a row reaches, at equal load
        return {"bytes": 2 * case["T"] * K + 4 * R + used * _fp4(N, K) + 2 * R * N, "flops": 2 * R * K * N}
    if op == "route":
        n = case["T"] * case["E"]
        size = 2 if case["dtype"] == "bf16" else 4
        picks = case["T"] * case["k"]
        return {"bytes": n * size * (2 if case["grad"] else 1) + picks * (12 if case["grad"] else 8), "flops": 8 * n}
    T, k, H = case["T"], case["k"], case["H"]
    grad = 2 * T * H + 2 * T * k * H + 4 * T * k if case["grad"] else 0
    return {"bytes": 2 * T * k * H + 2 * T * H + 16 * T * k + grad, "flops": (5 if case["grad"] else 2) * T * k * H}


# ---- the definitions in 64 bits --------------------------------------------------------------------

def _two64(e):
    return ((e.long() + 1023) << 52).view(torch.float64)


def _cast64(x):
    """The 4-bit cast's values from their definition: the nearest level, ties to the even code."""
    R, C = x.shape
    b = torch.nn.functional.pad(x.double(), (0, -C % 32)).view(R, -1, 32)
    top = b.abs().amax(2, keepdim=True)
    top = torch.where(top > 0, top, 6.0)
    e = torch.round(torch.log2(top / 6))
    e = e + (6 * _two64(e) < top).double() - (6 * _two64(e - 1) >= top).double()  # the least e with 6 * 2**e >= top
    e = e.clamp(-127, 127)
    a = b.abs() * _two64(-e)
    value = torch.zeros_like(a)
    for level, below, tie_up in ((.5, .25, False), (1, .75, True), (1.5, 1.25, False), (2, 1.75, True), (3, 2.5, False),
                                 (4, 3.5, True), (6, 5, False)):
        value = torch.where((a >= below) if tie_up else (a > below), float(level), value)
    return (torch.where(b < 0, -value, value) * _two64(e)).view(R, -1)[:, :C]


def _decode64(codes, plane, R, C):
    """A 4-bit matrix's values, read element by element from its layout."""
    r = torch.arange(R, device=codes.device)[:, None]
    c = torch.arange(C, device=codes.device)[None]
    tiles = -(-(codes.shape[1] // 16) // 4)
    code = (codes[r, c // 2].int() >> (4 * (c % 2))) & 15
    exp, man = (code >> 1) & 3, (code & 1).double()
    mag = torch.where(exp == 0, man / 2, (1 + man / 2) * _two64(exp - 1))
    blk = c // 32
    at = ((r // 128) * tiles + blk // 4) * 512 + 16 * (r % 32) + 4 * (r % 128 // 32) + blk % 4
    return torch.where(code >= 8, -mag, mag) * _two64(plane[at].long() - 127)


def _route64(s):
    l = s["logits"].double()
    score = torch.softmax(l, 1) if s["score"] == "softmax" else torch.sigmoid(l)
    key = l if s["b"] is None else score + s["b"].double()
    T, E = l.shape
    G = s["groups"]
    parts = key.view(T, G, E // G)
    if s["b"] is None:
        rank = parts.max(2).values
    else:
        rank = parts.topk(min(2, E // G), 2).values.sum(2)
    ahead = (rank[:, None, :] > rank[:, :, None]).sum(2)
    ahead += ((rank[:, None, :] == rank[:, :, None]) & torch.ones(G, G, device=l.device).tril(-1).bool()).sum(2)
    key = torch.where((ahead < s["topk_groups"])[:, :, None], parts, -math.inf).view(T, E)
    idx = key.sort(dim=1, descending=True, stable=True).indices[:, :s["k"]]
    leaf = l.requires_grad_()
    score = torch.softmax(leaf, 1) if s["score"] == "softmax" else torch.sigmoid(leaf)
    w = score.gather(1, idx)
    w = 2.5 * (w / w.sum(1, keepdim=True) if s["renorm"] else w)
    out = {"indices": None, "weights": w.detach()}
    if s["grad"]:
        out["dlogits"] = torch.autograd.grad(w, leaf, s["dw"].double())[0]
    return out


def exact(case, seed):
    s = prepare(case, seed)
    op = case["op"]
    if op == "cast":
        out = {"rows": _cast64(s["x"])}
        if s["cols"]:
            out["cols"] = _cast64(s["x"].t())
        return out
    if op == "linear":
        if 2 * case["M"] * case["N"] * case["K"] > 2e12:
            return None
        return _cast64(s["x"]) @ _decode64(*s["w"], s["N"], s["K"]).t()
    if op == "train":
        if 6 * case["M"] * case["N"] * case["K"] > 2e12:
            return None
        return {"y": _cast64(s["x"]) @ _decode64(*s["w"], s["N"], s["K"]).t(),
                "dx": _cast64(s["dy"]) @ _decode64(*s["wt"], s["K"], s["N"]).t(),
                "dw": _cast64(s["dy"].t()) @ _cast64(s["x"].t()).t()}
    if op == "experts":
        if 2 * case["T"] * case["k"] * case["N"] * case["K"] > 2e12:
            return None
        x = _cast64(s["x"])
        off = s["offsets"].tolist()
        y = torch.empty((off[-1], s["N"]), dtype=torch.float64, device="cuda")
        for g in range(s["E"]):
            if off[g + 1] > off[g]:
                w = _decode64(s["w"][0][g], s["w"][1][g], s["N"], s["K"])
                y[off[g]:off[g + 1]] = x[s["tokens"][off[g]:off[g + 1]].long()] @ w.t()
        return y
    if op == "route":
        return _route64(s)
    T, k = s["indices"].shape
    flat = s["indices"].flatten().long()
    slots = torch.argsort(torch.argsort(flat, stable=True)).view(T, k)
    y, w, d = s["y"].double(), s["weights"].double(), s["dout"].double()
    out = {"offsets": None, "slots": None, "tokens": None, "out": torch.einsum("tk,tkh->th", w, y[slots])}
    if s["grad"]:
        out["dweights"] = torch.einsum("th,tkh->tk", d, y[slots])
        dy = torch.zeros_like(y)
        dy[slots.flatten()] = (w[:, :, None] * d[:, None]).flatten(0, 1)
        out["dy"] = dy
    return out
