"""Cases of the expert block's operators: experts' products in MXFP8 with both gradients, bf16 tokens on 4-bit weights,
and the norms around a block fused with its gate and residual scale.

``run`` computes each operator in a plain form (elementary torch operations in fp32) or, with ``own`` set, through the
package's public calls.  Layouts shared by both: FP8 codes are uint8 [R, C]; rows are scaled in blocks of 32 along a
row, columns in blocks of 32 rows that start at each expert's first row.  Scales are E8M0 bytes in 128x4 tiles (entry
(r, c) of a tile at 16*(r % 32) + 4*(r % 128 // 32) + c), a plane per expert, one after the other: [rows_g, ceil(C/32)]
for the rows, [C, ceil(rows_g/32)] for the columns.  Experts' weights [E, N, K] are E groups of N rows.  A 4-bit matrix
[R, C] is uint8 codes [R, ceil(C/32)*16] (element 2i in the low half of byte i) and one such plane.
"""
import math

import torch

own = False


# ---- cases -----------------------------------------------------------------------------------------

def listed():
    return [
        # Sixteen tokens of a serving step, eight experts each, through 64 experts held in 8 bits.
        {"name": "experts8_64x128x7168x2048", "op": "experts8", "T": 16, "k": 8, "E": 64, "K": 7168, "N": 2048,
         "skew": 0.5, "grad": False, "fmt": "e4m3"},
        # A few hundred ragged rows over few experts, one of them without any: a small training step, gradients in E5M2.
        {"name": "experts8_train_8x777x2064x1040", "op": "experts8", "T": 259, "k": 3, "E": 8, "K": 2064, "N": 1040,
         "skew": 1.5, "grad": True, "fmt": "e5m2"},
        # A training step of a large expert layer: output, input gradient, fp32 weight gradient of 64 experts.
        {"name": "experts8_train_64x65536x7168x2048", "op": "experts8", "T": 8192, "k": 8, "E": 64, "K": 7168,
         "N": 2048, "skew": 0.3, "grad": True, "fmt": "e4m3"},
        # One token of a chat through an MLP's first layer whose weights are held in 4 bits.
        {"name": "linear4_1x8192x28672", "op": "linear4", "M": 1, "K": 8192, "N": 28672, "dtype": "bf16", "out": "bf16"},
        # A draft of seven tokens through a small square layer, fp32 out (logits of a head).
        {"name": "linear4_7x4096x4096", "op": "linear4", "M": 7, "K": 4096, "N": 4096, "dtype": "bf16", "out": "fp32"},
        # A batch of 61 chats, fp32 activations, a layer of odd width.
        {"name": "linear4_61x8200x8184", "op": "linear4", "M": 61, "K": 8200, "N": 8184, "dtype": "fp32", "out": "bf16"},
        # The serving step's tokens through 64 experts held in 4 bits, gathered by a plan.
        {"name": "experts4_64x128x7168x2048", "op": "experts4", "T": 16, "k": 8, "E": 64, "K": 7168, "N": 2048,
         "skew": 0.5, "dtype": "bf16"},
        # Two tokens through their few experts.
        {"name": "experts4_16x4x2048x1032", "op": "experts4", "T": 2, "k": 2, "E": 16, "K": 2048, "N": 1032,
         "skew": 0.0, "dtype": "bf16"},
        # The norms between two blocks in a serving step.
        {"name": "norm_16x7168", "op": "norm", "T": 16, "H": 7168, "y": "bf16", "h": "bf16", "post": True,
         "gate": "channel", "scale": 1.0, "grad": False},
        # The same of a training batch, the residual stream in fp32 and scaled.
        {"name": "norm_8192x7168_fp32", "op": "norm", "T": 8192, "H": 7168, "y": "bf16", "h": "fp32", "post": True,
         "gate": "channel", "scale": 0.9, "grad": False},
        # The gradients of a training batch, with those of both weights and of the gate.
        {"name": "norm_grad_8192x7168", "op": "norm", "T": 8192, "H": 7168, "y": "bf16", "h": "bf16", "post": True,
         "gate": "channel", "scale": 1.0, "grad": True},
        # The gradients of an odd number of tokens with a gate for each token and no norm behind the block.
        {"name": "norm_grad_1021x5000", "op": "norm", "T": 1021, "H": 5000, "y": "bf16", "h": "fp32", "post": False,
         "gate": "token", "scale": 0.5, "grad": True},
    ]


def _log(rng, lo, hi, step=1):
    v = int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))
    return max(step, v // step * step)


def draw(rng):
    op = rng.choice(["experts8", "linear4", "experts4", "norm"])
    if op == "experts8":
        E = rng.choice([1, 4, 8, 16, 64])
        return {"op": op, "T": _log(rng, 1, 8192), "k": rng.randint(1, min(E, 8)), "E": E, "K": _log(rng, 256, 7168, 16),
                "N": _log(rng, 128, 2048, 16), "skew": rng.choice([0.0, 0.3, 1.5]), "grad": rng.random() < 0.6,
                "fmt": rng.choice(["e4m3", "e5m2"])}
    if op == "linear4":
        return {"op": op, "M": _log(rng, 1, 64), "K": _log(rng, 256, 8192, 8), "N": _log(rng, 128, 28672, 8),
                "dtype": rng.choice(["bf16", "bf16", "fp32"]), "out": rng.choice(["bf16", "fp32"])}
    if op == "experts4":
        E = rng.choice([4, 8, 16, 64])
        return {"op": op, "T": _log(rng, 1, 64), "k": rng.randint(1, min(E, 8)), "E": E, "K": _log(rng, 512, 7168, 8),
                "N": _log(rng, 256, 2048, 8), "skew": rng.choice([0.0, 0.5]), "dtype": rng.choice(["bf16", "bf16", "fp32"])}
    while True:
        c = {"op": op, "T": _log(rng, 1, 16384), "H": _log(rng, 64, 16384, 8), "y": rng.choice(["bf16", "bf16", "fp32"]),
             "h": rng.choice(["bf16", "fp32"]), "post": rng.random() < 0.7, "gate": rng.choice(["none", "channel", "token"]),
             "scale": rng.choice([1.0, 0.7]), "grad": rng.random() < 0.6}
        if c["T"] * c["H"] <= 8192 * 7168:
            return c


# ---- inputs ----------------------------------------------------------------------------------------

def _gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(int(seed) * 1000003 + 29)
    return g


def _randn(g, *shape):
    return torch.randn(shape, generator=g, device="cuda", dtype=torch.float32)


def _rand(g, *shape):
    return torch.rand(shape, generator=g, device="cuda", dtype=torch.float32)


def _dtype(name):
    return {"bf16": torch.bfloat16, "fp32": torch.float32}[name]


def _fp8(name):
    return {"e4m3": torch.float8_e4m3fn, "e5m2": torch.float8_e5m2}[name]


def _activation(g, M, N):
    """Normal values under a spread of row scales, one in a thousand an outlier, one row in fifty zero."""
    x = _randn(g, M, N)
    x *= torch.exp(_randn(g, M, 1))
    x *= torch.where(_rand(g, M, N) < 1e-3, 40.0, 1.0)
    if M > 1:
        x *= (_rand(g, M, 1) >= 0.02).float()
    return x


def _pow2(e):
    """2**e in fp32 for integers -127 <= e <= 127, from the bits (e = -127 is subnormal)."""
    bits = torch.where(e > -127, (e + 127) << 23, torch.full_like(e, 1 << 22))
    return bits.to(torch.int32).view(torch.float32)


def _row_places(offsets, group, C):
    """Place of every row's every block in the planes of the rows [R, ceil(C/32)], and the planes' size."""
    rows = offsets[1:] - offsets[:-1]
    tiles = torch.nn.functional.pad(((rows + 127) // 128).cumsum(0), (1, 0))
    nb = -(-C // 32)
    kc = -(-nb // 4)
    r = torch.arange(group.numel(), device=group.device) - offsets[group]
    at = (tiles[group] + r // 128) * kc * 512 + 16 * (r % 32) + 4 * (r % 128 // 32)
    b = torch.arange(nb, device=group.device)
    return at[:, None] + (b // 4 * 512 + b % 4)[None], tiles[-1] * kc * 512


def _col_places(offsets, C):
    """Place of every 32-row block's every column in the planes of the columns [S, C], their size, each group's blocks."""
    rows = offsets[1:] - offsets[:-1]
    blocks, kt = (rows + 31) // 32, (rows + 127) // 128
    ct = -(-C // 128)
    first = torch.nn.functional.pad(blocks.cumsum(0), (1, 0))
    base = torch.nn.functional.pad((kt * ct * 512).cumsum(0), (1, 0))
    g = torch.repeat_interleave(torch.arange(rows.numel(), device=rows.device), blocks)
    i = torch.arange(g.numel(), device=rows.device) - first[g]
    j = torch.arange(C, device=rows.device)
    at = (base[g] + i // 4 * 512 + i % 4)[:, None] + (kt[g] * 512)[:, None] * (j // 128)[None]
    return at + (16 * (j % 32) + 4 * (j % 128 // 32))[None], base[-1], first


def _groups(offsets, R):
    return torch.repeat_interleave(torch.arange(offsets.numel() - 1, device=offsets.device), offsets[1:] - offsets[:-1],
                                   output_size=R)


def _exponent(amax, fmax):
    """Least e with fmax * 2**e >= amax, within E8M0's range (0 for an empty block)."""
    m, ex = torch.frexp(amax / fmax)  # fmax has few bits: the quotient rounds, but never across a power of two here
    e = (ex - (m == 0.5).to(ex.dtype)).clamp(-127, 127)
    return torch.where(amax == 0, torch.zeros_like(e), e).to(torch.int32)


def _cast8(x, offsets, fmt):
    """x [R, C] fp32 in 8 bits both ways, as a user's casts leave it: (row codes, row planes, column codes, column planes)."""
    R, C = x.shape
    t = _fp8(fmt)
    fmax = 448.0 if fmt == "e4m3" else 57344.0
    group = _groups(offsets, R)
    b = torch.nn.functional.pad(x, (0, -C % 32)).view(R, -1, 32)
    e = _exponent(b.abs().amax(2), fmax)
    row = (b * _pow2(-e)[:, :, None]).clamp(-fmax, fmax).flatten(1)[:, :C].to(t).view(torch.uint8).contiguous()
    at, size = _row_places(offsets, group, C)
    row_plane = torch.zeros(int(size), dtype=torch.uint8, device=x.device)
    row_plane[at] = (e + 127).to(torch.uint8)
    at, size, first = _col_places(offsets, C)
    S = at.shape[0]
    place = first[group] * 32 + torch.arange(R, device=x.device) - offsets[group]  # each row's place with whole blocks
    padded = torch.zeros((S * 32, C), device=x.device)
    padded[place] = x
    e = _exponent(padded.view(S, 32, C).abs().amax(1), fmax)
    col = (x * _pow2(-e)[place // 32]).clamp(-fmax, fmax).to(t).view(torch.uint8).contiguous()
    col_plane = torch.zeros(int(size), dtype=torch.uint8, device=x.device)
    col_plane[at] = (e + 127).to(torch.uint8)
    return row, row_plane, col, col_plane


def _pack4(w):
    """A layer's weights as a user keeps them: codes and GEMM-ready scale planes of w [B, R, C] (C % 32 == 0)."""
    B, R, C = w.shape
    b = w.float().view(B, R, -1, 32)
    e = _exponent(b.abs().amax(3), 6.0)
    v = b * _pow2(-e)[..., None]
    a = v.abs()
    a = torch.where(a < 2, torch.round(2 * a) / 2, torch.where(a < 4, torch.round(a), 2 * torch.round(a / 2))).clamp(max=6.0)
    code = (2.0 * a.clamp(max=2.0) + (a - 2.0).clamp(0.0, 2.0) + 0.5 * (a - 4.0).clamp(min=0.0)).to(torch.uint8)
    code = (code + 8 * (v < 0).to(torch.uint8)).view(B, R, -1)
    codes = code[..., 0::2] + 16 * code[..., 1::2]
    byte = torch.nn.functional.pad((e + 127).to(torch.uint8), (0, -(C // 32) % 4, 0, -R % 128))
    tiles = byte.view(B, byte.shape[1] // 128, 4, 32, byte.shape[2] // 4, 4)
    return codes.contiguous(), tiles.permute(0, 1, 4, 3, 2, 5).reshape(B, -1).contiguous()


def _weight4(g, B, R, C):
    return _pack4(torch.nn.functional.pad((_randn(g, B, R, C) * 0.02).to(torch.bfloat16), (0, -C % 32)))


def _choices(case, seed):
    """Rows of a batch sorted by expert, the experts loaded unequally: (tokens [R], experts [R], offsets [E + 1])."""
    g = _gen(seed + 7)
    E, T, k = case["E"], case["T"], case["k"]
    popularity = _randn(g, 1, E) * case["skew"]
    noise = -torch.log(-torch.log(_rand(g, T, E).clamp(1e-7, 1 - 1e-7)))
    if case["skew"] > 1 and k < E:
        noise[:, E // 2] = -100.0  # an expert that no token chooses
    chosen = (popularity + noise).topk(k, dim=1).indices.flatten()
    order = torch.sort(chosen, stable=True).indices
    offsets = torch.nn.functional.pad(torch.bincount(chosen, minlength=E).cumsum(0), (1, 0))
    return (order // k).to(torch.int32), chosen[order], offsets


def prepare(case, seed):
    g = _gen(seed)
    op = case["op"]
    s = dict(case)
    if op == "experts8":
        E, K, N = case["E"], case["K"], case["N"]
        tokens, s["expert_of"], s["offsets"] = _choices(case, seed)
        s["most"] = int((s["offsets"][1:] - s["offsets"][:-1]).max())
        s["x"] = _cast8(_activation(g, case["T"], K)[tokens.long()], s["offsets"], "e4m3")
        s["w_offsets"] = torch.arange(E + 1, device="cuda") * N
        s["w"] = _cast8(_randn(g, E * N, K) * 0.02, s["w_offsets"], "e4m3")
        if case["grad"]:
            dy = _randn(g, tokens.numel(), N) * torch.exp(_randn(g, tokens.numel(), 1)) * 1e-3
            s["dy"] = _cast8(dy, s["offsets"], case["fmt"])
    elif op == "linear4":
        s["x"] = _activation(g, case["M"], case["K"]).to(_dtype(case["dtype"]))
        codes, plane = _weight4(g, 1, case["N"], case["K"])
        s["w"] = (codes[0], plane[0])
    elif op == "experts4":
        s["x"] = _activation(g, case["T"], case["K"]).to(_dtype(case["dtype"]))
        s["tokens"], s["expert_of"], s["offsets"] = _choices(case, seed)
        s["most"] = int((s["offsets"][1:] - s["offsets"][:-1]).max())
        s["w"] = _weight4(g, case["E"], case["N"], case["K"])
    else:
        T, H = case["T"], case["H"]
        wide = torch.where(_rand(g, 1, H) < 2e-3, 30.0, 1.0)  # channels that carry much larger values, as trained models have
        s["block"] = (_randn(g, T, H) * torch.exp(0.5 * _randn(g, T, 1))).to(_dtype(case["y"]))
        s["stream"] = (_randn(g, T, H) * wide * torch.exp(0.3 * _randn(g, T, 1))).to(_dtype(case["h"]))
        s["w_pre"] = 1.0 + 0.2 * _randn(g, H)
        s["w_post"] = 0.5 + 0.1 * _randn(g, H) if case["post"] else None
        s["g"] = {"none": lambda: None, "channel": lambda: 0.3 + 0.1 * _randn(g, H),
                  "token": lambda: torch.sigmoid(_randn(g, T, 1))}[case["gate"]]()
        if case["grad"]:  # stream is then the one behind the block, as the forward pass left it
            s["d_h"] = (_randn(g, T, H) * 1e-3).to(_dtype(case["h"]))
            s["d_x"] = (_randn(g, T, H) * 1e-3).to(torch.bfloat16)
    return s


# ---- plain forms -----------------------------------------------------------------------------------

EPS = 1e-6


def _rows8(m, fmt, offsets):
    """The fp32 values of a matrix in 8 bits, from its rows' codes and scales."""
    codes, plane = m[0], m[1]
    R, C = codes.shape
    at, _ = _row_places(offsets, _groups(offsets, R), C)
    scale = _pow2(plane[at].int() - 127)
    v = torch.nn.functional.pad(codes.view(_fp8(fmt)).float(), (0, -C % 32)).view(R, -1, 32) * scale[:, :, None]
    return v.flatten(1)[:, :C]


def _cols8(m, fmt, offsets):
    """The fp32 values of a matrix in 8 bits, from its columns' codes and scales."""
    codes, plane = m[2], m[3]
    R, C = codes.shape
    group = _groups(offsets, R)
    at, _, first = _col_places(offsets, C)
    scale = _pow2(plane[at].int() - 127)
    block = first[group] + (torch.arange(R, device=codes.device) - offsets[group]) // 32
    return codes.view(_fp8(fmt)).float() * scale[block]


def _padded(s, v):
    """Rows by expert [E, most, C], zeros where an expert has fewer, and each row's place in its expert."""
    at = s["offsets"][:-1, None] + torch.arange(s["most"], device=v.device)
    live = at < s["offsets"][1:, None]
    place = torch.arange(v.shape[0], device=v.device) - s["offsets"][s["expert_of"]]
    return v[at.clamp(max=v.shape[0] - 1)] * live[:, :, None], place


def _experts8(s):
    E, N, K = s["E"], s["N"], s["K"]
    x, place = _padded(s, _rows8(s["x"], "e4m3", s["offsets"]))
    w = _rows8(s["w"], "e4m3", s["w_offsets"]).view(E, N, K)
    out = {"y": torch.bmm(x, w.transpose(1, 2))[s["expert_of"], place].to(torch.bfloat16)}
    if s["grad"]:
        dy, _ = _padded(s, _rows8(s["dy"], s["fmt"], s["offsets"]))
        w = _cols8(s["w"], "e4m3", s["w_offsets"]).view(E, N, K)
        out["dx"] = torch.bmm(dy, w)[s["expert_of"], place].to(torch.bfloat16)
        dy, _ = _padded(s, _cols8(s["dy"], s["fmt"], s["offsets"]))
        x, _ = _padded(s, _cols8(s["x"], "e4m3", s["offsets"]))
        out["dw"] = torch.bmm(dy.transpose(1, 2), x)
    return out


def _unpack4(codes, plane, R, C):
    """The fp32 values [..., R, C] of a 4-bit matrix held as codes and scale plane."""
    levels = torch.tensor([0, .5, 1, 1.5, 2, 3, 4, 6, -0., -.5, -1, -1.5, -2, -3, -4, -6], device=codes.device)
    q = levels[torch.stack((codes & 15, codes >> 4), -1).flatten(-2).int()]
    nb = q.shape[-1] // 32
    lead = plane.shape[:-1]
    byte = plane.view(-1, -(-R // 128), -(-nb // 4), 32, 4, 4).permute(0, 1, 4, 3, 2, 5)
    byte = byte.reshape(*lead, -(-R // 128) * 128, -(-nb // 4) * 4)[..., :R, :nb]
    return (q.unflatten(-1, (nb, 32)) * _pow2(byte.int() - 127)[..., None]).flatten(-2)[..., :C]


def _experts4(s):
    x, place = _padded(s, s["x"].float()[s["tokens"].long()])
    y = torch.bmm(x, _unpack4(*s["w"], s["N"], s["K"]).transpose(1, 2))
    return y[s["expert_of"], place].to(torch.bfloat16)


def _norm(s):
    y, h = s["block"].float(), s["stream"].float()
    gate = 1.0 if s["g"] is None else s["g"]
    if not s["grad"]:
        u = y
        if s["post"]:
            u = y * torch.rsqrt((y * y).mean(1, keepdim=True) + EPS) * s["w_post"]
        h = (s["scale"] * h + gate * u).to(_dtype(s["h"]))  # the stream as it is kept; the next norm reads it
        v = h.float()
        x = v * torch.rsqrt((v * v).mean(1, keepdim=True) + EPS) * s["w_pre"]
        return {"h": h, "x": x.to(torch.bfloat16)}
    r = torch.rsqrt((h * h).mean(1, keepdim=True) + EPS)
    d, n = s["d_x"].float(), h * r
    t = d * s["w_pre"]
    total = s["d_h"].float() + r * (t - n * (t * n).mean(1, keepdim=True))
    out = {"h": (s["scale"] * total).to(_dtype(s["h"])), "w_pre": (d * n).sum(0)}
    u, du = y, gate * total
    if s["post"]:
        r = torch.rsqrt((y * y).mean(1, keepdim=True) + EPS)
        n = y * r
        u = n * s["w_post"]
        out["w_post"] = (du * n).sum(0)
        t = du * s["w_post"]
        out["y"] = (r * (t - n * (t * n).mean(1, keepdim=True))).to(_dtype(s["y"]))
    else:
        out["y"] = du.to(_dtype(s["y"]))
    if s["g"] is not None:
        out["gate"] = (total * u).sum(0) if s["gate"] == "channel" else (total * u).sum(1, keepdim=True)
    return out


def _run_plain(s):
    op = s["op"]
    if op == "experts8":
        return _experts8(s)
    if op == "linear4":
        return (s["x"].float() @ _unpack4(*s["w"], s["N"], s["K"]).t()).to(_dtype(s["out"]))
    return _experts4(s) if op == "experts4" else _norm(s)


# ---- the package's calls ---------------------------------------------------------------------------

def _run_own(s):
    import mxfp8_block_scaled_04_gb300 as mx

    op = s["op"]
    if op == "experts8":
        x, w = mx.MXFP8Tensor(*s["x"], None), mx.MXFP8Tensor(*s["w"], None)
        out = {"y": mx.matmul_mxfp8_grouped(x, s["offsets"], w)}
        if s["grad"]:
            dy = mx.MXFP8Tensor(*s["dy"], None)
            out["dx"] = mx.matmul_mxfp8_grouped_dgrad(dy, s["offsets"], w, grad_fmt=s["fmt"])
            out["dw"] = mx.matmul_mxfp8_grouped_wgrad(dy, x, s["offsets"], grad_fmt=s["fmt"])
        return out
    if op == "linear4":
        return mx.linear_mxfp4(s["x"], mx.MXFP4Matrix(*s["w"], s["N"], s["K"]), out_dtype=_dtype(s["out"]))
    if op == "experts4":
        return mx.linear_mxfp4_grouped(s["x"], s["offsets"], mx.MXFP4Matrix(*s["w"], s["N"], s["K"]), rows=s["tokens"])
    how = dict(post_weight=s["w_post"], gate=s["g"], scale=s["scale"], eps=EPS)
    if not s["grad"]:
        r = mx.block_norm(s["block"], s["stream"], s["w_pre"], **how)
        return {"h": r.h, "x": r.x}
    d = mx.block_norm_backward(s["d_h"], s["d_x"], s["block"], s["stream"], s["w_pre"], **how)
    out = {"h": d.h, "w_pre": d.pre_weight}
    if s["post"]:
        out["w_post"] = d.post_weight
    out["y"] = d.y
    if s["g"] is not None:
        out["gate"] = d.gate
    return out


def run(state):
    return _run_own(state) if own else _run_plain(state)


# ---- what a pass cannot do without -----------------------------------------------------------------

def work(case):
    op = case["op"]
    if op == "norm":
        T, H = case["T"], case["H"]
        y, h = (2 if case[n] == "bf16" else 4 for n in "yh")
        if case["grad"]:  # y (only for a norm or a gate), the stream, both gradients in; two gradients out
            used = y if case["post"] or case["gate"] != "none" else 0
            return {"bytes": T * H * (used + h + h + 2 + h + y), "flops": (28 if case["post"] else 18) * T * H}
        return {"bytes": T * H * (y + h + h + 2), "flops": (10 if case["post"] else 7) * T * H}
    K, N = case["K"], case["N"]
    if op == "linear4":
        M = case["M"]
        return {"bytes": M * K * (2 if case["dtype"] == "bf16" else 4) + N * K * 17 / 32 + M * N * (2 if case["out"] == "bf16" else 4),
                "flops": 2 * M * K * N}
    R, E = case["T"] * case["k"], case["E"]
    used = E * (1 - (1 - case["k"] / E) ** case["T"])  # experts that a row reaches, at equal load
    if op == "experts4":
        return {"bytes": case["T"] * K * (2 if case["dtype"] == "bf16" else 4) + 4 * R + used * N * K * 17 / 32 + 2 * R * N, "flops": 2 * R * K * N}
    forward = R * K * 33 / 32 + used * N * K * 33 / 32 + 2 * R * N
    if not case["grad"]:
        return {"bytes": forward, "flops": 2 * R * K * N}
    return {"bytes": forward + R * N * 33 / 32 + used * N * K * 33 / 32 + 2 * R * K + R * (N + K) * 33 / 32 + 4 * E * N * K,
            "flops": 6 * R * K * N}


# ---- the definitions in 64 bits --------------------------------------------------------------------

def _two64(e):
    return ((e.long() + 1023) << 52).view(torch.float64)


def _tile64(plane, rows, blocks):
    """Scales [rows, blocks] of one plane, tile by tile."""
    kc = -(-blocks // 4)
    t = plane.view(-(-rows // 128), kc, 32, 4, 4)
    return _two64(t.transpose(2, 3).transpose(1, 2).transpose(2, 3).reshape(-1, kc * 4).long() - 127)[:rows, :blocks]


def _value64(codes, fmt):
    """FP8 codes by their fields: sign, exponent, mantissa."""
    c = codes.long()
    mbits, bias = (3, 7) if fmt == "e4m3" else (2, 15)
    e, m = (c & 127) >> mbits, (c & ((1 << mbits) - 1)).double() / (1 << mbits)
    mag = torch.where(e == 0, m * 2.0 ** (1 - bias), (1 + m) * _two64(e - bias))
    return torch.where(c >= 128, -mag, mag)


def _each64(m, fmt, offsets, by_rows):
    """One expert's rows after the other, in 64 bits."""
    codes, plane = (m[0], m[1]) if by_rows else (m[2], m[3])
    C, at = codes.shape[1], 0
    for a, b in zip(offsets[:-1], offsets[1:]):
        n = b - a
        shape = (n, -(-C // 32)) if by_rows else (C, -(-n // 32))
        size = -(-shape[0] // 128) * -(-shape[1] // 4) * 512
        if n == 0:
            yield torch.zeros((0, C), dtype=torch.float64, device=codes.device)
            continue
        scale = _tile64(plane[at:at + size], *shape)
        at += size
        scale = scale.repeat_interleave(32, 1)[:, :C] if by_rows else scale.t().repeat_interleave(32, 0)[:n]
        yield _value64(codes[a:b], fmt) * scale


def _decode64(codes, plane, R, C):
    """A 4-bit matrix's values, read element by element from its layout."""
    c = torch.arange(C, device=codes.device)
    code = (codes.long()[:, c // 2] >> (4 * (c % 2))) & 15
    exp, man = (code >> 1) & 3, (code & 1).double()
    mag = torch.where(exp == 0, man / 2, (1 + man / 2) * _two64(exp - 1))
    scale = _tile64(plane, R, codes.shape[1] // 16)
    return torch.where(code >= 8, -mag, mag) * scale.repeat_interleave(32, 1)[:, :C]


def exact(case, seed):
    op = case["op"]
    if op in ("experts8", "experts4"):
        if (6 if case.get("grad") else 2) * case["T"] * case["k"] * case["N"] * case["K"] > 2e12:
            return None
    s = prepare(case, seed)
    if op == "experts8":
        off, woff = s["offsets"].tolist(), s["w_offsets"].tolist()
        out = {"y": torch.cat([x @ w.t() for x, w in zip(_each64(s["x"], "e4m3", off, True), _each64(s["w"], "e4m3", woff, True))])}
        if s["grad"]:
            out["dx"] = torch.cat([d @ w for d, w in zip(_each64(s["dy"], s["fmt"], off, True), _each64(s["w"], "e4m3", woff, False))])
            out["dw"] = torch.stack([d.t() @ x for d, x in zip(_each64(s["dy"], s["fmt"], off, False), _each64(s["x"], "e4m3", off, False))])
        return out
    if op == "linear4":
        return s["x"].double() @ _decode64(*s["w"], s["N"], s["K"]).t()
    if op == "experts4":
        off, x = s["offsets"].tolist(), s["x"].double()
        return torch.cat([x[s["tokens"][a:b].long()] @ _decode64(s["w"][0][e], s["w"][1][e], s["N"], s["K"]).t()
                          for e, (a, b) in enumerate(zip(off[:-1], off[1:])) if b > a])

    def rms(v, w):
        return v / torch.sqrt(torch.sum(v ** 2, 1, keepdim=True) / s["H"] + EPS) * w

    y, h, w_pre = s["block"].double(), s["stream"].double(), s["w_pre"].double()
    w_post = None if s["w_post"] is None else s["w_post"].double()
    gate = None if s["g"] is None else s["g"].double()
    leaves = [t.requires_grad_() for t in (y, w_post, gate) if t is not None] if s["grad"] else []

    def behind():
        v = y if w_post is None else rms(y, w_post)
        return v if gate is None else v * gate

    if not s["grad"]:
        h = s["scale"] * h + behind()
        return {"h": h, "x": rms(h, w_pre)}
    h.requires_grad_()
    w_pre.requires_grad_()
    dh, dw = torch.autograd.grad(rms(h, w_pre), (h, w_pre), s["d_x"].double())
    total = dh + s["d_h"].double()
    grads = iter(torch.autograd.grad(behind(), leaves, total))
    out = {"h": s["scale"] * total, "w_pre": dw, "y": next(grads)}
    if w_post is not None:
        out["w_post"] = next(grads)
    if gate is not None:
        out["gate"] = next(grads)
    return out
