"""Plain 64-bit implementations of the MXFP4 cast, the products and the expert-layer operators (numpy / torch CPU).

Written from the definitions (levels and ties spelled out, no bit tricks), apart from the package.
"""
import numpy as np
import torch

LEVELS = np.array([0, 0.5, 1, 1.5, 2, 3, 4, 6])
EVEN = np.array([True, False] * 4)  # mantissa bit 0


def block_exponent(amax: float) -> int:
    """Least e in [-127, 127] with 6 * 2**e >= amax (0 for an empty block)."""
    if amax == 0:
        return 0
    e = -127
    while 6.0 * 2.0 ** e < amax:
        e += 1
    return min(e, 127)


def encode(v: np.ndarray) -> np.ndarray:
    """E2M1 codes of v (float64): nearest level, ties to the even code, sign kept."""
    a = np.abs(v)[..., None]
    d = np.abs(a - LEVELS)
    best = d.min(-1, keepdims=True)
    near = d == best                      # one level, or two at a tie
    even = near & EVEN
    code = np.where(near.sum(-1) > 1, even.argmax(-1), near.argmax(-1))
    return (code + 8 * np.signbit(v)).astype(np.uint8)


def quantize(x: torch.Tensor):
    """(codes [R, 16 * ceil(C/32)], scale bytes [R, ceil(C/32)]) of x [R, C] along its rows."""
    x = x.detach().double().cpu().numpy()
    R, C = x.shape
    nb = -(-C // 32)
    pad = np.zeros((R, nb * 32))
    pad[:, :C] = x
    b = pad.reshape(R, nb, 32)
    codes = np.zeros((R, nb, 32), np.uint8)
    scale = np.zeros((R, nb), np.uint8)
    with np.errstate(invalid="ignore"):
        amax = np.abs(b).max(-1)
    amax[~np.isfinite(b).all(-1)] = np.nan
    values, inverse = np.unique(amax, return_inverse=True)
    exps = np.array([block_exponent(v) if np.isfinite(v) else 128 for v in values])[inverse].reshape(R, nb)
    scale[:] = exps + 127
    good = exps < 128
    codes[good] = encode(b[good] * 2.0 ** -exps[good][:, None].astype(np.float64))
    codes = codes.reshape(R, nb * 32)
    return codes[:, 0::2] | (codes[:, 1::2] << 4), scale


def plane(scale: np.ndarray) -> np.ndarray:
    """The GEMM-ready plane of scale bytes [R, nb], element by element."""
    R, nb = scale.shape
    rt, ct = -(-R // 128), -(-nb // 4)
    out = np.zeros(rt * ct * 512, np.uint8)
    for r in range(R):
        for b in range(nb):
            out[((r // 128) * ct + b // 4) * 512 + 16 * (r % 32) + 4 * (r % 128 // 32) + b % 4] = scale[r, b]
    return out


def values(codes: np.ndarray, scale: np.ndarray, C: int) -> torch.Tensor:
    """float64 values [R, C] from codes and scale bytes [R, nb]."""
    q = np.stack((codes & 15, codes >> 4), -1).reshape(codes.shape[0], -1)
    v = np.where(q >= 8, -1.0, 1.0) * LEVELS[q & 7]
    s = np.where(scale == 255, np.nan, 2.0 ** (scale.astype(np.float64) - 127))
    return torch.from_numpy((v.reshape(len(v), -1, 32) * s[..., None]).reshape(len(v), -1)[:, :C].copy())


def cast(x: torch.Tensor) -> torch.Tensor:
    """What the cast of x stands for, float64."""
    return values(*quantize(x), x.shape[1])


def product_bound(a: torch.Tensor, b: torch.Tensor, bf16: bool):
    """(a @ b.T, allowed error) in float64.  Products are exact; every one of the K additions may drop up to one
    unit of the last of 24 bits of a partial sum, which is at most sum |a||b|; bf16 adds half
    a unit of the last of 8 bits, 2^-8 of a value just above a power of two."""
    ref = a @ b.t()
    tol = a.shape[1] * 2.0 ** -23 * (a.abs() @ b.abs().t())
    return ref, tol + (2.0 ** -8 * (ref.abs() + tol) if bf16 else 0.0)


def scores(logits: torch.Tensor, score: str) -> torch.Tensor:
    l = logits.double()
    if score == "sigmoid":
        return torch.sigmoid(l)
    p = torch.softmax(l, 1)
    return torch.where((l == -np.inf).all(1, keepdim=True), torch.zeros_like(p), p)


def choose(key: torch.Tensor, k: int, groups: int, topk_groups: int, two: bool) -> torch.Tensor:
    """Indices [T, k] by falling key among the best groups (lists and sorted(), ties to the lower index)."""
    T, E = key.shape
    gs = E // groups
    out = torch.zeros((T, k), dtype=torch.int32)
    rank_nan = lambda v: -np.inf if v != v else v  # noqa: E731
    for t in range(T):
        row = [float(v) for v in key[t]]
        is_nan = [v != v for v in row]
        allowed = list(range(E))
        if topk_groups < groups:
            ranks = []
            for g in range(groups):
                part = sorted((v for v in row[g * gs:(g + 1) * gs]), key=rank_nan, reverse=True)
                ranks.append(part[0] + part[1] if two and gs > 1 else part[0])
            best = sorted(range(groups), key=lambda g: (ranks[g] != ranks[g], -rank_nan(ranks[g]), g))[:topk_groups]
            allowed = [e for e in allowed if e // gs in best]
        order = sorted(allowed, key=lambda e: (is_nan[e], -rank_nan(row[e]), e))
        out[t] = torch.tensor(order[:k], dtype=torch.int32)
    return out


def route_weights(p: torch.Tensor, idx: torch.Tensor, renorm: bool, scale: float) -> torch.Tensor:
    w = p.gather(1, idx.long())
    if renorm:
        s = w.sum(1, keepdim=True)
        w = torch.where(s == 0, torch.zeros_like(w), w / torch.where(s == 0, torch.ones_like(s), s))
    return scale * w


def plan(indices: torch.Tensor, E: int):
    """(offsets, slots, tokens) by appending the choices to one list per expert."""
    T, k = indices.shape
    lists = [[] for _ in range(E + 1)]
    for i, e in enumerate(indices.flatten().tolist()):
        lists[e if 0 <= e < E else E].append(i)
    offsets, slots, tokens = [0], [0] * (T * k), []
    for e, members in enumerate(lists):
        for i in members:
            slots[i] = len(tokens) if e < E else -2 - len(tokens)
            tokens.append(i // k if e < E else -1)
        if e < E:
            offsets.append(len(tokens))
    return (torch.tensor(offsets), torch.tensor(slots, dtype=torch.int32).view(T, k), torch.tensor(tokens, dtype=torch.int32))
