"""Microscaled 4-bit rows and the expert router from their definitions, in 64 bits."""

import math

import numpy as np

HALF_STEP = {"f32": 2.0 ** -24, "f16": 2.0 ** -11, "bf16": 2.0 ** -8}
TINY = {"f32": 2.0 ** -150, "f16": 2.0 ** -25, "bf16": 2.0 ** -134}  # half the spacing of the subnormals
LEVELS = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0)


def dtypes():
    import torch

    return {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}


def quantize(x):
    """(codes, scale bytes) of x (..., C), one number a code: nearest level to |x| / scale, ties to the even code."""
    import torch

    C = x.shape[-1]
    b = torch.nn.functional.pad(x.double(), (0, -C % 32)).unflatten(-1, (-1, 32))
    m = b.abs().amax(-1)
    ok = torch.isfinite(b).all(-1)
    e = torch.frexp(torch.where(ok, m, 1.0)).exponent - 1  # floor(log2 m); of 0: -1, which the maximum takes away
    e = torch.where(m == 0, 0, (e + 125).clamp(min=0))
    y = b.abs() / torch.exp2(e.double() - 127)[..., None]
    levels = torch.tensor(LEVELS, dtype=torch.float64, device=x.device)
    far = (y[..., None] - levels).abs()
    least = far.amin(-1, keepdim=True)
    near = far == least  # one level, or the two of a tie
    number = torch.arange(8, device=x.device)
    first = torch.where(near, number, 9).amin(-1)
    last = torch.where(near, number, -1).amax(-1)
    code = torch.where(first % 2 == 0, first, last) + 8 * torch.signbit(b).long()
    code = torch.where(ok[..., None], code, 0)
    return code.flatten(-2)[..., :C], torch.where(ok, e, 255)


def pack(code):
    """Codes (..., C), a number each, two to a byte."""
    import torch

    code = torch.nn.functional.pad(code.to(torch.uint8), (0, code.shape[-1] % 2))
    return (code[..., 0::2] | (code[..., 1::2] << 4)).contiguous()


def values(q, e, C):
    """float64 values of packed codes and scale bytes; NaN in blocks of 255."""
    import torch

    code = torch.stack([q & 15, q >> 4], -1).flatten(-2)[..., :C].long()
    table = torch.tensor([*LEVELS, *(-v for v in LEVELS)], dtype=torch.float64, device=q.device)
    scale = torch.where(e == 255, math.nan, torch.exp2(e.double() - 127))
    return table[code] * scale.repeat_interleave(32, -1)[..., :C]


def product(a, b, act=None, slope=0.0):
    """(a . b^T, |a| . |b|^T) of float64 rows, the first through the activation (a NaN stays one)."""
    import torch

    c, s = torch.mm(a, b.t().contiguous()), torch.mm(a.abs(), b.abs().t().contiguous())
    if act == "relu":
        c = torch.where(c <= 0, 0.0, c)
    elif act == "leaky_relu":
        c = torch.where(c <= 0, c * float(np.float32(slope)), c)
        s = s * max(1.0, abs(slope))
    return c, s


def check_product(got, ref, mag, K, out, extra=0.0):
    """|got - ref| within K roundings of float32 of the sum of magnitudes (and `extra` relative), and the output's."""
    import torch

    bound = mag * (K + 1) * 2.0 ** -24 + ref.abs() * extra + 2.0 ** -126
    if out != "f32":
        bound = bound + (ref.abs() + bound) * HALF_STEP[out] + TINY[out]
    err = (got.double() - ref).abs()
    bad = ~(err <= bound)
    assert not bad.any(), f"{int(bad.sum())} cells, first {bad.nonzero()[0].tolist()}: {float(err[bad].max())}"


def best(key, count):
    """Indices of the `count` largest along the last dimension, the lowest index first among equals; the size where
    only -inf is left."""
    import torch

    key, n = key.clone(), key.shape[-1]
    at = torch.arange(n, device=key.device)
    ids = []
    for _ in range(count):
        v = key.amax(-1, keepdim=True)
        i = torch.where((key == v) & (v > -math.inf), at, n).amin(-1, keepdim=True)
        ids.append(i)
        key = torch.where(at == i, -math.inf, key)
    return torch.cat(ids, -1)


def scores(x, score):
    """float64 scores; -inf gives 0, and rows of nothing but -inf zeros."""
    import torch

    if score == "sigmoid":
        return 1 / (1 + torch.exp(-x))
    top = x.amax(-1, keepdim=True)
    p = torch.exp(x - torch.where(top == -math.inf, 0.0, top))
    total = p.sum(-1, keepdim=True)
    return p / torch.where(total == 0, 1.0, total)


def weights(x, ids, score, renormalize, factor):
    """float64 weights of chosen experts from float64 logits; 0 for ids outside the experts."""
    import torch

    E = x.shape[1]
    held = (ids >= 0) & (ids < E)
    at = torch.where(held, ids, 0).long()
    if renormalize:
        # shifted by the largest chosen logit below 0, so that sums of tiny scores stay sums
        c = torch.gather(x, 1, at)
        c = torch.where(held, c, -math.inf)
        top = c.amax(-1, keepdim=True)
        top = top.clamp(max=0) if score == "sigmoid" else top
        top = torch.where(top == -math.inf, 0.0, top).detach()
        s = torch.exp(c - top) if score == "softmax" else torch.exp(c.clamp(max=0) - top) / (1 + torch.exp(-c.abs()))
        s = torch.where(held, s, 0.0)
        total = s.sum(-1, keepdim=True)
        return factor * s / torch.where(total == 0, 1.0, total)
    return torch.where(held, factor * torch.gather(scores(x, score), 1, at), 0.0)


def choose(x, topk, score, bias=None, groups=1, top_groups=None, group_best=2):
    """Chosen ids (-1: none left) from float64 logits without NaN."""
    import torch

    E = x.shape[1]
    s = scores(x, score) + (0 if bias is None else bias.double())
    s = torch.where(x == -math.inf, -math.inf, s)
    key = x if bias is None else s
    if top_groups is not None and top_groups < groups:
        of = s if bias is not None or group_best > 1 else x
        v = torch.sort(of.unflatten(1, (groups, -1)), -1, descending=True).values[..., :group_best]
        total = torch.where(v == -math.inf, 0.0, v).sum(-1)
        kept = best(torch.where(v[..., 0] == -math.inf, -math.inf, total), top_groups)
        group = torch.arange(E, device=x.device) // (E // groups)
        key = torch.where((group[None, :, None] == kept[:, None, :]).any(-1), key, -math.inf)
    ids = best(key, topk)
    return torch.where(ids == E, -1, ids)
