"""The microscaled 4-bit operators and the expert router: cases, inputs, plain forms and calls.

A row in microscaled 4-bit form (mx4) has blocks of 32 elements.  A block has one scale byte E, the power of two
2^(E - 127) (255: the block is NaN), and per element a 4-bit code: a sign and one of 0, 0.5, 1, 1.5, 2, 3, 4, 6.  Two
codes share a byte, the first in the low half.

Four operators, by the "op" of a case:
  product     C = act(sum_k A[i][k] * B[j][k]) of operands in that form, the tokens' given or made from 16- or 32-bit
              activations within the pass; with groups > 1 the slabs of a mixture of experts, whose row counts are on
              the GPU
  round       rows (or columns) to that form and back: what training with 4-bit weights computes with
  route       each token's experts and their weights, from the router's logits
  route_grad  the gradient of the logits from those weights' gradients
"""

from __future__ import annotations

import math

import torch

own = False

DTYPES = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}
SIZES = {"f32": 4, "f16": 2, "bf16": 2}
BLOCK = 32
LEVELS = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0)


def _product(name, m, n, k, x, out, groups=1, tokens=0, act="none"):
    """x: the activations' type, or "mx4" where the tokens come as codes; tokens: rows routed to the groups in total."""
    return {"name": name, "op": "product", "m": m, "n": n, "k": k, "x": x, "out": out, "groups": groups,
            "tokens": tokens, "act": act}


def _round(name, r, c, x, out, turned=False):
    """turned: x is stored c x r, so that a block's elements lie a row apart."""
    return {"name": name, "op": "round", "r": r, "c": c, "x": x, "out": out, "turned": turned}


def _routed(name, op, tokens, experts, topk, dtype, score, bias=False, groups=1, top_groups=1, best=2,
            renormalize=True, factor=1.0, padded=0, down=0):
    """padded: tokens at the end of the batch that are only padding (all their logits -inf); down: experts that are out
    of service (their logits -inf)."""
    return {"name": name, "op": op, "tokens": tokens, "experts": experts, "topk": topk, "dtype": dtype, "score": score,
            "bias": bias, "groups": groups, "top_groups": top_groups, "best": best, "renormalize": renormalize,
            "factor": factor, "padded": padded, "down": down}


def listed():
    return [
        # one token of a decoding step through a square projection: bf16 activations quantised on the way
        _product("token_1x8192x8192", 1, 8192, 8192, "bf16", "bf16"),
        # the decode shape of the skinny workload: 16 sequences, one token each, 16384 channels
        _product("decode_16x16384x8192", 16, 16384, 8192, "mx4", "f16"),
        # the ragged workload: no size a multiple of anything, rows at odd addresses, float32 results
        _product("ragged_1000x1500x777", 1000, 1500, 777, "mx4", "f32", act="relu"),
        # a long prompt (or a large batch) through a square projection: the headline workload in 4 bits
        _product("prompt_8192x8192x8192", 8192, 8192, 8192, "mx4", "bf16"),
        # the grouped workload: 8 experts of up to 4096 rows, 16384 rows routed, activations quantised in their slabs
        _product("experts_8x4096x2048x4096", 4096, 2048, 4096, "bf16", "bf16", groups=8, tokens=16384),
        # a weight matrix of a training step
        _round("round_16384x4096", 16384, 4096, "bf16", "bf16"),
        # an operand of a weight gradient's product: blocks along the tokens of odd-sized float32 gradients
        _round("round_columns_1500x8195", 1500, 8195, "f32", "f32", turned=True),
        # routing a decoding step: 64 tokens to 8 of 256 experts in 4 of 8 groups, with a bias for balance
        _routed("route_64x256", "route", 64, 256, 8, "f32", "sigmoid", True, 8, 4, 2, True, 2.5),
        # routing a batch of long prompts the same way, the last tokens of it padding
        _routed("route_65536x256", "route", 65536, 256, 8, "f32", "sigmoid", True, 8, 4, 2, True, 2.5, padded=4099),
        # the router of the grouped workload: 8192 tokens to 2 of 8 experts
        _routed("route_8192x8", "route", 8192, 8, 2, "bf16", "softmax"),
        # a training step's way back through the router of the long batch
        _routed("route_grad_65536x256", "route_grad", 65536, 256, 8, "f32", "sigmoid", factor=2.5, padded=4099),
        # the gradient of a small router whose weights are the probabilities themselves
        _routed("route_grad_1000x60", "route_grad", 1000, 60, 4, "bf16", "softmax", renormalize=False),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def _size(rng, lo, hi):
    """A size spread over the logarithm of its range: every second one a multiple of 128 where it is large enough."""
    v = _log(rng, lo, hi)
    return v // 128 * 128 if v >= 256 and rng.random() < 0.5 else v


def draw(rng):
    op = rng.choice(["product", "product", "experts", "round", "route", "route_grad"])
    if op == "product":
        m, n, k = _size(rng, 1, 8192), _size(rng, 64, 16384), _size(rng, 64, 16384)
        while m * n * k > 8192 ** 3:
            m = max(1, m // 2)
        c = _product("", m, n, k, rng.choice(["mx4", "mx4", "bf16", "f16", "f32"]), rng.choice(["bf16", "f16", "f32"]),
                     act=rng.choice(["none", "none", "relu", "leaky_relu"]))
    elif op == "experts":
        groups = rng.choice([2, 4, 8, 16, 32])
        m, n, k = _size(rng, 8, 4096), _size(rng, 64, 4096), _size(rng, 64, 4096)
        while groups * m * n * k > 8 * 4096 * 2048 * 4096:
            m = max(1, m // 2)
        c = _product("", m, n, k, rng.choice(["mx4", "bf16", "f16"]), rng.choice(["bf16", "f16", "f32"]), groups=groups,
                     tokens=max(1, int(groups * m * rng.uniform(0.2, 0.7))))
    elif op == "round":
        r, n = _size(rng, 1, 32768), _size(rng, 32, 16384)
        while r * n > 16384 * 4096:
            r = max(1, r // 2)
        c = _round("", r, n, rng.choice(["bf16", "f16", "f32"]), rng.choice(["bf16", "f16", "f32"]),
                   rng.random() < 0.4)
    else:
        experts, groups = rng.choice([(8, 1), (16, 1), (60, 1), (64, 1), (64, 8), (128, 1), (160, 8), (256, 8), (256, 1),
                                      (384, 1), (512, 16)])
        top_groups = rng.randint(1, groups)
        topk = min(rng.choice([1, 2, 3, 4, 6, 8]), experts // groups * top_groups)
        score = rng.choice(["softmax", "sigmoid"])
        c = _routed("", op, _size(rng, 1, 32768 if experts > 256 else 65536), experts, topk,
                    rng.choice(["f32", "f32", "bf16", "f16"]), score, rng.random() < 0.5, groups, top_groups,
                    rng.choice([1, 2]), rng.random() < 0.6, rng.choice([1.0, 2.5]), rng.choice([0, 0, 1]),
                    rng.choice([0, 0, 3]))
        c["padded"] *= c["tokens"] // 17
        if op == "route_grad" and topk == 1:
            c["renormalize"] = False  # the weight would be a constant
    del c["name"]
    return c


# ---- inputs -------------------------------------------------------------------------------------------------


def _generator(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return g


def _activations(shape, dtype, g):
    """Normal values with a few channels 8 to 20 times as large, as hidden states have them."""
    x = torch.randn(shape, generator=g, device="cuda", dtype=torch.float32)
    k = shape[-1]
    loud = torch.randperm(k, generator=g, device="cuda")[: max(1, k // 256)]
    x[..., loud] *= 8.0 + 12.0 * torch.rand(loud.numel(), generator=g, device="cuda")
    return x.to(dtype)


def _blocks(x):
    """x (..., C) in float32 as (..., blocks, 32), zeros behind C."""
    x = x.to(torch.float32)
    pad = -x.shape[-1] % BLOCK
    if pad:
        x = torch.cat([x, x.new_zeros((*x.shape[:-1], pad))], -1)
    return x.reshape(*x.shape[:-1], -1, BLOCK)


def _plain_codes(x):
    """(magnitudes' level numbers, signs, scale bytes) of blocks: the largest magnitude's exponent less 2, but at
    least 0, is the scale byte; levels by comparison, ties to the even one."""
    bits = x.view(torch.int32) & 0x7FFFFFFF
    e = ((bits.amax(-1) >> 23) - 2).clamp(min=0)
    inverse = ((254 - e) << 23).view(torch.float32)
    y = (x * inverse[..., None]).abs()
    level = ((y > 0.25).to(torch.uint8) + (y >= 0.75) + (y > 1.25) + (y >= 1.75) + (y > 2.5) + (y >= 3.5) + (y > 5.0))
    return level, x < 0, e.to(torch.uint8)


def _plain_pack(x):
    """(codes, scale bytes) of x (..., C), two codes to a byte."""
    c = x.shape[-1]
    level, minus, e = _plain_codes(_blocks(x))
    code = (level + 8 * minus.to(torch.uint8)).flatten(-2)[..., : c + c % 2]
    return (code[..., 0::2] | (code[..., 1::2] << 4)).contiguous(), e.contiguous()


def _plain_values(q, e, c):
    """float32 values (..., c) of codes and scale bytes."""
    code = torch.stack([q & 15, q >> 4], -1).flatten(-2)[..., :c].int()
    table = torch.tensor([s * v for s in (1.0, -1.0) for v in LEVELS], device=q.device)
    # the power of two by its bits; that of byte 0 lies below the normal range
    e = e.int()
    scale = torch.where(e > 0, e << 23, 1 << 22).view(torch.float32)
    return table[code] * torch.repeat_interleave(scale, BLOCK, -1)[..., :c]


def _logits(case, g):
    """Logits of a router with favoured experts."""
    t, e = case["tokens"], case["experts"]
    x = torch.randn((t, e), generator=g, device="cuda") + 0.5 * torch.randn((e,), generator=g, device="cuda")
    if case["down"]:
        x[:, torch.randperm(e, generator=g, device="cuda")[: case["down"]]] = -math.inf
    if case["padded"]:
        x[t - case["padded"]:] = -math.inf
    return x.to(DTYPES[case["dtype"]])


def prepare(case, seed):
    g = _generator(seed)
    s = {"case": case}
    if case["op"] == "product":
        G, m, n, k = case["groups"], case["m"], case["n"], case["k"]
        x = _activations((G, m, k), DTYPES.get(case["x"], torch.bfloat16), g)
        s["b"], s["sb"] = _plain_pack(torch.randn((G, n, k), generator=g, device="cuda") * (1.0 / math.sqrt(k)))
        if case["x"] == "mx4":
            s["a"], s["sa"] = _plain_pack(x)
        else:
            s["x"] = x.contiguous()
            # room for the codes and scales of the tokens
            s["ws"] = torch.empty((G * m * k + 4096,), dtype=torch.uint8, device="cuda")
        s["c"] = torch.zeros((G, m, n), dtype=DTYPES[case["out"]], device="cuda")
        if G > 1:
            share = torch.rand((G,), generator=g, device="cuda") + 0.25
            rows = torch.floor(share / share.sum() * case["tokens"]).clamp(max=m)
            s["rows"] = rows.to(torch.int32)
        return s
    if case["op"] == "round":
        r, c = case["r"], case["c"]
        x = _activations((r, c), DTYPES[case["x"]], g)
        s["x"] = x.t().contiguous().t() if case["turned"] else x
        s["q"] = torch.empty((r, (c + 1) // 2), dtype=torch.uint8, device="cuda")
        s["e"] = torch.empty((r, (c + BLOCK - 1) // BLOCK), dtype=torch.uint8, device="cuda")
        s["y"] = torch.empty((r, c), dtype=DTYPES[case["out"]], device="cuda")
        return s
    t, e, k = case["tokens"], case["experts"], case["topk"]
    s["logits"] = _logits(case, g)
    # a balance bias, as it stands after some training
    s["bias"] = 0.1 * torch.randn((e,), generator=g, device="cuda") if case["bias"] else None
    s["ids"] = torch.empty((t, k), dtype=torch.int32, device="cuda")
    s["w"] = torch.empty((t, k), dtype=torch.float32, device="cuda")
    if case["op"] == "route_grad":
        s["ids"].copy_(_plain_route(s, case)[0])
        s["dw"] = torch.randn((t, k), generator=g, device="cuda")
        s["dx"] = torch.empty_like(s["logits"])
    return s


# ---- one pass -----------------------------------------------------------------------------------------------


def _act(c, act):
    if act == "none":
        return c
    return torch.where(c > 0, c, torch.zeros_like(c) if act == "relu" else 0.01 * c)


def _plain_product(s, case):
    k = case["k"]
    a, sa = (s["a"], s["sa"]) if case["x"] == "mx4" else _plain_pack(s["x"])
    acc = torch.bmm(_plain_values(a, sa, k), _plain_values(s["b"], s["sb"], k).transpose(1, 2))
    c = _act(acc, case["act"]).to(s["c"].dtype)
    if case["groups"] > 1:
        held = torch.arange(case["m"], device=c.device)[None, :] < s["rows"][:, None]
        c = torch.where(held[..., None], c, s["c"])
    return c


def _plain_scores(logits, score):
    """Scores in 64 bits: a choice between two experts may hang on less than 32 hold."""
    x = logits.double()
    if score == "sigmoid":
        return torch.sigmoid(x)
    top = x.amax(-1, keepdim=True)
    p = torch.exp(x - torch.where(top == -math.inf, 0.0, top))
    return p / p.sum(-1, keepdim=True)


def _plain_route(s, case):
    """(ids, weights): the experts with the best keys (score plus bias) among those of the best groups, in order; ties
    to the lowest index, -1 (and weight 0) where none is left."""
    t, e, k, G = case["tokens"], case["experts"], case["topk"], case["groups"]
    none = s["logits"] == -math.inf
    score = _plain_scores(s["logits"], case["score"])
    key = score if s["bias"] is None else score + s["bias"].double()
    key = torch.where(none, -math.inf, key)
    if case["top_groups"] < G:
        by = torch.sort(key.reshape(t, G, e // G), dim=-1, descending=True).values[..., : case["best"]]
        of = torch.where(by[..., 0] == -math.inf, -math.inf, torch.where(by == -math.inf, 0.0, by).sum(-1))
        order = torch.sort(of, dim=-1, descending=True, stable=True).indices[:, : case["top_groups"]]
        held = torch.zeros((t, G), dtype=torch.bool, device=key.device).scatter_(1, order, True)
        key = torch.where(torch.repeat_interleave(held, e // G, -1), key, -math.inf)
    best, ids = torch.sort(key, dim=-1, descending=True, stable=True)
    best, ids = best[:, :k], ids[:, :k]
    w = torch.where(best == -math.inf, 0.0, torch.gather(score, 1, ids))
    if case["renormalize"]:
        total = w.sum(-1, keepdim=True)
        w = w / torch.where(total == 0, 1.0, total)
    return torch.where(best == -math.inf, -1, ids).to(torch.int32), (w * case["factor"]).to(torch.float32)


def _plain_route_grad(s, case):
    """With p the chosen scores, their gradients g, and for renormalised weights q = p / sum p:
        softmax  factor * s_e * (g_e - sum g p)     over all experts, or factor * q (g - sum g q) over the chosen
        sigmoid  factor * s_e * (1 - s_e) * g_e,    or factor * q (1 - s_e) (g - sum g q)"""
    x = s["logits"].to(torch.float32)
    held = s["ids"] >= 0
    ids = s["ids"].clamp(min=0).long()
    g = torch.where(held, s["dw"] * case["factor"], 0.0)
    if case["score"] == "softmax":
        top = x.amax(-1, keepdim=True)
        p = torch.exp(x - torch.where(top == -math.inf, 0.0, top))
        total = p.sum(-1, keepdim=True)
        p = p / torch.where(total == 0, 1.0, total)
        left = torch.ones_like(p)
    else:
        p, left = torch.sigmoid(x), torch.sigmoid(-x)
    chosen = torch.where(held, torch.gather(p, 1, ids), 0.0)
    if case["renormalize"]:
        total = chosen.sum(-1, keepdim=True)
        q = chosen / torch.where(total == 0, 1.0, total)
        d = q * torch.gather(left, 1, ids) * (g - (g * q).sum(-1, keepdim=True))
        return torch.zeros_like(x).scatter_add_(1, ids, d).to(s["dx"].dtype)
    spread = torch.zeros_like(x).scatter_add_(1, ids, g)
    if case["score"] == "softmax":
        return (p * (spread - (g * chosen).sum(-1, keepdim=True))).to(s["dx"].dtype)
    return (p * left * spread).to(s["dx"].dtype)


def run(state):
    s, case = state, state["case"]
    if own:
        return _own(s, case)
    if case["op"] == "product":
        return _plain_product(s, case)
    if case["op"] == "round":
        q, e = _plain_pack(s["x"])
        return _plain_values(q, e, case["c"]).to(s["y"].dtype)
    return _plain_route(s, case) if case["op"] == "route" else _plain_route_grad(s, case)


def _own(s, case):
    import tiled_shared_memory_amd as tsm

    if case["op"] == "product":
        act = None if case["act"] == "none" else case["act"]
        a, sa = (s["a"], s["sa"]) if case["x"] == "mx4" else (s["x"], None)
        return tsm.matmul_mx4(a, sa, s["b"].transpose(1, 2), s["sb"], rows=s.get("rows"), out=s["c"], activation=act,
                              workspace=s.get("ws"))
    if case["op"] == "round":
        q, e = tsm.quantize_mx4(s["x"], out=s["q"], scale=s["e"])
        return tsm.dequantize_mx4(q, e, out=s["y"])
    if case["op"] == "route":
        return tsm.route_tokens(s["logits"], case["topk"], score=case["score"], bias=s["bias"], groups=case["groups"],
                                top_groups=case["top_groups"], group_best=case["best"],
                                renormalize=case["renormalize"], factor=case["factor"], ids=s["ids"], weights=s["w"])
    return tsm.route_tokens_backward(s["dw"], s["logits"], s["ids"], score=case["score"],
                                     renormalize=case["renormalize"], factor=case["factor"], out=s["dx"])


# ---- what a pass cannot do without ----------------------------------------------------------------------------


def _mx4_bytes(rows, c):
    return rows * ((c + 1) // 2 + (c + BLOCK - 1) // BLOCK)


def work(case):
    if case["op"] == "product":
        G, m, n, k = case["groups"], case["m"], case["n"], case["k"]
        rows = min(case["tokens"], G * m) if G > 1 else m
        x = _mx4_bytes(rows, k) if case["x"] == "mx4" else rows * k * SIZES[case["x"]]
        return {"bytes": x + _mx4_bytes(G * n, k) + rows * n * SIZES[case["out"]], "flops": 2 * rows * n * k}
    if case["op"] == "round":
        r, c = case["r"], case["c"]
        return {"bytes": r * c * (SIZES[case["x"]] + SIZES[case["out"]]) + _mx4_bytes(r, c), "flops": 3 * r * c}
    t, e, k, es = case["tokens"], case["experts"], case["topk"], SIZES[case["dtype"]]
    if case["op"] == "route":
        return {"bytes": t * e * es + 8 * t * k, "flops": 4 * t * e}
    # a softmax's own probabilities need every logit, the others only the chosen experts'
    read = e if case["score"] == "softmax" and not case["renormalize"] else k
    return {"bytes": t * (read + e) * es + 8 * t * k, "flops": 6 * t * read}


# ---- the definitions in 64 bits -------------------------------------------------------------------------------


def _exact_round(x):
    """The values that a row's codes stand for: in each block the multiples of half its unit 2^(floor(log2 m) - 2) up to
    2 units, of one up to 4, of two up to 6, whichever is nearest (the even multiple of two)."""
    c = x.shape[-1]
    b = torch.nn.functional.pad(x.double(), (0, -c % BLOCK)).unflatten(-1, (-1, BLOCK))
    m = b.abs().max(dim=-1, keepdim=True).values
    unit = torch.exp2((torch.frexp(m).exponent - 3).clamp(min=-127).double())
    y = b / unit
    octave = (torch.frexp(y.abs()).exponent - 1).clamp(min=0)
    step = torch.exp2(octave.double() - 1)
    v = (torch.round(y / step) * step).clamp(-6, 6) * unit
    return v.flatten(-2)[..., :c]


def _exact_decode(q, e, c):
    lo, hi = (q % 16).double(), (q // 16).double()
    n = torch.stack([lo, hi], -1).flatten(-2)[..., :c]
    sign, n = torch.where(n >= 8, -1.0, 1.0), n % 8
    v = torch.where(n < 2, n / 2, (1 + (n % 2) / 2) * torch.exp2(torch.floor(n / 2) - 1))
    at = torch.arange(c, device=q.device) // BLOCK
    return sign * v * torch.exp2(e.double() - 127)[..., at]


def _exact_best(key, count):
    """(values, indices) of the `count` largest along the last dimension, the lowest index first among equals; the
    index of -inf is the size."""
    key, n = key.clone(), key.shape[-1]
    at = torch.arange(n, device=key.device)
    values, ids = [], []
    for _ in range(count):
        v = key.max(dim=-1, keepdim=True).values
        i = torch.where((key == v) & (v > -math.inf), at, n).min(dim=-1, keepdim=True).values
        values.append(v)
        ids.append(i)
        key = torch.where(at == i, -math.inf, key)
    return torch.cat(values, -1), torch.cat(ids, -1)


def _exact_weights(x, ids, case):
    """Weights of chosen experts (`ids`, the expert count where there is none) from float64 logits."""
    t, e = x.shape
    finite = torch.where(x == -math.inf, -1e30, x)
    score = torch.softmax(finite, -1) if case["score"] == "softmax" else 1 / (1 + torch.exp(-finite))
    score = torch.cat([score, torch.zeros((t, 1), dtype=torch.float64, device=x.device)], 1)
    w = torch.take_along_dim(score, ids, 1)
    if case["renormalize"]:
        w = w / (w.sum(-1, keepdim=True) + (ids == e).all(-1, keepdim=True))
    return w * case["factor"]


def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "product":
        c, k = s["c"].double(), case["k"]
        for g in range(case["groups"]):
            m = int(s["rows"][g]) if case["groups"] > 1 else case["m"]
            if m == 0:
                continue
            a = _exact_decode(s["a"][g, :m], s["sa"][g, :m], k) if case["x"] == "mx4" else _exact_round(s["x"][g, :m])
            r = torch.mm(a, _exact_decode(s["b"][g], s["sb"][g], k).t().contiguous())
            if case["act"] == "relu":
                r = r.clamp(min=0)
            elif case["act"] == "leaky_relu":
                # the slope as the float32 that the call takes
                r = torch.maximum(r, r * float(torch.tensor(0.01, dtype=torch.float32)))
            c[g, :m] = r
        return c
    if case["op"] == "round":
        return _exact_round(s["x"])
    x, e = s["logits"].double(), case["experts"]
    if case["op"] == "route":
        score = torch.softmax(torch.where(x == -math.inf, -1e30, x), -1) if case["score"] == "softmax" else \
            1 / (1 + torch.exp(-x))
        key = torch.where(x == -math.inf, x, score + (0 if s["bias"] is None else s["bias"].double()))
        G = case["groups"]
        if case["top_groups"] < G:
            v = _exact_best(key.unflatten(1, (G, -1)), case["best"])[0]
            v = torch.where(v[..., 0] > -math.inf, v.masked_fill(v == -math.inf, 0).sum(-1), -math.inf)
            kept = _exact_best(v, case["top_groups"])[1]
            group = torch.arange(e, device=x.device) // (e // G)
            key = torch.where((group[None, :, None] == kept[:, None, :]).any(-1), key, -math.inf)
        return None, _exact_weights(x, _exact_best(key, case["topk"])[1], case)
    ids = torch.where(s["ids"] < 0, e, s["ids"].long())
    with torch.enable_grad():
        # a score of 0, or as good as 0, with a finite exponential
        x = torch.where(x == -math.inf, -1e30 if case["score"] == "softmax" else -600.0, x).requires_grad_(True)
        w = _exact_weights(x, ids, case)
        return torch.autograd.grad((w * s["dw"].double()).sum(), x)[0]
