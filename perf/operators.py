"""The int8 products with scales and the expert routing operators: cases, inputs, plain forms and calls.

Four operators, by the "op" of a case:
  product   C = act(sa[i] * sb[j] * sum_k A[i][k] * B[j][k]) for int8 codes A (tokens) and B (channels), the tokens'
            codes given or made from 16- or 32-bit activations within the pass; with groups > 1 the slabs of a
            mixture of experts, whose row counts are on the GPU
  sort      each (token, choice) gets a row in its expert's slab, in token order; counts per expert
  dispatch  token rows copied into the slabs, and the gradient (sums of slab rows)
  combine   weighted sums of slab rows, and the gradients of the slabs and of the weights
"""

from __future__ import annotations

import math

import torch

own = False

DTYPES = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}
SIZES = {"f32": 4, "f16": 2, "bf16": 2, "i8": 1}


def _product(name, m, n, k, x, out, groups=1, tokens=0, act="none"):
    """x: the activations' type, or "i8" where the tokens come as codes; tokens: rows routed to the groups in total."""
    return {"name": name, "op": "product", "m": m, "n": n, "k": k, "x": x, "out": out, "groups": groups,
            "tokens": tokens, "act": act}


def _routed(name, op, tokens, topk, experts, capacity, hidden=0, dtype="bf16", backward=False, padded=0):
    """padded: tokens at the end of the batch that are only padding (their expert ids are -1)."""
    return {"name": name, "op": op, "tokens": tokens, "topk": topk, "experts": experts, "capacity": capacity,
            "hidden": hidden, "dtype": dtype, "backward": backward, "padded": padded}


def listed():
    return [
        # one token of a decoding step through a square projection: bf16 activations quantised on the way
        _product("token_1x8192x8192", 1, 8192, 8192, "bf16", "bf16"),
        # the decode shape of the skinny workload: 16 sequences, one token each, 16384 channels
        _product("decode_16x16384x8192", 16, 16384, 8192, "i8", "f16"),
        # the ragged workload: no size a multiple of anything, codes at odd addresses, float32 results
        _product("ragged_1000x1500x777", 1000, 1500, 777, "i8", "f32", act="relu"),
        # a long prompt (or a large batch) through a square projection: the headline workload in int8
        _product("prompt_8192x8192x8192", 8192, 8192, 8192, "i8", "bf16"),
        # the grouped workload: 8 experts of up to 4096 rows, 16384 rows routed, activations quantised in their slabs
        _product("experts_8x4096x2048x4096", 4096, 2048, 4096, "bf16", "bf16", groups=8, tokens=16384),
        # routing a decoding step: 64 tokens, 8 of 256 experts each
        _routed("sort_64x8_of_256", "sort", 64, 8, 256, 64),
        # routing a batch of long prompts, the last tokens of it padding
        _routed("sort_65536x8_of_256", "sort", 65536, 8, 256, 2560, padded=4099),
        # the rows of the grouped workload: 8192 tokens to 2 of 8 experts
        _routed("dispatch_8192x2_h4096", "dispatch", 8192, 2, 8, 4096, hidden=4096, dtype="bf16"),
        # the gradient of a small odd-sized layer's dispatch
        _routed("dispatch_grad_1000x4_h1500", "dispatch", 1000, 4, 16, 400, hidden=1500, dtype="f32", backward=True),
        # a decoding step's way back from the experts
        _routed("combine_32x8_h4096", "combine", 32, 8, 64, 32, hidden=4096, dtype="f16"),
        # the grouped workload's way back
        _routed("combine_8192x2_h4096", "combine", 8192, 2, 8, 4096, hidden=4096, dtype="bf16"),
        # and its training step: gradients of the slabs and of the router's weights
        _routed("combine_grad_8192x2_h4096", "combine", 8192, 2, 8, 4096, hidden=4096, dtype="bf16", backward=True),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def _size(rng, lo, hi):
    """A size spread over the logarithm of its range: every second one a multiple of 128 where it is large enough."""
    v = _log(rng, lo, hi)
    return v // 128 * 128 if v >= 256 and rng.random() < 0.5 else v


def draw(rng):
    op = rng.choice(["product", "product", "experts", "sort", "dispatch", "combine"])
    if op == "product":
        m, n, k = _size(rng, 1, 8192), _size(rng, 64, 16384), _size(rng, 64, 16384)
        while m * n * k > 8192 ** 3:
            m = max(1, m // 2)
        c = _product("", m, n, k, rng.choice(["i8", "i8", "bf16", "f16", "f32"]), rng.choice(["bf16", "f16", "f32"]),
                     act=rng.choice(["none", "none", "relu", "leaky_relu"]))
    elif op == "experts":
        groups = rng.choice([2, 4, 8, 16, 32])
        m, n, k = _size(rng, 8, 4096), _size(rng, 64, 4096), _size(rng, 64, 4096)
        while groups * m * n * k > 8 * 4096 * 2048 * 4096:
            m = max(1, m // 2)
        c = _product("", m, n, k, rng.choice(["i8", "bf16", "f16"]), rng.choice(["bf16", "f16", "f32"]), groups=groups,
                     tokens=max(1, int(groups * m * rng.uniform(0.2, 0.7))))
    else:
        experts = rng.choice([4, 8, 16, 60, 64, 128, 256])
        topk = rng.choice([1, 2, 3, 4, 6, 8])
        topk = min(topk, experts)
        tokens = _size(rng, 1, 65536 if op == "sort" else 16384)
        hidden = 0 if op == "sort" else _size(rng, 64, 8192)
        while tokens * topk * hidden > 8192 * 2 * 4096:
            tokens = max(1, tokens // 2)
        capacity = max(1, min(tokens, int(math.ceil(tokens * topk / experts * rng.uniform(1.0, 3.0)))))
        c = _routed("", op, tokens, topk, experts, capacity, hidden, rng.choice(["bf16", "f16", "f32"]),
                    op != "sort" and rng.random() < 0.5, rng.choice([0, tokens // 17]))
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
    loud = torch.randint(0, k, (max(1, k // 256),), generator=g, device="cuda")
    x[..., loud] *= 8.0 + 12.0 * torch.rand(loud.numel(), generator=g, device="cuda")
    return x.to(dtype)


def _plain_codes(x):
    """(codes as float32 whole numbers, scales): the plain form of the row quantisation."""
    x = x.to(torch.float32)
    amax = x.abs().amax(-1, keepdim=True)
    codes = torch.where(amax > 0, torch.round(127.0 * x.double() / amax.double()).to(torch.float32), torch.zeros_like(x))
    return codes, (amax / 127.0)[..., 0]


def _plain_sort(ids, experts, capacity):
    """(positions, counts) of expert ids (tokens, topk); ids outside [0, experts) get no row."""
    flat = ids.reshape(-1).long()
    key = torch.where((flat >= 0) & (flat < experts), flat, experts)
    by, order = torch.sort(key, stable=True)
    edges = torch.arange(experts + 2, device=ids.device)
    starts = torch.searchsorted(by, edges)
    rank_sorted = torch.arange(by.numel(), device=ids.device) - starts[by]
    rank = torch.empty_like(rank_sorted)
    rank[order] = rank_sorted
    pos = torch.where((key < experts) & (rank < capacity), key * capacity + rank, -1)
    return pos.to(torch.int32).reshape(ids.shape), (starts[1:experts + 1] - starts[:experts]).to(torch.int32)


def _choices(case, g):
    """(ids int32, weights float32) of each token's experts: the top choices of a router with favoured experts."""
    t, k, e = case["tokens"], case["topk"], case["experts"]
    logits = torch.randn((t, e), generator=g, device="cuda") + 0.5 * torch.randn((e,), generator=g, device="cuda")
    top, ids = torch.topk(logits, k, dim=-1)
    ids = ids.to(torch.int32)
    if case["padded"]:
        ids[t - case["padded"]:] = -1
    return ids.contiguous(), torch.softmax(top, -1).contiguous()


def prepare(case, seed):
    g = _generator(seed)
    s = {"case": case}
    if case["op"] == "product":
        G, m, n, k = case["groups"], case["m"], case["n"], case["k"]
        xt = DTYPES.get(case["x"], torch.bfloat16)
        x = _activations((G, m, k), xt, g)
        w = torch.randn((G, n, k), generator=g, device="cuda") * (1.0 / math.sqrt(k))
        wq, ws = _plain_codes(w)
        s["b"], s["sb"] = wq.to(torch.int8).contiguous(), ws.contiguous()
        if case["x"] == "i8":
            xq, xs = _plain_codes(x)
            s["a"], s["sa"] = xq.to(torch.int8).contiguous(), xs.contiguous()
        else:
            s["x"] = x.contiguous()
            s["a"] = torch.empty((G, m, k), dtype=torch.int8, device="cuda")
            s["sa"] = torch.empty((G, m), dtype=torch.float32, device="cuda")
        s["c"] = torch.zeros((G, m, n), dtype=DTYPES[case["out"]], device="cuda")
        if G > 1:
            share = torch.rand((G,), generator=g, device="cuda") + 0.25
            rows = torch.floor(share / share.sum() * case["tokens"]).clamp(max=m)
            s["rows"] = rows.to(torch.int32)
        return s
    ids, weights = _choices(case, g)
    t, h, rows = case["tokens"], case["hidden"], case["experts"] * case["capacity"]
    if case["op"] == "sort":
        s["ids"] = ids
        s["pos"] = torch.empty_like(ids)
        s["counts"] = torch.empty((case["experts"],), dtype=torch.int32, device="cuda")
        s["ws"] = torch.empty((16 << 20,), dtype=torch.uint8, device="cuda")
        return s
    s["pos"], s["w"] = _plain_sort(ids, case["experts"], case["capacity"])[0], weights
    dt = DTYPES[case["dtype"]]
    if case["op"] == "dispatch" and not case["backward"]:
        s["x"] = _activations((t, h), dt, g)
    else:
        # rows that no token has hold what was left there: they must not count
        s["slab"] = torch.randn((rows, h), generator=g, device="cuda").to(dt)
    if case["op"] == "combine" and case["backward"]:
        s["dy"] = torch.randn((t, h), generator=g, device="cuda").to(dt)
    if (case["op"] == "dispatch") == case["backward"] and not (case["op"] == "combine" and case["backward"]):
        s["y"] = torch.empty((t, h), dtype=dt, device="cuda")
    else:
        # one row more than the slabs have, for the plain form's entries without a row
        s["out"] = torch.zeros((rows + 1, h), dtype=dt, device="cuda")
        s["dw"] = torch.empty_like(weights)
    return s


# ---- one pass -----------------------------------------------------------------------------------------------


def _act(c, act):
    if act == "none":
        return c
    return torch.where(c > 0, c, torch.zeros_like(c) if act == "relu" else 0.01 * c)


def _plain_product(s):
    case = s["case"]
    a, sa = (s["a"], s["sa"]) if case["x"] == "i8" else _plain_codes(s["x"])
    acc = torch.bmm(a.to(torch.float32), s["b"].to(torch.float32).transpose(1, 2))
    c = _act(acc * sa[..., None] * s["sb"][:, None, :], case["act"]).to(s["c"].dtype)
    if case["groups"] > 1:
        held = torch.arange(case["m"], device=c.device)[None, :] < s["rows"][:, None]
        c = torch.where(held[..., None], c, s["c"])
    return c


def _rows_of(slab, pos):
    """(tokens, topk, hidden) float32: each choice's slab row, zeros for a choice without one."""
    r = slab[pos.clamp(min=0).long()].to(torch.float32)
    return torch.where((pos >= 0)[..., None], r, torch.zeros_like(r))


def _plain_put(out, pos, rows):
    """out with `rows` (tokens, topk, hidden) at their positions; a choice without one goes to the row past the slabs."""
    at = torch.where(pos >= 0, pos, out.shape[0] - 1).long().reshape(-1)
    out[at] = rows.reshape(at.numel(), -1).to(out.dtype)
    return out[:-1]


def run(state):
    s, case = state, state["case"]
    if own:
        return _own(s, case)
    if case["op"] == "product":
        return _plain_product(s)
    if case["op"] == "sort":
        return _plain_sort(s["ids"], case["experts"], case["capacity"])
    if case["op"] == "dispatch":
        if case["backward"]:
            return _rows_of(s["slab"], s["pos"]).sum(1).to(s["y"].dtype)
        return _plain_put(s["out"], s["pos"], s["x"][:, None, :].expand(-1, case["topk"], -1))
    if not case["backward"]:
        return (_rows_of(s["slab"], s["pos"]) * s["w"][..., None]).sum(1).to(s["y"].dtype)
    dy = s["dy"].to(torch.float32)[:, None, :]
    return _plain_put(s["out"], s["pos"], dy * s["w"][..., None]), (_rows_of(s["slab"], s["pos"]) * dy).sum(-1)


def _own(s, case):
    import tiled_shared_memory_amd as tsm

    if case["op"] == "product":
        if case["x"] != "i8":
            tsm.quantize(s["x"], rows=s.get("rows"), out=s["a"], scale=s["sa"])
        act = None if case["act"] == "none" else case["act"]
        return tsm.matmul_i8(s["a"], s["sa"], s["b"].transpose(1, 2), s["sb"], rows=s.get("rows"), out=s["c"],
                             activation=act)
    if case["op"] == "sort":
        return tsm.sort_tokens(s["ids"], case["experts"], case["capacity"], positions=s["pos"], counts=s["counts"],
                               workspace=s["ws"])
    if case["op"] == "dispatch":
        if case["backward"]:
            return tsm.dispatch_tokens_backward(s["slab"], s["pos"], out=s["y"])
        return tsm.dispatch_tokens(s["x"], s["pos"], out=s["out"][:-1])
    if not case["backward"]:
        return tsm.combine_tokens(s["slab"], s["pos"], s["w"], out=s["y"])
    return tsm.combine_tokens_backward(s["dy"], s["slab"], s["pos"], s["w"], out=s["out"][:-1], dweights=s["dw"])


# ---- what a pass cannot do without ----------------------------------------------------------------------------


def work(case):
    if case["op"] == "product":
        G, m, n, k = case["groups"], case["m"], case["n"], case["k"]
        rows = min(case["tokens"], G * m) if G > 1 else m
        x = rows * k * SIZES[case["x"]] + (4 * rows if case["x"] == "i8" else 0)
        return {"bytes": x + G * n * (k + 4) + rows * n * SIZES[case["out"]], "flops": 2 * rows * n * k}
    t, k, e = case["tokens"] - case["padded"], case["topk"], case["experts"]
    if case["op"] == "sort":
        n = case["tokens"] * k
        return {"bytes": 8 * n + 4 * e, "flops": n}
    es, h = SIZES[case["dtype"]], case["hidden"]
    held = min(t * k, e * case["capacity"])
    if case["op"] == "dispatch":
        return {"bytes": (case["tokens"] if case["backward"] else t) * h * es + held * h * es + 4 * case["tokens"] * k,
                "flops": held * h if case["backward"] else 0}
    if case["backward"]:
        return {"bytes": t * h * es + 2 * held * h * es + 12 * case["tokens"] * k, "flops": 3 * held * h}
    return {"bytes": case["tokens"] * h * es + held * h * es + 8 * case["tokens"] * k, "flops": 2 * held * h}


# ---- the definitions in 64 bits -------------------------------------------------------------------------------


def exact(case, seed):
    if case["op"] == "sort":
        return None  # whole numbers only
    s = prepare(case, seed)
    if case["op"] == "product":
        c = s["c"].double()
        for g in range(case["groups"]):
            m = int(s["rows"][g]) if case["groups"] > 1 else case["m"]
            if m == 0:
                continue
            if case["x"] == "i8":
                a = s["a"][g, :m].double() * s["sa"][g, :m, None].double()
            else:
                # the values that the codes stand for: the nearest multiple of a 127th of the row's largest magnitude
                x = s["x"][g, :m].double()
                step = x.abs().max(dim=1, keepdim=True).values / 127
                a = torch.where(step > 0, torch.round(x * 127 / (127 * step)) * step, 0.0)
            b = s["b"][g].double() * s["sb"][g, :, None].double()
            r = torch.mm(a, b.t().contiguous())
            if case["act"] == "relu":
                r = r.clamp(min=0)
            elif case["act"] == "leaky_relu":
                # the slope as the float32 that the call takes
                r = torch.maximum(r, r * float(torch.tensor(0.01, dtype=torch.float32)))
            c[g, :m] = r
        return c
    t, k, h = case["tokens"], case["topk"], case["hidden"]
    pos, w = s["pos"].long(), s["w"].double()
    if case["op"] == "dispatch" and not case["backward"]:
        out = torch.zeros((case["experts"] * case["capacity"], h), dtype=torch.float64, device="cuda")
        for j in range(k):
            ok = pos[:, j] >= 0
            out[pos[ok, j]] = s["x"][ok].double()
        return out
    slab = s["slab"]
    if case["op"] == "combine" and case["backward"]:
        dslab = torch.zeros((slab.shape[0], h), dtype=torch.float64, device="cuda")
        dw = torch.zeros((t, k), dtype=torch.float64, device="cuda")
        for j in range(k):
            ok = pos[:, j] >= 0
            dy = s["dy"][ok].double()
            dslab[pos[ok, j]] = dy * w[ok, j, None]
            dw[ok, j] = torch.linalg.vecdot(dy, slab[pos[ok, j]].double())
        return dslab, dw
    y = torch.zeros((t, h), dtype=torch.float64, device="cuda")
    for j in range(k):
        ok = pos[:, j] >= 0
        rows = slab[pos[ok, j]].double()
        y[ok] += rows * w[ok, j, None] if case["op"] == "combine" else rows
    return y
