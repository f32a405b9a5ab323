"""The expert router on the GPU, against float64: its choices exactly, its weights and gradients within the roundings
of float32, and a run of it with the other routing calls.

With D the largest distance of a chosen (for a softmax's own probabilities, of any) logit from the row's reference,
exp() of a distance is off by (D + 4) 2^-23 relative, and so is the sum, which adds 24 + topk roundings; quotient and
factor add two.  An error relative to each score is at most UNIT = (2 D + 24 + topk) 2^-23.
"""

import math

import pytest

import mx4_ref as ref
from gpu_util import say
from mx4_ref import HALF_STEP, TINY, check_product, dtypes

import tiled_shared_memory_amd as tsm

pytestmark = pytest.mark.gpu


def gen(seed):
    import torch

    return torch.Generator(device="cuda").manual_seed(seed)


def unit(x, topk):
    import torch

    d = torch.where(torch.isfinite(x), x.abs(), 0.0).amax(-1, keepdim=True)  # from 0 and from the largest: at most 2 d
    return (4 * d + 24 + topk) * 2.0 ** -23


def check_weights(w, ids, x, score, renormalize, factor):
    want = ref.weights(x, ids.long(), score, renormalize, factor)
    err = (w.double() - want).abs()
    bad = ~(err <= want.abs() * unit(x, ids.shape[1]) + 2.0 ** -126)
    assert not bad.any(), f"{int(bad.sum())} weights, {float((err / want.abs()).nan_to_num().max())}"


# experts, topk, groups, top_groups, group_best
LAYOUTS = [(1, 1, 1, 1, 1), (8, 2, 1, 1, 1), (8, 8, 1, 1, 1), (16, 4, 4, 2, 2), (17, 3, 1, 1, 1), (60, 4, 1, 1, 1),
           (60, 6, 12, 5, 2), (64, 8, 8, 3, 1), (64, 64, 1, 1, 1), (66, 5, 33, 20, 2), (128, 8, 64, 9, 2),
           (130, 10, 1, 1, 1), (160, 6, 8, 3, 1), (160, 6, 8, 3, 2), (6, 2, 3, 2, 2), (45, 7, 9, 4, 2), (100, 8, 4, 2, 2), (33, 8, 3, 2, 1),
           (500, 8, 4, 2, 2), (256, 8, 8, 4, 2), (256, 8, 1, 1, 1), (256, 33, 4, 3, 2),
           (384, 8, 1, 1, 1), (500, 7, 4, 2, 2), (512, 16, 16, 9, 2), (512, 64, 2, 1, 1)]


@pytest.mark.parametrize("layout", LAYOUTS, ids=lambda v: "x".join(map(str, v)))
@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("biased", [False, True], ids=["plain", "bias"])
@pytest.mark.parametrize("fmt", ["f32", "f16", "bf16"])
def test_route(layout, score, biased, fmt):
    """Every way to choose, with experts out of service and padded tokens; what lies behind the results stays."""
    import torch

    E, k, G, top, nbest = layout
    g = gen(E * 7 + k)
    for T, pad in ((1, 0), (203, 3)):
        store = torch.randn((T, E + pad), generator=g, device="cuda") * 2
        if T > 1:
            store[T // 2] = -math.inf
            store[5:9, E // 2:] = -math.inf
            store[9, :] = 0.25
            store[10:20] = (store[10:20] * 2).round() / 2  # many equal ones
            store[20:24] *= 6
        store = store.to(dtypes()[fmt])
        x = store[:, :E]
        bias = 0.1 * torch.randn((E,), generator=g, device="cuda") if biased else None
        if biased and E > 4:
            bias[1] = -math.inf
        say(f"[gpu] route {layout} {score} {'bias' if biased else ''} {fmt} {T}")
        buf = torch.full((2, T * k + 64), 5, dtype=torch.int32, device="cuda")
        ids, w = buf[0, :T * k].view(T, k), buf[1, :T * k].view(torch.float32).view(T, k)
        for renormalize, factor in ((True, 2.5), (False, 1.0)):
            tsm.route_tokens(x, k, score=score, bias=bias, groups=G, top_groups=top, group_best=nbest,
                             renormalize=renormalize, factor=factor, ids=ids, weights=w)
            xd = x.double()
            want = ref.choose(xd, k, score, bias, G, top, nbest)
            assert torch.equal(ids.long(), want), (ids.long() != want).nonzero()[:4].tolist()
            check_weights(w, ids, xd, score, renormalize, factor)
            assert (buf[:, T * k:] == 5).all()


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
def test_near_ties(score):
    """Keys that float32 cannot tell apart are told apart, in the order and at the border: biases that all but cancel
    the scores' differences, by one step of float32 either way."""
    import torch

    g = gen(2)
    T, E, k = 512, 64, 6
    x = torch.randn((T, E), generator=g, device="cuda")
    x[:] = x[0]  # one row of logits, so that one bias cancels them all
    s = ref.scores(x[:1].double(), score)[0]
    bias = (0.75 - s).float()
    step = torch.randint(-1, 2, (T, E), generator=g, device="cuda").double() * 2.0 ** -23
    x = (x.double() + step).float()
    say(f"[gpu] route near ties {score}")
    for kw in ({}, {"groups": 8, "top_groups": 3, "group_best": 2}):
        ids, w = tsm.route_tokens(x, k, score=score, bias=bias, **kw)
        want = ref.choose(x.double(), k, score, bias, kw.get("groups", 1), kw.get("top_groups"), 2)
        assert torch.equal(ids.long(), want)
        check_weights(w, ids, x.double(), score, True, 1.0)
    # a bias of zeros chooses as none does, saturated scores among them
    x = torch.randn((T, E), generator=g, device="cuda") * 8
    assert torch.equal(tsm.route_tokens(x, k, score=score, bias=torch.zeros(E, device="cuda"))[0],
                       tsm.route_tokens(x, k, score=score)[0])


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("E,k,G,top", [(8, 2, 1, 1), (8, 8, 1, 1), (16, 4, 4, 2), (16, 8, 8, 5), (60, 8, 1, 1),
                                       (64, 8, 8, 3), (128, 8, 8, 4), (128, 8, 1, 1), (256, 8, 8, 4), (256, 7, 1, 1),
                                       (512, 8, 16, 4), (160, 6, 8, 3), (100, 8, 4, 2), (500, 8, 4, 2)])
@pytest.mark.parametrize("near", [3, 9, 40])
def test_some_near_ties(E, k, G, top, near, score):
    """Tokens some of whose experts, inside the choice, at its border and past it, and in groups at theirs, have keys
    nearer than float32 holds: fewer than the lanes of a token, and more."""
    import torch

    g = gen(E + near)
    T = 700
    x = torch.randn((1, E), generator=g, device="cuda").expand(T, E)
    s = ref.scores(x[:1].double(), score)[0]
    bias = 0.2 * torch.randn(E, generator=g, device="cuda")
    key = s + bias
    at = key.argsort(descending=True)
    lo = max(0, min(k, E) - (near + 1) // 2)
    close = at[lo:lo + near]
    bias[close] = (key[close[:1]] - s[close]).float()  # equal to within a rounding of the bias
    step = torch.randint(-1, 2, (T, E), generator=g, device="cuda").double() * 2.0 ** -23
    x = (x.double() + step).float()
    say(f"[gpu] route some near ties {E} {k} {G} {near} {score}")
    ids, w = tsm.route_tokens(x, k, score=score, bias=bias, groups=G, top_groups=top)
    want = ref.choose(x.double(), k, score, bias, G, top, 2)
    assert torch.equal(ids.long(), want), (ids.long() != want).nonzero()[:4].tolist()
    check_weights(w, ids, x.double(), score, True, 1.0)


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
def test_far_logits(score):
    """Logits far from 0: weights neither overflow nor vanish where they are renormalised."""
    import torch

    x = torch.tensor([[-300.0, -301, -302, -500], [3e38, 1e38, -3e38, 0], [-3e38, -3.1e38, -math.inf, -math.inf],
                      [100, 99, 98, -100], [-100, -100, -100, -100]], device="cuda")
    say(f"[gpu] route far logits {score}")
    ids, w = tsm.route_tokens(x, 2, score=score)
    want = ref.choose(x.double(), 2, "softmax")
    assert torch.equal(ids.long(), want)
    assert torch.isfinite(w).all()
    check_weights(w[[0, 3, 4]], ids[[0, 3, 4]], x[[0, 3, 4]].double(), score, True, 1.0)
    assert (w.sum(-1) - 1).abs().max() < 2.0 ** -20


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("biased", [False, True], ids=["plain", "bias"])
def test_nan_and_infinite_logits(score, biased):
    """A NaN (for a softmax, +inf) gives its token weights of NaN and the ids of its largest logits; other tokens of
    the same wave are as without it."""
    import torch

    g = gen(4)
    T, E, k = 40, 48, 4
    x = torch.randn((T, E), generator=g, device="cuda")
    bias = 0.2 * torch.randn((E,), generator=g, device="cuda") if biased else None
    kw = dict(score=score, bias=bias, groups=4, top_groups=2)
    clean_ids, clean_w = tsm.route_tokens(x, k, **kw)
    y = x.clone()
    y[3, 7] = math.nan
    y[17, 40] = math.inf
    y[18, :] = math.nan
    say(f"[gpu] route NaN {score}")
    ids, w = tsm.route_tokens(y, k, **kw)
    bad = [3, 17, 18] if score == "softmax" else [3, 18]
    held = torch.ones(T, dtype=torch.bool, device="cuda")
    held[[3, 17, 18]] = False
    assert torch.equal(ids[held], clean_ids[held]) and torch.equal(w[held], clean_w[held])
    largest = ref.choose(torch.where(torch.isnan(y), -math.inf, y).double(), k, "softmax")
    for t in bad:
        assert torch.equal(ids[t].long(), largest[t])
        assert torch.isnan(w[t][ids[t] >= 0]).all() and (w[t][ids[t] < 0] == 0).all()
    assert (ids[18] == -1).all()
    if score == "sigmoid":
        want = ref.choose(y[17:18].double(), k, score, bias, 4, 2, 2)
        assert torch.equal(ids[17:18].long(), want)
        check_weights(w[17:18], ids[17:18], y[17:18].double(), score, True, 1.0)


def grad_reference(x, ids, dw, score, renormalize, factor):
    """float64 gradient by autograd from the definition; -inf logits (whose score is 0) get 0."""
    import torch

    with torch.enable_grad():
        none = x == -math.inf
        v = torch.where(none, 0.0, x).requires_grad_(True)
        masked = torch.where(none, -1e30 if score == "softmax" else -600.0, v)
        w = ref.weights(masked, ids, score, renormalize, factor)
        return torch.autograd.grad((w * dw.double()).sum(), v)[0]


@pytest.mark.parametrize("E,k", [(1, 1), (8, 2), (16, 16), (60, 4), (64, 3), (128, 8), (160, 6), (256, 8), (256, 64),
                                 (384, 5), (512, 8)])
@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("renormalize", [False, True], ids=["scores", "renormalised"])
@pytest.mark.parametrize("fmt", ["f32", "f16", "bf16"])
def test_backward(E, k, score, renormalize, fmt):
    """Against autograd in float64: tokens without an expert, with fewer, with one twice, and with ids out of range."""
    import torch

    g = gen(E + k)
    for T, pad in ((1, 0), (101, 5)):
        store = torch.randn((T, E + pad), generator=g, device="cuda")
        if T > 1:
            store[7, E // 2:] = -math.inf
            store[8] = -math.inf
        store = store.to(dtypes()[fmt])
        x = store[:, :E]
        ids = tsm.route_tokens(x, k, score=score)[0]
        if T > 1:
            ids[11, 0] = -1
            ids[12] = -1
            ids[13, -1] = ids[13, 0]
            ids[14, 0] = E + 3
            ids[15, 0] = 7 if E > 7 else 0  # whatever that gives: ids need not be the best
        dw = torch.randn((T, k), generator=g, device="cuda")
        buf = torch.full((T + 1, E + pad), 7.0, dtype=x.dtype, device="cuda")
        say(f"[gpu] route backward {E} {k} {score} {renormalize} {fmt} {T}")
        out = tsm.route_tokens_backward(dw, x, ids, score=score, renormalize=renormalize, factor=1.5, out=buf[:T, :E])
        xd = x.double()
        want = grad_reference(xd, ids.long(), dw, score, renormalize, 1.5)
        # each entry's terms: its own score times its gradient, and the scores' mean of the gradients
        held = (ids >= 0) & (ids < E)
        at = torch.where(held, ids, 0).long()
        p = ref.weights(xd, ids.long(), score, renormalize, 1.0)
        mean = (p * dw.abs().double()).sum(-1, keepdim=True)
        own = torch.zeros_like(xd).scatter_add_(1, at, torch.where(held, 1.5 * p * (dw.abs().double() + mean), 0.0))
        if score == "softmax" and not renormalize:
            own = own + 1.5 * ref.scores(xd, score) * mean
        bound = own * 2 * unit(xd, k) + 2.0 ** -126
        bound = bound + (want.abs() + bound) * (HALF_STEP[fmt] if fmt != "f32" else 0) + TINY[fmt]
        err = (out.double() - want).abs()
        assert (err <= bound).all(), f"{float((err - bound).max())} at {(err - bound).argmax()}"
        assert (buf[T] == 7.0).all() and (buf[:, E:] == 7.0).all()


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("renormalize", [False, True], ids=["scores", "renormalised"])
def test_backward_against_differences(score, renormalize):
    """<gradient, direction> against the change of <weights, dweights> along it, from the forward call's definition
    in 64 bits: differences over 2^-16 are off by their third-order term, below 2^-30 here."""
    import torch

    g = gen(9)
    T, E, k = 64, 32, 4
    x = torch.randn((T, E), generator=g, device="cuda")
    ids, _ = tsm.route_tokens(x, k, score=score, renormalize=renormalize)
    dw, d = torch.randn((T, k), generator=g, device="cuda"), torch.randn((T, E), generator=g, device="cuda").double()
    say("[gpu] route backward differences")
    got = (tsm.route_tokens_backward(dw, x, ids, score=score, renormalize=renormalize).double() * d).sum(-1)
    h = 2.0 ** -16

    def at(v):
        return (ref.weights(v, ids.long(), score, renormalize, 1.0) * dw.double()).sum(-1)

    want = (at(x.double() + h * d) - at(x.double() - h * d)) / (2 * h)
    size = (dw.abs().double().sum(-1) * d.abs().amax(-1))
    assert ((got - want).abs() <= size * (2 * unit(x.double(), k)[:, 0] + E * 2.0 ** -24) + 2.0 ** -26).all()


def test_many_tokens_on_another_stream_and_captured():
    """More tokens than one round of workgroups; a stream of its own; captured with its gradient and replayed."""
    import torch

    g = gen(6)
    T, E, k = 70001, 256, 8
    x = torch.randn((T, E), generator=g, device="cuda")
    bias = 0.1 * torch.randn((E,), generator=g, device="cuda")
    kw = dict(score="sigmoid", bias=bias, groups=8, top_groups=4, factor=2.5)
    say("[gpu] route many tokens")
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    ids, w = tsm.route_tokens(x, k, stream=side, **kw)
    side.synchronize()
    assert torch.equal(ids.long(), ref.choose(x.double(), k, "sigmoid", bias, 8, 4, 2))
    check_weights(w, ids, x.double(), "sigmoid", True, 2.5)
    small = x[:600].clone()
    sid, sw = torch.empty((600, k), dtype=torch.int32, device="cuda"), torch.empty((600, k), device="cuda")
    dx, dw = torch.empty_like(small), torch.randn((600, k), generator=g, device="cuda")
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        tsm.route_tokens(small, k, ids=sid, weights=sw, **kw)
        tsm.route_tokens_backward(dw, small, sid, score="sigmoid", factor=2.5, out=dx)
    for r in range(4):
        small.copy_(torch.randn((600, E), generator=g, device="cuda"))
        dw.copy_(torch.randn((600, k), generator=g, device="cuda"))
        graph.replay()
        torch.cuda.synchronize()
        want_ids, want_w = tsm.route_tokens(small, k, **kw)
        assert torch.equal(sid, want_ids) and torch.equal(sw, want_w), r
        assert torch.equal(dx, tsm.route_tokens_backward(dw, small, want_ids, score="sigmoid", factor=2.5)), r


def test_expert_layer():
    """Logits to experts to results and back, as a layer runs: the router's product, the choice, the sort, slabs,
    4-bit products with activations quantised on the way, the weighted sum; and the gradients of weights and logits."""
    import torch

    g = gen(12)
    T, H, F, E, k, cap = 150, 256, 320, 16, 3, 64
    x = torch.randn((T, H), generator=g, device="cuda").to(torch.bfloat16)
    gate = torch.randn((E, H), generator=g, device="cuda").to(torch.bfloat16) / 16
    up, up_s = tsm.quantize_mx4(torch.randn((E, F, H), generator=g, device="cuda") / 16)
    down, down_s = tsm.quantize_mx4(torch.randn((E, H, F), generator=g, device="cuda") / 16)
    say("[gpu] mx4 expert layer")
    logits = tsm.matmul(x, gate.t())
    logits[T - 7:] = -math.inf  # padded tokens
    ids, w = tsm.route_tokens(logits, k, score="sigmoid", factor=1.5)
    pos, counts = tsm.sort_tokens(ids, E, cap)
    slab = tsm.dispatch_tokens(x, pos, slots=E * cap)
    h = tsm.matmul_mx4(slab.view(E, cap, H), None, up.transpose(1, 2), up_s, rows=counts, activation="relu",
                       out_dtype=torch.bfloat16)
    o = tsm.matmul_mx4(h, None, down.transpose(1, 2), down_s, rows=counts)
    y = tsm.combine_tokens(o.view(E * cap, H), pos, w)

    want_ids = ref.choose(logits.double(), k, "sigmoid")
    assert torch.equal(ids.long(), want_ids) and (ids[T - 7:] == -1).all()
    assert torch.equal(counts.long(), torch.bincount(want_ids[want_ids >= 0], minlength=E))
    # token by token, from the rounded values that the layer itself passes on
    rows = torch.zeros((T, k, H), dtype=torch.float64, device="cuda")
    for e in range(E):
        t, j = (want_ids == e).nonzero(as_tuple=True)
        if t.numel() == 0:
            continue
        assert t.numel() <= cap
        xq, xs = ref.quantize(x[t])
        hidden, mag = ref.product(ref.values(ref.pack(xq), xs, H), ref.values(up[e], up_s[e], H), "relu")
        got_h = h[e, :t.numel()]
        check_product(got_h, hidden, mag, H, "bf16")
        hq, hs = ref.quantize(got_h)
        res, mag = ref.product(ref.values(ref.pack(hq), hs, F), ref.values(down[e], down_s[e], F))
        check_product(o[e, :t.numel()], res, mag, F, "f32")
        rows[t, j] = o[e, :t.numel()].double()
    want = (rows * w.double()[..., None]).sum(1)
    assert ((y.double() - want).abs() <= (k + 1) * 2.0 ** -24 * (rows.abs() * w.double()[..., None]).sum(1)).all()
    assert (y[T - 7:] == 0).all()

    dy = torch.randn((T, H), generator=g, device="cuda")
    _, dw = tsm.combine_tokens_backward(dy, o.view(E * cap, H), pos, w)
    dlogits = tsm.route_tokens_backward(dw, logits, ids, score="sigmoid", factor=1.5)
    want_dw = (rows * dy.double()[:, None, :]).sum(-1)
    tol = H * 2.0 ** -24 * (rows.abs() * dy.abs().double()[:, None, :]).sum(-1)
    assert ((dw.double() - want_dw).abs() <= tol + 1e-30).all()
    full = grad_reference(logits.double(), ids.long(), dw, "sigmoid", True, 1.5)
    size = 1.5 * dw.abs().double().sum(-1, keepdim=True)
    assert ((dlogits.double() - full).abs() <= size * 2 * unit(logits.double(), k)).all()
    assert (dlogits[T - 7:] == 0).all()
