"""The router's choice on the GPU where float32 keys do not decide it, against float64."""

import math

import pytest

import mx4_ref as ref
from gpu_util import say
from mx4_ref import dtypes

import tiled_shared_memory_amd as tsm

pytestmark = pytest.mark.gpu


def gen(seed):
    import torch

    return torch.Generator(device="cuda").manual_seed(seed)


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("E,k", [(5, 4), (8, 8), (33, 6), (60, 8), (64, 5), (100, 8), (129, 7), (255, 8), (300, 8), (500, 3),
                                 (60, 12), (500, 20)])
@pytest.mark.parametrize("fmt", ["f32", "bf16"])
def test_biases_of_the_lowest_value(E, k, score, fmt):
    """Experts masked by a bias of float32's lowest value, fewer left than are chosen: the masked ones follow, the lowest
    index first, and none that has a logit of -inf, nor a number past the last expert."""
    import torch

    g = gen(E + k)
    x = torch.randn((67, E), generator=g, device="cuda").to(dtypes()[fmt])
    x[5, : E // 2] = -math.inf
    x[66, 1] = -math.inf
    for left in (0, 1, k - 1, k):
        bias = torch.full((E,), torch.finfo(torch.float32).min, device="cuda")
        at = torch.randperm(E, generator=g, device="cuda")[:left]
        bias[at] = 0.1 * torch.randn(left, generator=g, device="cuda")
        say(f"[gpu] route biases of the lowest value {E} {k} {score} {fmt} {left}")
        ids, w = tsm.route_tokens(x, k, score=score, bias=bias)
        assert torch.equal(ids.long(), ref.choose(x.double(), k, score, bias))
        assert torch.isfinite(w).all()


@pytest.mark.parametrize("E,k,G,top,nbest", [(480, 12, 2, 1, 2), (480, 9, 2, 1, 1), (510, 16, 2, 1, 1), (390, 64, 2, 1, 2),
                                             (504, 8, 3, 1, 2), (453, 4, 3, 2, 2), (483, 20, 3, 2, 1), (511, 6, 7, 3, 2),
                                             (512, 9, 2, 1, 2), (495, 5, 33, 17, 2)])
@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("biased", [False, True], ids=["plain", "bias"])
@pytest.mark.parametrize("fmt", ["f32", "f16", "bf16"])
def test_the_last_expert_of_large_groups(E, k, G, top, nbest, score, biased, fmt):
    """The first and the last expert of every group in its turn the best of a token."""
    import torch

    g = gen(E + k)
    T = 8 * G
    x = torch.randn((T, E), generator=g, device="cuda")
    t, n = torch.arange(T, device="cuda"), E // G
    x[t, t % G * n + t // G % 2 * (n - 1)] += 9
    x[:, E - 1] += 4 * (t % 3 == 0)
    x = x.to(dtypes()[fmt])
    bias = 0.1 * torch.randn(E, generator=g, device="cuda") if biased else None
    say(f"[gpu] route last experts {E} {k} {G} {top} {nbest} {score} {biased} {fmt}")
    ids, _ = tsm.route_tokens(x, k, score=score, bias=bias, groups=G, top_groups=top, group_best=nbest)
    assert torch.equal(ids.long(), ref.choose(x.double(), k, score, bias, G, top, nbest))


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("size", [1.0, 16.0, 1000.0, 30000.0])
@pytest.mark.parametrize("E,k,G,top", [(256, 8, 8, 3), (160, 6, 8, 4), (60, 4, 12, 5), (512, 8, 16, 7), (256, 16, 8, 3),
                                       (240, 12, 6, 2), (512, 10, 64, 20)])
def test_groups_whose_biases_cancel(E, k, G, top, size, score):
    """Groups of one expert with a large bias and one with as large a one below zero: their sums are as near as those
    biases' roundings leave them, far nearer than the keys' own."""
    import torch

    g = gen(E + G)
    T, n = 500, E // G
    for turn in range(4):
        x = torch.randn((1, E), generator=g, device="cuda")
        s = ref.scores(x.double(), score)[0].view(G, n)
        bias = torch.full((G, n), -8.0 * size, device="cuda")
        bias[:, 0] = size * (1 + torch.rand(G, generator=g, device="cuda"))
        bias[:, 1] = -(bias[:, 0].double() + s[:, 0] + s[:, 1]).float()
        bias = bias[:, torch.randperm(n, generator=g, device="cuda")].reshape(E)
        step = min(1.0, size * 2.0 ** -22 * (E if score == "softmax" else 4))  # moves a score by a rounding of its key
        x = x + step * torch.randn((T, E), generator=g, device="cuda")
        say(f"[gpu] route cancelling biases {E} {k} {G} {size} {score}")
        ids, _ = tsm.route_tokens(x, k, score=score, bias=bias, groups=G, top_groups=top, group_best=2)
        want = ref.choose(x.double(), k, score, bias, G, top, 2)
        assert torch.equal(ids.long(), want), f"{int((ids.long() != want).any(1).sum())} tokens"


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("nbest", [1, 2])
@pytest.mark.parametrize("E,k,G,top", [(64, 8, 8, 3), (60, 8, 12, 4), (160, 7, 8, 2), (300, 6, 3, 2), (512, 8, 64, 9),
                                       (64, 12, 8, 2), (160, 33, 8, 3), (504, 20, 3, 2), (512, 64, 16, 5)])
def test_groups_of_the_lowest_value(E, k, G, top, nbest, score):
    """Groups masked by biases of float32's lowest value, whose sums pass its range, beside groups out of service and
    others that a token has no logits for: the masked ones are still chosen before those."""
    import torch

    g = gen(E + k + G)
    T, n = 96, E // G
    low = torch.finfo(torch.float32).min
    for left in (0, 1, top - 1, top + 1):
        x = torch.randn((T, G, n), generator=g, device="cuda")
        x[torch.rand((T, G), generator=g, device="cuda") < 0.4] = -math.inf
        x[5] = -math.inf
        bias = torch.full((G, n), low, device="cuda")
        bias[torch.randperm(G, generator=g, device="cuda")[:left]] = 0.0
        bias[G // 2, 1:] = low / 2
        if left:
            bias[0] = -math.inf
        x, bias = x.view(T, E), bias.view(E)
        say(f"[gpu] route groups of the lowest value {E} {k} {G} {top} {nbest} {score} {left}")
        ids, w = tsm.route_tokens(x, k, score=score, bias=bias, groups=G, top_groups=top, group_best=nbest)
        assert torch.equal(ids.long(), ref.choose(x.double(), k, score, bias, G, top, nbest))
        assert torch.isfinite(w).all()


def microseconds(call, turns=15):
    import torch

    call()
    times = []
    for _ in range(turns):
        start, end = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
        start.record()
        call()
        end.record()
        end.synchronize()
        times.append(start.elapsed_time(end) * 1e3)
    return sorted(times)[turns // 2]


@pytest.mark.parametrize("score,biased", [("softmax", False), ("softmax", True), ("sigmoid", True)])
@pytest.mark.parametrize("E,k,G,top,pow2", [(60, 4, 12, 5, 16), (45, 7, 9, 4, 16), (33, 8, 3, 2, 4), (160, 6, 5, 2, 8)])
def test_any_number_of_groups_takes_the_usual_way(E, k, G, top, pow2, score, biased):
    """Groups that are not a power of two are chosen as quickly as as large ones that are: what fills them up is no near
    tie, which would have every token decided again in float64 (five times as long)."""
    import torch

    g = gen(E)
    say(f"[gpu] route time of {G} groups {score} {biased}")
    took = []
    for experts, groups in ((E, G), (E // G * pow2, pow2)):
        x = torch.randn((65536, experts), generator=g, device="cuda")
        bias = 0.1 * torch.randn(experts, generator=g, device="cuda") if biased else None
        ids, w = tsm.route_tokens(x, k, score=score, bias=bias, groups=groups, top_groups=top)
        took.append(microseconds(lambda: tsm.route_tokens(x, k, score=score, bias=bias, groups=groups, top_groups=top,
                                                          ids=ids, weights=w)))
    assert took[0] <= 2 * took[1], took


@pytest.mark.parametrize("k", [8, 16])
@pytest.mark.parametrize("masked", ["logits", "bias"])
def test_a_group_out_of_service_takes_the_usual_way(k, masked):
    """A whole group without an expert to choose costs nothing, and its absence shows in no choice."""
    import torch

    g = gen(k)
    E, G, top = 256, 8, 4
    x = torch.randn((65536, E), generator=g, device="cuda")
    bias = 0.1 * torch.randn(E, generator=g, device="cuda")
    kw = dict(score="sigmoid", groups=G, top_groups=top)
    say(f"[gpu] route time of a group out of service {k} {masked}")
    ids, w = tsm.route_tokens(x, k, bias=bias, **kw)
    usual = microseconds(lambda: tsm.route_tokens(x, k, bias=bias, ids=ids, weights=w, **kw))
    (x.view(-1, G, E // G) if masked == "logits" else bias.view(1, G, E // G))[:, 3] = -math.inf
    took = microseconds(lambda: tsm.route_tokens(x, k, bias=bias, ids=ids, weights=w, **kw))
    assert torch.equal(ids.long(), ref.choose(x.double(), k, "sigmoid", bias, G, top, 2))
    assert took <= 2 * usual, (took, usual)


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("near", [3, 9, 40])
@pytest.mark.parametrize("E,k,G,top", [(64, 12, 1, 1), (256, 16, 8, 4), (512, 33, 16, 9), (504, 8, 3, 1), (504, 20, 3, 2),
                                       (130, 64, 1, 1), (512, 64, 64, 30), (60, 4, 12, 5), (16, 9, 4, 3)])
def test_near_ties_of_many_choices(E, k, G, top, near, score):
    """Keys that float32 cannot tell apart inside the choice, at its border and past it, of more than 8 choices and of
    groups that are no power of two."""
    import torch

    g = gen(E + near)
    T = 400
    x = torch.randn((1, E), generator=g, device="cuda").expand(T, E)
    s = ref.scores(x[:1].double(), score)[0]
    bias = 0.2 * torch.randn(E, generator=g, device="cuda")
    key = s + bias
    close = key.argsort(descending=True)[max(0, k - (near + 1) // 2):][:near]
    bias[close] = (key[close[:1]] - s[close]).float()
    x = (x.double() + torch.randint(-1, 2, (T, E), generator=g, device="cuda").double() * 2.0 ** -23).float()
    say(f"[gpu] route near ties of many choices {E} {k} {G} {near} {score}")
    for nbest in (1, 2):
        ids, _ = tsm.route_tokens(x, k, score=score, bias=bias, groups=G, top_groups=top, group_best=nbest)
        assert torch.equal(ids.long(), ref.choose(x.double(), k, score, bias, G, top, nbest))


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("E,k,G,top", [(64, 6, 8, 3), (60, 8, 12, 5), (256, 8, 1, 1), (256, 16, 8, 4), (504, 8, 3, 2)])
def test_infinite_biases(E, k, G, top, score):
    """Biases of +inf choose their experts first, in the order of their indices; of -1e9 last."""
    import torch

    g = gen(E + k)
    x = torch.randn((300, E), generator=g, device="cuda")
    for share in (0.01, 0.1, 0.9):
        at = torch.rand(E, generator=g, device="cuda") < share
        for value in (math.inf, -1e9):
            bias = torch.where(at, value, 0.1 * torch.randn(E, generator=g, device="cuda"))
            say(f"[gpu] route infinite biases {E} {k} {G} {score} {share} {value}")
            for nbest in (1, 2):
                ids, w = tsm.route_tokens(x, k, score=score, bias=bias, groups=G, top_groups=top, group_best=nbest)
                assert torch.equal(ids.long(), ref.choose(x.double(), k, score, bias, G, top, nbest))
                assert torch.isfinite(w).all()


@pytest.mark.parametrize("k", [8, 12])
@pytest.mark.parametrize("nbest", [1, 2])
@pytest.mark.parametrize("biased", [False, True], ids=["plain", "bias"])
def test_groups_of_infinite_and_of_the_largest_keys(k, nbest, biased):
    """Sigmoid scores of logits of +inf, and biases of +inf, beside float32's largest value in groups before them."""
    import torch

    g = gen(k)
    E, G, top = 64, 8, 2
    big = torch.finfo(torch.float32).max
    x = torch.randn((64, E), generator=g, device="cuda")
    bias = 0.1 * torch.randn(E, generator=g, device="cuda") if biased else None
    row = torch.arange(64, device="cuda")
    for at, value in ((row % 24, big), (row % 24 + 8, big), (row * 7 % E, math.inf), (row * 5 % 40 + 24, math.inf)):
        if biased:
            bias[at[:2] if value == big else at[2:4]] = value
        else:
            x[row, at] = value
    say(f"[gpu] route groups of infinite keys {k} {nbest} {biased}")
    ids, w = tsm.route_tokens(x, k, score="sigmoid", bias=bias, groups=G, top_groups=top, group_best=nbest)
    assert torch.equal(ids.long(), ref.choose(x.double(), k, "sigmoid", bias, G, top, nbest))
    assert torch.isfinite(w).all()
