"""4-bit products whose 256-tiles do not fill whole rounds of the CUs, with the counts on the GPU: the two launches, which
find each for itself from the counts where the rounds end, write every element once.  Against float64."""

import pytest

import mx4_ref as ref
from gpu_util import say
from mx4_ref import check_product, dtypes
from test_mx4 import gen, operand

import tiled_shared_memory_amd as tsm

pytestmark = pytest.mark.gpu

G, M, N, K = 144, 1000, 200, 384  # up to 4 row tiles a group, one column tile, a last slab of half its elements
FEW = 33  # this many leftover tiles and more take a round


def cus():
    import torch

    return torch.cuda.get_device_properties(0).multi_processor_count


def totals():
    """Tiles of 256 x 256 in all, by name."""
    n = cus()
    return {"none": 0, "few": 5, "below": FEW, "round_less_1": n - 1, "round": n, "round_1": n + 1, "most": n + FEW - 1,
            "too_many": n + FEW, "two_rounds": 2 * n, "two_1": 2 * n + 1}


def counts_of(total, g):
    """Counts of `total` row tiles: random ones, some 0, below it and above M."""
    import torch

    tiles = torch.zeros(G, dtype=torch.long)
    order = torch.randperm(G, generator=g, device="cuda").cpu().tolist()
    left = total
    for i, e in enumerate(order):
        least = max(0, left - 4 * (G - 1 - i))
        tiles[e] = min(left, max(least, e * 7 % 5))
        left -= int(tiles[e])
    assert left == 0
    rows = tiles * 256 - torch.randint(0, 256, (G,), generator=g, device="cuda").cpu()
    rows = torch.where(tiles == 4, torch.where(torch.arange(G) % 3 == 0, M + 7, 769 + rows % 232), rows)
    rows = torch.where(tiles == 0, -(torch.arange(G) % 2) * 3, rows)
    held = rows.clamp(0, M)
    assert int(((held + 255) // 256).sum()) == total
    return rows.to(torch.int32).cuda(), held.tolist()


@pytest.fixture(scope="module")
def problem():
    import torch

    g = gen(31)
    a, sa, va = (t.reshape(G, M, -1) for t in operand(G * M, K, 0, 0, g))
    b, sb, vb = (t.reshape(G, N, -1) for t in operand(G * N, K, 0, 0, g, 112, 124))
    want, mag = torch.bmm(va, vb.transpose(1, 2).contiguous()), torch.bmm(va.abs(), vb.abs().transpose(1, 2).contiguous())
    return a, sa, b, sb, want, mag


def kernel_name(a, sa, b, sb, c, batch, rows):
    return tsm.tsm_gemm_mx4_kernel_name(M, N, K, a, K // 2, M * K // 2, sa, K // 32, M * K // 32, b, K // 2, N * K // 2, sb,
                                        K // 32, N * K // 32, c, N, M * N, batch, rows, tsm.TSM_F32)


@pytest.mark.parametrize("out", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("total", ["none", "few", "below", "round_less_1", "round", "round_1", "most", "too_many",
                                   "two_rounds", "two_1"])
def test_counts_around_whole_rounds(problem, total, out):
    """Every remainder that changes the launches; scales of NaN past the counts, results there stay."""
    import torch

    a, sa, b, sb, want, mag = problem
    g = gen(len(total))
    rows, held = counts_of(totals()[total], g)
    own = torch.arange(M, device="cuda")[None, :] < rows[:, None]
    s = torch.where(own[..., None], sa.long(), 255).to(torch.uint8)
    c = torch.full((G, M, N), 55.0, dtype=dtypes()[out], device="cuda")
    say(f"[gpu] mx4 counts around whole rounds {total} {out}")
    assert kernel_name(a, s, b, sb, c, G, rows) == "mx4_tile_256x256x256"
    tsm.matmul_mx4(a, s, b.transpose(1, 2), sb, rows=rows, out=c)
    assert (c[~own] == 55.0).all()
    check_product(c[own], want[own], mag[own], K, out)


def test_counts_that_change_between_replays(problem):
    """One captured call, whose rounds end elsewhere with every count it is replayed with."""
    import torch

    a, sa, b, sb, want, mag = problem
    g = gen(8)
    cases = [counts_of(t, g)[0] for t in totals().values()]
    rows, c = cases[-1].clone(), torch.empty((G, M, N), device="cuda")
    say("[gpu] mx4 counts that change between replays")
    tsm.matmul_mx4(a, sa, b.transpose(1, 2), sb, rows=rows, out=c)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        tsm.matmul_mx4(a, sa, b.transpose(1, 2), sb, rows=rows, out=c)
    for case in cases + cases[:3]:
        rows.copy_(case)
        c.fill_(55.0)
        graph.replay()
        torch.cuda.synchronize()
        own = torch.arange(M, device="cuda")[None, :] < case[:, None]
        assert (c[~own] == 55.0).all()
        check_product(c[own], want[own], mag[own], K, "f32")


@pytest.mark.parametrize("left", [1, 4, FEW - 1, FEW])
def test_batches_around_whole_rounds(problem, left):
    """A strided batch without counts whose last tiles are left over, and one that leaves too many of them."""
    import torch

    a, sa, b, sb, want, mag = problem
    batch, m = (cus() + left), 200  # one tile each
    at = torch.arange(batch, device="cuda")
    a, sa = (t[at % G, :m].contiguous() for t in (a, sa))
    b, sb = (t[at * 5 % G].contiguous() for t in (b, sb))
    c = torch.full((batch, m + 1, N), 55.0, device="cuda")
    va, vb = ref.values(a, sa, K), ref.values(b, sb, K)
    say(f"[gpu] mx4 batch around whole rounds {left}")
    tsm.matmul_mx4(a, sa, b.transpose(1, 2), sb, out=c[:, :m])
    assert (c[:, m] == 55.0).all()
    vb = vb.transpose(1, 2).contiguous()
    check_product(c[:, :m], torch.bmm(va, vb), torch.bmm(va.abs(), vb.abs()), K, "f32")
