"""Tokens sorted by expert, into the slabs and back, with gradients, on the GPU against float64.

Positions and counts are whole numbers and equal; dispatched rows are copies.  A
weighted sum of k rows makes k float32 roundings of partial sums no larger than
sum |w x|; a dot product over H makes at most H (+ 8 for the final tree); a
16-bit result adds half a step.
"""

import numpy as np
import pytest

from gpu_util import say

import tiled_shared_memory_amd as tsm

pytestmark = pytest.mark.gpu

HALF_STEP = {"f32": 0.0, "f16": 2.0 ** -11, "bf16": 2.0 ** -8}
TINY = {"f32": 0.0, "f16": 2.0 ** -25, "bf16": 0.0}


def dtypes():
    import torch

    return {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16, "i8": torch.int8}


def plain_sort(ids, experts, capacity):
    T, k = ids.shape
    pos = np.full((T, k), -1, np.int32)
    counts = np.zeros(experts, np.int32)
    if T * k > 100000:  # the same, expert by expert
        flat, out = ids.reshape(-1), pos.reshape(-1)
        for e in range(experts):
            at = np.flatnonzero(flat == e)
            counts[e] = at.size
            out[at[:capacity]] = e * capacity + np.arange(min(at.size, capacity))
        return pos, counts
    for t in range(T):
        for j in range(k):
            e = int(ids[t, j])
            if 0 <= e < experts:
                if counts[e] < capacity:
                    pos[t, j] = e * capacity + counts[e]
                counts[e] += 1
    return pos, counts


SORTS = [(0, 3, 4, 5), (5, 0, 4, 5), (1, 1, 1, 1), (1, 8, 8, 1), (64, 8, 256, 64), (1000, 2, 8, 300), (1024, 8, 512, 40),
         (1025, 8, 60, 150), (4096, 2, 3, 5000), (4097, 2, 500, 7), (20000, 3, 16, 4000), (9000, 1, 1, 9000),
         (140000, 8, 37, 30000), (2100000, 2, 5, 900000)]


@pytest.mark.parametrize("T,k,E,cap", SORTS)
@pytest.mark.parametrize("wide", [False, True], ids=["i32", "i64"])
def test_sort(T, k, E, cap, wide):
    """One workgroup and several, skewed choices, ids outside the experts, capacities that drop."""
    import torch

    rng = np.random.default_rng(T + k + E)
    ids = np.minimum(rng.geometric(3.0 / (E + 2), (T, k)) - 1, E + 1) if E > 2 else rng.integers(0, E, (T, k))
    ids = np.where(rng.random((T, k)) < 0.05, -1, ids).astype(np.int64)
    if wide and T > 2 and k:
        ids[1, 0], ids[2, 0] = 2 ** 32 + 1, -2 ** 40  # outside, though their low halves are not
    pos, counts = plain_sort(ids, E, cap)
    dev = torch.from_numpy(ids if wide else ids.astype(np.int32)).cuda()
    say(f"[gpu] sort {T}x{k} of {E} cap {cap} {dev.dtype}")
    ws = tsm.sort_workspace_for(dev, E)
    assert (ws is None) == (T * k <= 8192)
    for _ in range(2):
        if ws is not None:
            ws.fill_(255)
        p, c = tsm.sort_tokens(dev, E, cap, workspace=ws)
        assert np.array_equal(c.cpu().numpy(), counts)
        assert np.array_equal(p.cpu().numpy(), pos)
    # a column slice of a wider table
    if T and k:
        table = torch.full((T, k + 3), -1, dtype=dev.dtype, device="cuda")
        table[:, 1:1 + k] = dev
        p, c = tsm.sort_tokens(table[:, 1:1 + k], E, cap)
        assert np.array_equal(c.cpu().numpy(), counts) and np.array_equal(p.cpu().numpy(), pos)


def routed(T, k, E, cap, seed, drop=0.1):
    """Positions with some choices dropped, and random weights."""
    import torch

    rng = np.random.default_rng(seed)
    ids = np.where(rng.random((T, k)) < drop, -1, rng.integers(0, E, (T, k)))
    if T > 3:
        ids[3] = -1  # a token without any expert
    pos, counts = plain_sort(ids, E, cap)
    w = rng.standard_normal((T, k)).astype(np.float32)
    return torch.from_numpy(pos).cuda(), torch.from_numpy(w).cuda(), counts


ROWS = [  # T, k, E, cap, H, leading dimension of rows - H
    (1, 1, 1, 1, 1, 0), (1, 8, 8, 2, 4096, 0), (37, 2, 4, 20, 7, 0), (50, 3, 5, 33, 64, 8), (33, 4, 8, 20, 1500, 0),
    (20, 5, 6, 30, 1501, 3), (64, 8, 16, 40, 128, 0), (130, 1, 4, 40, 8200, 0), (9, 9, 3, 40, 2048, 1),
    (1000, 2, 8, 260, 512, 0), (6, 70, 12, 60, 100, 0)]


def value(shape, dt, gen):
    import torch

    if dt == torch.int8:
        return torch.randint(-128, 128, shape, generator=gen, device="cuda", dtype=torch.int8)
    return torch.randn(shape, generator=gen, device="cuda").to(dt)


def with_ld(x, pad, fill):
    """x as a view of rows `pad` longer, starting one element into its buffer; the buffer for checking the padding."""
    import torch

    T, H = x.shape
    buf = torch.full((T * (H + pad) + 1,), fill, dtype=x.dtype, device="cuda")
    v = buf[1 if pad else 0:].as_strided((T, H), (H + pad, 1))
    v.copy_(x)
    return v, buf


@pytest.mark.parametrize("case", ROWS, ids=lambda c: "x".join(map(str, c)))
@pytest.mark.parametrize("fmt", ["f32", "f16", "bf16", "i8"])
def test_dispatch(case, fmt):
    import torch

    T, k, E, cap, H, pad = case
    g = torch.Generator(device="cuda").manual_seed(T + H)
    pos, _, _ = routed(T, k, E, cap, T + H)
    x, _ = with_ld(value((T, H), dtypes()[fmt], g), pad, 1)
    slabs, buf = with_ld(torch.full((E * cap, H), 33, dtype=x.dtype, device="cuda"), pad, 55)
    scale = torch.rand(T, generator=g, device="cuda")
    ss = torch.full((E * cap,), 44.0, device="cuda")
    say(f"[gpu] dispatch {case} {fmt}")
    tsm.dispatch_tokens(x, pos, out=slabs, scale=scale, out_scale=ss)
    want = torch.full((E * cap, H), 33, dtype=x.dtype, device="cuda")
    want_s = torch.full((E * cap,), 44.0, device="cuda")
    for t in range(T):
        for j in range(k):
            p = int(pos[t, j])
            if p >= 0:
                want[p], want_s[p] = x[t], scale[t]
    assert torch.equal(slabs, want) and torch.equal(ss, want_s)
    if pad:
        at = torch.ones(buf.numel(), dtype=torch.bool, device="cuda")
        at[1:].as_strided((E * cap, H), (H + pad, 1)).fill_(False)
        assert (buf[at] == 55).all()
    plain = torch.full_like(slabs, 33)
    tsm.dispatch_tokens(x, pos, out=plain)
    assert torch.equal(plain, want)


def reference(slab, pos, w):
    """float64 sums and the sums of magnitudes."""
    import torch

    T, k = pos.shape
    y = torch.zeros((T, slab.shape[1]), dtype=torch.float64, device="cuda")
    mag = torch.zeros_like(y)
    for j in range(k):
        ok = pos[:, j] >= 0
        r = slab[pos[ok, j].long()].double() * (w[ok, j, None].double() if w is not None else 1.0)
        y[ok] += r
        mag[ok] += r.abs()
    return y, mag


def within(got, ref, bound, fmt):
    import torch

    bound = bound + (ref.abs() + bound) * HALF_STEP[fmt] + TINY[fmt]
    err = (got.double() - ref).abs()
    bad = ~(err <= bound)
    assert not bad.any(), f"{int(bad.sum())} off, first {bad.nonzero()[0].tolist()}"
    assert torch.isfinite(got).all()


@pytest.mark.parametrize("case", ROWS, ids=lambda c: "x".join(map(str, c)))
@pytest.mark.parametrize("fmt", ["f32", "f16", "bf16"])
def test_combine_and_gradients(case, fmt):
    """Rows without an entry hold NaN: they must not count.  NaN weights of choices without a position neither."""
    import torch

    T, k, E, cap, H, pad = case
    g = torch.Generator(device="cuda").manual_seed(T * 3 + H)
    pos, w, _ = routed(T, k, E, cap, T + H + 1)
    held = torch.zeros(E * cap, dtype=torch.bool, device="cuda")
    held[pos[pos >= 0].long()] = True
    raw = value((E * cap, H), dtypes()[fmt], g)
    raw[~held] = float("nan")
    slabs, _ = with_ld(raw, pad, float("nan"))
    w[pos < 0] = float("nan")
    clean = torch.where(held[:, None], raw, torch.zeros_like(raw))
    say(f"[gpu] combine {case} {fmt}")
    y, ybuf = with_ld(torch.full((T, H), float("nan"), dtype=raw.dtype, device="cuda"), pad, 55.0)
    tsm.combine_tokens(slabs, pos, w, out=y)
    ref, mag = reference(clean, pos, w)
    within(y, ref, k * 2.0 ** -24 * mag, fmt)
    if pad:
        at = torch.ones(ybuf.numel(), dtype=torch.bool, device="cuda")
        at[1:].as_strided((T, H), (H + pad, 1)).fill_(False)
        assert (ybuf[at] == 55.0).all()
    # the gradient of dispatch
    dx = tsm.dispatch_tokens_backward(slabs, pos)
    ref, mag = reference(clean, pos, None)
    within(dx, ref, k * 2.0 ** -24 * mag, fmt)
    # the gradients of combine
    dy, _ = with_ld(value((T, H), dtypes()[fmt], g), pad, 1.0)
    ds, _ = with_ld(torch.full((E * cap, H), 33.0, dtype=raw.dtype, device="cuda"), pad, 55.0)
    ds, dw = tsm.combine_tokens_backward(dy, slabs, pos, w, out=ds)
    for j in range(k):
        ok = pos[:, j] >= 0
        at = pos[ok, j].long()
        d64 = dy[ok].double()
        within(ds[at], d64 * w[ok, j, None].double(), (d64 * w[ok, j, None].double()).abs() * 2.0 ** -24, fmt)
        prod = d64 * clean[at].double()
        assert (dw[~ok, j] == 0).all()
        err = (dw[ok, j].double() - prod.sum(-1)).abs()
        assert (err <= (H + 8) * 2.0 ** -24 * prod.abs().sum(-1)).all()
    assert (ds[~held] == 33.0).all()
    # without weights: ones
    ds1, _ = tsm.combine_tokens_backward(dy, slabs, pos, None)
    for j in range(k):
        ok = pos[:, j] >= 0
        assert torch.equal(ds1[pos[ok, j].long()], dy[ok])
    assert (ds1[~held] == 0).all()


def test_gradients_against_differences():
    """Central differences of a scalar loss of combine(dispatch(x)) in every x and weight (float32 kernels, the
    function is bilinear, so a difference over a step of 1 is exact up to the sums' roundings)."""
    import torch

    T, k, E, cap, H = 6, 3, 4, 4, 10
    g = torch.Generator(device="cuda").manual_seed(0)
    pos, w, _ = routed(T, k, E, cap, 2, drop=0.2)
    x, dy = value((T, H), torch.float32, g), value((T, H), torch.float32, g)

    def loss(x, w):
        s = tsm.dispatch_tokens(x, pos, out=torch.zeros((E * cap, H), device="cuda"))
        return float((tsm.combine_tokens(s, pos, w).double() * dy.double()).sum())

    say("[gpu] routing gradients against differences")
    s = tsm.dispatch_tokens(x, pos, out=torch.zeros((E * cap, H), device="cuda"))
    ds, dw = tsm.combine_tokens_backward(dy, s, pos, w)
    dx = tsm.dispatch_tokens_backward(ds, pos)
    # the loss sums T * H = 60 products of magnitude below 4 * 3 * 3 * 4 = 144, each y with k + 1 roundings
    tol = 2 * 60 * 144 * (k + 3) * 2.0 ** -24
    for t in range(T):
        for i in range(H):
            d = torch.zeros_like(x)
            d[t, i] = 1.0
            assert abs((loss(x + d, w) - loss(x - d, w)) / 2 - float(dx[t, i])) <= tol
        for j in range(k):
            d = torch.zeros_like(w)
            d[t, j] = 1.0
            assert abs((loss(x, w + d) - loss(x, w - d)) / 2 - float(dw[t, j])) <= tol


def test_positions_outside_the_slabs_are_ignored():
    import torch

    say("[gpu] positions outside")
    pos = torch.tensor([[0, 7], [2 ** 31 - 1, 3], [-2 ** 31, 4]], dtype=torch.int32, device="cuda")
    x = torch.arange(1, 4, device="cuda", dtype=torch.float32)[:, None].expand(3, 40).contiguous()
    s = tsm.dispatch_tokens(x, pos, out=torch.zeros((4, 40), device="cuda"))
    assert [float(v) for v in s[:, 0]] == [1.0, 0.0, 0.0, 2.0]
    y = tsm.combine_tokens(s, pos)
    assert [float(v) for v in y[:, 0]] == [1.0, 2.0, 0.0]
    ds, dw = tsm.combine_tokens_backward(x, s, pos)
    assert [float(v) for v in ds[:, 0]] == [1.0, 0.0, 0.0, 2.0]
    assert (dw[2] == 0).all() and dw[0, 1] == 0 and dw[1, 0] == 0


def test_scales_without_elements():
    import torch

    say("[gpu] dispatch of scales alone")
    pos = torch.tensor([[2, 0], [-1, 1]], dtype=torch.int32, device="cuda")
    s = torch.tensor([5.0, 7.0], device="cuda")
    _, ss = tsm.dispatch_tokens(torch.empty((2, 0), device="cuda"), pos, slots=3, scale=s)
    assert ss.tolist() == [5.0, 7.0, 5.0]


def test_slabs_past_4_gib():
    """Slab rows whose byte offsets pass 2^32."""
    import torch

    rows, H = 300000, 8192
    say("[gpu] slabs past 4 GiB")
    slabs = torch.zeros((rows, H), dtype=torch.bfloat16, device="cuda")
    x = torch.randn((4, H), device="cuda").to(torch.bfloat16)
    pos = torch.tensor([[rows - 1], [0], [262144], [262143]], dtype=torch.int32, device="cuda")
    tsm.dispatch_tokens(x, pos, out=slabs)
    assert torch.equal(slabs[pos[:, 0].long()], x) and int((slabs != 0).any(1).sum()) == 4
    assert torch.equal(tsm.combine_tokens(slabs, pos), x)
    ds, dw = tsm.combine_tokens_backward(x, slabs, pos, out=torch.zeros_like(slabs))
    assert torch.equal(ds, slabs)
    assert torch.allclose(dw[:, 0].double(), (x.double() ** 2).sum(1), rtol=(H + 8) * 2.0 ** -24, atol=0)


def test_other_stream_needs_its_workspace():
    import torch

    ids = torch.zeros((5000, 2), dtype=torch.int32, device="cuda")
    side = torch.cuda.Stream()
    with pytest.raises(tsm.TsmError):
        tsm.sort_tokens(ids, 4, 10000, stream=side)
    say("[gpu] sort on a stream of its own")
    ws = tsm.sort_workspace_for(ids, 4)
    torch.cuda.synchronize()
    pos, counts = tsm.sort_tokens(ids, 4, 10000, workspace=ws, stream=side)
    side.synchronize()
    assert counts.tolist() == [10000, 0, 0, 0] and torch.equal(pos.view(-1).cpu(), torch.arange(10000, dtype=torch.int32))


def test_without_slab_rows():
    import torch

    say("[gpu] no slab rows")
    pos = torch.tensor([[0, 3], [1, -1]], dtype=torch.int32, device="cuda")
    empty = torch.empty((0, 40), device="cuda")
    assert (tsm.combine_tokens(empty, pos, torch.ones((2, 2), device="cuda")) == 0).all()
    ds, dw = tsm.combine_tokens_backward(torch.ones((2, 40), device="cuda"), empty, pos)
    assert ds.shape == (0, 40) and (dw == 0).all()
    assert tsm.dispatch_tokens(torch.ones((2, 40), device="cuda"), pos, slots=0).shape == (0, 40)
    none = torch.empty((3, 0), dtype=torch.int32, device="cuda")
    assert (tsm.combine_tokens(torch.ones((4, 40), device="cuda"), none) == 0).all()


def layer(x, ids, w, up, down, E, cap):
    """A 16-bit expert layer: sort, dispatch, two grouped products, combine."""
    import torch

    T, H = x.shape
    F = up.shape[1]
    pos, counts = tsm.sort_tokens(ids, E, cap)
    s = tsm.dispatch_tokens(x, pos, slots=E * cap)
    h = torch.empty((E * cap, F), dtype=x.dtype, device="cuda")
    tsm.gemm_grouped(cap, F, H, s, H, tsm.TSM_ROW, cap * H, up, H, tsm.TSM_COL, F * H, h, F, cap * F, counts, E,
                     tsm.TSM_BF16_BF16)
    o = torch.empty((E * cap, H), dtype=x.dtype, device="cuda")
    tsm.gemm_grouped(cap, H, F, h, F, tsm.TSM_ROW, cap * F, down, F, tsm.TSM_COL, H * F, o, H, cap * H, counts, E,
                     tsm.TSM_BF16_BF16)
    return tsm.combine_tokens(o, pos, w)


def layer_i8(x, ids, w, up, down, E, cap):
    """The same with int8 weights: tokens quantised once, their codes dispatched, hidden rows quantised in the slabs."""
    import torch

    (qu, su), (qd, sd) = up, down
    T, H = x.shape
    pos, counts = tsm.sort_tokens(ids, E, cap)
    q, s = tsm.quantize(x)
    slab, ss = tsm.dispatch_tokens(q, pos, slots=E * cap, scale=s)
    h = tsm.matmul_i8(slab.view(E, cap, H), ss.view(E, cap), qu.transpose(1, 2), su, rows=counts, activation="relu",
                      out_dtype=x.dtype)
    hq, hs = tsm.quantize(h, rows=counts)
    o = tsm.matmul_i8(hq, hs, qd.transpose(1, 2), sd, rows=counts, out_dtype=x.dtype)
    return tsm.combine_tokens(o.view(E * cap, H), pos, w)


@pytest.mark.parametrize("T,k,E,cap,H,F", [(1, 2, 8, 1, 256, 512), (100, 2, 8, 60, 256, 384), (700, 4, 16, 180, 130, 70)])
def test_expert_layer(T, k, E, cap, H, F):
    """The operators in a row, 16-bit and int8, eager and captured: the 16-bit layer against float64 within its
    roundings, the int8 one against the same steps in float64 from the codes."""
    import torch

    g = torch.Generator(device="cuda").manual_seed(T)
    rng = np.random.default_rng(T)
    x = torch.randn((T, H), generator=g, device="cuda").to(torch.bfloat16)
    ids = torch.from_numpy(np.stack([rng.permutation(E)[:k] for _ in range(T)])).cuda()
    w = torch.softmax(torch.randn((T, k), generator=g, device="cuda"), -1)
    up = (torch.randn((E, F, H), generator=g, device="cuda") / H ** 0.5).to(torch.bfloat16)
    down = (torch.randn((E, H, F), generator=g, device="cuda") / F ** 0.5).to(torch.bfloat16)
    say(f"[gpu] expert layer T={T} E={E}")
    y = layer(x, ids, w, up, down, E, cap)
    pos, _ = plain_sort(ids.cpu().numpy(), E, cap)
    ref = torch.zeros((T, H), dtype=torch.float64, device="cuda")
    mag = torch.zeros_like(ref)
    # per row: h = x U, o = h D, each sum's float32 roundings (H or F steps) and one bf16 rounding (2^-8 relative to
    # the value, bounded by the sum of magnitudes), the second product carrying the first's error
    for t in range(T):
        for j in range(k):
            if pos[t, j] < 0:
                continue
            e = int(ids[t, j])
            U, D = up[e].double(), down[e].double()
            h, o_mag = U @ x[t].double(), D.abs() @ (U.abs() @ x[t].double().abs())
            ref[t] += w[t, j].double() * (D @ h)
            mag[t] += w[t, j].double() * o_mag
    bound = mag * (2 * 2.0 ** -8 + (H + F + k + 4) * 2.0 ** -24) * 1.01
    assert ((y.double() - ref).abs() <= bound + ref.abs() * 2.0 ** -8 * 1.01).all()

    qup, qdown = tsm.quantize(up), tsm.quantize(down)
    y8 = layer_i8(x, ids, w, qup, qdown, E, cap)
    q, s = tsm.quantize(x)
    for t in range(0, T, max(1, T // 40)):
        acc = torch.zeros(H, dtype=torch.float64, device="cuda")
        mag = torch.zeros(H, dtype=torch.float64, device="cuda")
        for j in range(k):
            if pos[t, j] < 0:
                continue
            e = int(ids[t, j])
            h = tsm.matmul_i8(q[t:t + 1], s[t:t + 1], qup[0][e].t(), qup[1][e], activation="relu",
                              out_dtype=torch.bfloat16)
            hq, hs = tsm.quantize(h)
            o = (hq[0].double() @ qdown[0][e].double().t().contiguous()) * hs.double() * qdown[1][e].double()
            acc += w[t, j].double() * o
            mag += w[t, j].double() * o.abs()
        # three float32 roundings and a bf16 one per row, k in the sum, and the result's
        bound = mag * (2.0 ** -8 + (k + 4) * 2.0 ** -24) * 1.01 + acc.abs() * 2.0 ** -8 * 1.01
        assert ((y8[t].double() - acc).abs() <= bound).all()

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        layer(x, ids, w, up, down, E, cap)
        layer_i8(x, ids, w, qup, qdown, E, cap)
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        ya = layer(x, ids, w, up, down, E, cap)
        yb = layer_i8(x, ids, w, qup, qdown, E, cap)
    for i in range(3):
        x.copy_(torch.randn((T, H), generator=g, device="cuda").to(torch.bfloat16))
        ids.copy_(torch.from_numpy(np.stack([rng.permutation(E)[:k] for _ in range(T)])).cuda())
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(ya, layer(x, ids, w, up, down, E, cap))
        assert torch.equal(yb, layer_i8(x, ids, w, qup, qdown, E, cap))


@pytest.mark.parametrize("as_handle", [False, True], ids=["stream", "handle"])
def test_results_on_a_stream_of_their_own(as_handle):
    """Calls on a side stream that allocate their results, while the current stream is busy and then writes into blocks
    that it has given back to torch: every result is that of the same call on the current stream."""
    import torch

    g = torch.Generator(device="cuda").manual_seed(4)
    T, k, E, cap, H, N = 300, 2, 8, 90, 512, 256
    ids = torch.randint(0, E, (T, k), generator=g, device="cuda")
    x, dy = value((T, H), torch.float32, g), value((T, H), torch.float32, g)
    slab = value((E * cap, H), torch.float32, g)
    wt = torch.rand((T, k), generator=g, device="cuda")
    w = torch.randint(-128, 128, (N, H), generator=g, device="cuda", dtype=torch.int8)
    pos, _ = tsm.sort_tokens(ids, E, cap)
    q, s = tsm.quantize(x)
    held = torch.zeros(E * cap, dtype=torch.bool, device="cuda")
    held[pos[pos >= 0].long()] = True
    calls = {
        "quantize": lambda **kw: tsm.quantize(x, **kw),
        "matmul_i8": lambda **kw: (tsm.matmul_i8(q, s, w.t(), None, **kw),),
        "sort": lambda **kw: tsm.sort_tokens(ids, E, cap, **kw),
        "dispatch": lambda **kw: tuple(t[held] for t in tsm.dispatch_tokens(q, pos, slots=E * cap, scale=s, **kw)),
        "combine": lambda **kw: (tsm.combine_tokens(slab, pos, wt, **kw),),
        "dispatch gradient": lambda **kw: (tsm.dispatch_tokens_backward(slab, pos, **kw),),
        "combine gradients": lambda **kw: tsm.combine_tokens_backward(dy, slab, pos, wt, **kw)}
    big = torch.randn((4096, 4096), generator=g, device="cuda")
    side = torch.cuda.Stream()
    for name, call in calls.items():
        say(f"[gpu] {name} on a side stream")
        want = call()
        torch.cuda.synchronize()
        for _ in range(6):
            torch.mm(big, big)
        blocks = [torch.empty_like(t) for t in want for _ in range(4)]
        for b in blocks:
            b.fill_(77)
        del blocks, b
        if name == "dispatch":  # (its rows are picked on the stream, too)
            with torch.cuda.stream(side):
                got = call(stream=side.cuda_stream if as_handle else side)
        else:
            got = call(stream=side.cuda_stream if as_handle else side)
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(got, want)), name


@pytest.mark.parametrize("T,k", [(10, 3), (5000, 2), (137500, 8)])
def test_sort_without_experts(T, k):
    """No experts: every position is -1, however many workgroups the entries take."""
    import torch

    ids = torch.zeros((T, k), dtype=torch.int64, device="cuda")
    pos = torch.full((T + 1, k), 7, dtype=torch.int32, device="cuda")
    say(f"[gpu] sort {T}x{k} of no experts")
    _, counts = tsm.sort_tokens(ids, 0, 5, positions=pos[:T])
    assert counts.numel() == 0 and (pos[:T] == -1).all() and (pos[T] == 7).all()
