"""Microscaled 4-bit quantisation and products on the GPU, against float64.

Codes, scales and values are compared bit for bit.  Products of two elements are
exact, so a product carries the roundings of its float32 sums: at most K of them,
each 2^-24 of the sum of magnitudes; a leaky ReLU adds one, a 16-bit output half
a step of its format.
"""

import math

import pytest

import mx4_ref as ref
from gpu_util import say
from mx4_ref import check_product, dtypes

import tiled_shared_memory_amd as tsm

pytestmark = pytest.mark.gpu


def gen(seed):
    import torch

    return torch.Generator(device="cuda").manual_seed(seed)


def strided(rows, cols, ld, fill=0xFF, dtype=None):
    """A (rows, cols) view with leading dimension ld, one element into its buffer when ld is odd; and the buffer."""
    import torch

    off = ld % 2
    buf = torch.full((rows * ld + off + 16,), fill, dtype=dtype or torch.uint8, device="cuda")
    return buf[off:].as_strided((rows, cols), (ld, 1)), buf


def operand(rows, C, pad_q, pad_s, g, lo=118, hi=134):
    """Random codes and scales of rows of C elements in rows with padding, whatever lies behind them 0xff (scales of
    NaN, odd half bytes that do not count); and their values."""
    import torch

    kb, nb = (C + 1) // 2, (C + 31) // 32
    q, _ = strided(rows, kb, kb + pad_q)
    s, _ = strided(rows, nb, nb + pad_s)
    q.copy_(torch.randint(0, 256, (rows, kb), generator=g, device="cuda", dtype=torch.uint8))
    s.copy_(torch.randint(lo, hi, (rows, nb), generator=g, device="cuda", dtype=torch.uint8))
    return q, s, ref.values(q, s, C)


# ---- quantisation ---------------------------------------------------------------------------------------------


def special(rows, C, dtype, g):
    """Values over the whole range: ties, blocks of zeros, of subnormals, of the largest, of NaN and infinities."""
    import torch

    x = torch.randn((rows, C), generator=g, device="cuda")
    kind = torch.randint(0, 8, (rows, (C + 31) // 32), generator=g, device="cuda").repeat_interleave(32, -1)[:, :C]
    grid = torch.tensor([0, 0.125, 0.25, 0.375, 0.5, 0.75, 1.25, 1.75, 2.5, 3.5, 5, 5.5, 6, 7, 7.5], device="cuda")
    ties = grid[torch.randint(0, 15, (rows, C), generator=g, device="cuda")] * torch.sign(x)
    x = torch.where(kind == 1, ties, x)
    x = torch.where(kind == 2, 0.0 * x, x)
    top = torch.finfo(dtype).max
    x = torch.where(kind == 3, (x.clamp(-1, 1) * 0.99).double() * top, x.double())
    x = torch.where(kind == 4, x * torch.finfo(dtype).smallest_normal, x)
    x = torch.where((kind == 5) & (torch.rand(x.shape, generator=g, device="cuda") < 0.03), math.nan, x)
    x = torch.where((kind == 6) & (torch.rand(x.shape, generator=g, device="cuda") < 0.03), -math.inf, x)
    return x.to(dtype)


QUANT_SHAPES = [(1, 1), (1, 32), (3, 31), (5, 33), (64, 100), (17, 777), (65, 256), (2, 4096), (300, 1027), (9, 8200),
                (129, 64), (1, 40000), (4097, 40)]


@pytest.mark.parametrize("R,C", QUANT_SHAPES)
@pytest.mark.parametrize("fmt", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("turned", [False, True], ids=["rows", "columns"])
def test_quantize(R, C, fmt, turned):
    """Codes and scales bit for bit, in rows of any alignment whose padding stays as it was."""
    import torch

    g = gen(R * 3 + C)
    say(f"[gpu] quantize_mx4 {R}x{C} {fmt} {'columns' if turned else 'rows'}")
    x = special(R, C, dtypes()[fmt], g)
    if turned:
        store, _ = strided(C, R, R + 3, 0, x.dtype)
        store.copy_(x.t())
        x = store.t()
    else:
        store, _ = strided(R, C, C + 5, 0, x.dtype)
        store.copy_(x)
        x = store
    q, qbuf = strided(R, (C + 1) // 2, (C + 1) // 2 + 3, 0xA5)
    s, sbuf = strided(R, (C + 31) // 32, (C + 31) // 32 + 2, 0x5A)
    q0, s0 = qbuf.clone(), sbuf.clone()
    tsm.quantize_mx4(x, out=q, scale=s)
    code, e = ref.quantize(x)
    assert torch.equal(s.long(), e)
    assert torch.equal(q, ref.pack(code))
    q.fill_(0xA5)
    s.fill_(0x5A)
    assert torch.equal(qbuf, q0) and torch.equal(sbuf, s0)


def test_quantize_groups_and_counts():
    """Only the rows below each count are read (the others hold NaN) and written, in both layouts."""
    import torch

    g = gen(5)
    G, R, C = 5, 70, 200
    rows = torch.tensor([70, 0, 1, 65, 90], dtype=torch.int32, device="cuda")
    held = torch.arange(R, device="cuda")[None, :] < rows[:, None]
    x = torch.where(held[..., None], torch.randn((G, R, C), generator=g, device="cuda"), math.nan)
    code, e = ref.quantize(x)
    for turned in (False, True):
        v = x.transpose(1, 2).contiguous().transpose(1, 2) if turned else x
        q = torch.full((G, R, C // 2), 7, dtype=torch.uint8, device="cuda")
        s = torch.full((G, R, 7), 9, dtype=torch.uint8, device="cuda")
        say(f"[gpu] quantize_mx4 groups turned={turned}")
        tsm.quantize_mx4(v, rows=rows, out=q, scale=s)
        assert torch.equal(q[held], ref.pack(code)[held]) and torch.equal(s[held].long(), e[held])
        assert (q[~held] == 7).all() and (s[~held] == 9).all()
        y = torch.full((G, R, C), 3.0, device="cuda")
        tsm.dequantize_mx4(q, s, rows=rows, out=y)
        assert torch.equal(y[held].double(), ref.values(q[held], s[held], C)) and (y[~held] == 3.0).all()


@pytest.mark.parametrize("fmt", ["f32", "f16", "bf16"])
def test_dequantize_every_code_and_scale(fmt):
    """Every code in every place with every scale, rounded once."""
    import torch

    q = torch.arange(256, dtype=torch.uint8, device="cuda").repeat(16)[:256 * 16].reshape(1, -1)
    q = q.expand(256, -1).contiguous()  # 8192 elements a row
    s = torch.arange(256, dtype=torch.uint8, device="cuda")[:, None].expand(-1, 256).contiguous()
    say(f"[gpu] dequantize_mx4 every scale {fmt}")
    y = tsm.dequantize_mx4(q, s, out_dtype=dtypes()[fmt])
    want = ref.values(q, s, 8192).to(dtypes()[fmt])
    assert torch.equal(torch.isnan(y), torch.isnan(want))
    assert torch.equal(torch.nan_to_num(y), torch.nan_to_num(want))
    assert torch.equal(torch.signbit(y[:255]), torch.signbit(want[:255]))


@pytest.mark.parametrize("R,C", [(1, 1), (3, 31), (33, 777), (5, 8191), (70, 64)])
@pytest.mark.parametrize("fmt", ["f32", "f16", "bf16"])
def test_round_trip(R, C, fmt):
    """Back to values, in rows with padding; quantising them again changes nothing."""
    import torch

    g = gen(R + C)
    say(f"[gpu] mx4 round trip {R}x{C} {fmt}")
    x = torch.randn((R, C), generator=g, device="cuda").to(dtypes()[fmt])
    q, s = tsm.quantize_mx4(x)
    y, buf = strided(R, C, C + 3, 3.0, x.dtype)
    before = buf.clone()
    tsm.dequantize_mx4(q, s, out=y)
    assert torch.equal(y.double(), ref.values(q, s, C))
    again, s2 = tsm.quantize_mx4(y)
    assert torch.equal(tsm.dequantize_mx4(again, s2, columns=C).double(), y.double())
    y.fill_(3.0)
    assert torch.equal(buf, before)


# ---- products -------------------------------------------------------------------------------------------------

SHAPES = [  # M, N, K, padding of codes' and scales' rows, ldc - N
    (1, 1, 1, 0, 0, 0), (1, 8192, 8192, 0, 0, 0), (1, 130, 4096, 0, 0, 0), (1, 33, 15, 0, 0, 0), (3, 100, 17, 1, 2, 3),
    (16, 512, 2048, 0, 0, 0), (16, 1000, 777, 0, 0, 0), (7, 640, 1024, 16, 16, 0), (33, 65, 129, 3, 1, 0),
    (64, 128, 128, 0, 0, 0), (48, 4096, 512, 0, 0, 0), (100, 300, 4099, 5, 3, 1), (128, 256, 16384, 0, 0, 0),
    (256, 256, 8192, 0, 0, 0), (1000, 1500, 777, 0, 0, 0), (513, 770, 1024, 0, 0, 6), (2048, 2560, 1280, 0, 0, 0),
    (2300, 4104, 640, 16, 4, 8), (2049, 4090, 256, 0, 0, 0), (3000, 5000, 100, 0, 0, 0), (5, 70000, 64, 0, 0, 0),
    (70000, 5, 64, 0, 0, 0), (40, 40, 100001, 0, 0, 0), (17, 33, 255, 0, 0, 0), (64, 64, 257, 7, 5, 0)]


@pytest.mark.parametrize("shape", SHAPES, ids=lambda s: "x".join(map(str, s[:3])) + ("" if not any(s[3:]) else "_ld"))
@pytest.mark.parametrize("out", ["f32", "f16", "bf16"])
def test_product(shape, out):
    """Every kernel's shapes; what lies behind the operands' rows does not count, C's padding stays as it was."""
    import torch

    M, N, K, pq, ps, pc = shape
    g = gen(M * 7 + N * 3 + K)
    a, sa, va = operand(M, K, pq, ps, g)
    b, sb, vb = operand(N, K, pq, ps, g, 112, 124)
    buf = torch.full((M + 1, N + pc), 77.0, dtype=dtypes()[out], device="cuda")
    c = buf[:M, :N]
    name = tsm.tsm_gemm_mx4_kernel_name(M, N, K, a, a.shape[1] + pq, 0, sa, sa.shape[1] + ps, 0, b, b.shape[1] + pq, 0,
                                        sb, sb.shape[1] + ps, 0, c, N + pc, 0, 1, None, 0)
    say(f"[gpu] mx4 product {shape} {out} {name}")
    tsm.gemm_mx4(M, N, K, a, a.shape[1] + pq, sa, sa.shape[1] + ps, b, b.shape[1] + pq, sb, sb.shape[1] + ps, c, N + pc,
                 {"f32": tsm.TSM_F32, "f16": tsm.TSM_F16, "bf16": tsm.TSM_BF16}[out])
    check_product(c, *ref.product(va, vb), K, out)
    assert (buf[M] == 77.0).all() and (buf[:, N:] == 77.0).all()


@pytest.mark.parametrize("out", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("M,N,K,pad", [(256, 256, 256 * n, 0) for n in range(1, 28)]
                         + [(1, 8, 256, 0), (257, 264, 768, 16), (700, 520, 256, 32), (255, 1032, 3328, 0)])
def test_large_tiles(monkeypatch, M, N, K, pad, out):
    """The 256 x 256 kernel, forced: every count of slabs in and after its loop, ragged M and N, padded rows, an
    activation, a batch, and grouped counts."""
    import torch

    monkeypatch.setenv("TSM_GEMM_KERNEL", "mx4_tile_256x256x256")
    g = gen(M + N + K)
    dt = dtypes()[out]
    a, sa, va = operand(M, K, pad, pad // 4, g)
    b, sb, vb = operand(N, K, pad, pad // 4, g, 112, 124)
    buf = torch.full((M + 1, N + 8), 77.0, dtype=dt, device="cuda")
    say(f"[gpu] mx4 large tiles {M}x{N}x{K} {out}")
    tsm.matmul_mx4(a, sa, b.t(), sb, out=buf[:M, :N], activation="leaky_relu", slope=0.5)
    check_product(buf[:M, :N], *ref.product(va, vb, "leaky_relu", 0.5), K, out, 2.0 ** -24)
    assert (buf[M] == 77.0).all() and (buf[:, N:] == 77.0).all()
    a3, sa3, va3 = (t.reshape(5, M, -1) for t in operand(5 * M, K, 0, 0, g))
    b3, sb3, vb3 = (t.reshape(5, N, -1) for t in operand(5 * N, K, 0, 0, g, 112, 124))
    plain = tsm.matmul_mx4(a3, sa3, b3.transpose(1, 2), sb3, out_dtype=dt)
    rows = torch.tensor([M, 0, M // 2, M + 5, 1], dtype=torch.int32, device="cuda")
    c = torch.full((5, M, N), 55.0, dtype=dt, device="cuda")
    tsm.matmul_mx4(a3, sa3, b3.transpose(1, 2), sb3, rows=rows, out=c)
    for z, m in enumerate([M, 0, M // 2, M, 1]):
        check_product(plain[z], *ref.product(va3[z], vb3[z]), K, out)
        assert torch.equal(c[z, :m], plain[z, :m]) and (c[z, m:] == 55.0).all()


@pytest.mark.parametrize("out", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("M,N,K,pad", [(300, 520, 128 * n, 0) for n in range(1, 29)]
                         + [(257, 513, 640, 0), (513, 257, 1152, 1), (256, 1001, 128, 3), (700, 262, 4224, 2),
                            (255, 255, 256, 1), (511, 300, 384, 4)])
def test_large_tiles_of_half_slabs_and_odd_columns(monkeypatch, M, N, K, pad, out):
    """A last slab of half its elements; results whose rows, or their first element, are not at 16 bytes; scales of NaN
    and codes behind the operands' rows."""
    import torch

    monkeypatch.setenv("TSM_GEMM_KERNEL", "mx4_tile_256x256x256")
    g = gen(M + N * 3 + K + pad)
    say(f"[gpu] mx4 large tiles {M}x{N}x{K}+{pad} {out}")
    a, sa, va = operand(M, K, 16 * (pad % 2), 4 * (pad % 2), g)
    b, sb, vb = operand(N, K, 32 * (pad % 2), 8 * (pad % 2), g, 112, 124)
    buf = torch.full(((M + 1) * (N + pad) + 1,), 77.0, dtype=dtypes()[out], device="cuda")
    c = buf[pad % 2:].as_strided((M, N), (N + pad, 1))
    tsm.matmul_mx4(a, sa, b.t(), sb, columns=K, out=c)
    check_product(c, *ref.product(va, vb), K, out)
    c.fill_(77.0)
    assert (buf == 77.0).all()


@pytest.mark.parametrize("out", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("M,N,K,pad", [(130, 200, 128 * n, 0) for n in range(1, 20)]
                         + [(1, 1, 128, 0), (64, 64, 256, 0), (65, 127, 1152, 1), (129, 257, 4224, 1), (1000, 70, 640, 1)])
@pytest.mark.parametrize("T", [64, 128])
def test_middle_tiles(monkeypatch, T, M, N, K, pad, out):
    """The kernels with a ring of copies, forced: every count of slabs in and after a turn of the ring, a last one of
    half its elements, ragged M and N, results at odd addresses, a batch and grouped counts; scales of NaN and codes
    behind the operands' rows."""
    import torch

    monkeypatch.setenv("TSM_GEMM_KERNEL", f"mx4_ring_{T}x{T}x256")
    g = gen(M + N * 3 + K + T)
    dt = dtypes()[out]
    say(f"[gpu] mx4 middle tiles {T} {M}x{N}x{K}+{pad} {out}")
    a, sa, va = operand(M, K, 16 * pad, 4 * pad, g)
    b, sb, vb = operand(N, K, 48 * pad, 8 * pad, g, 112, 124)
    buf = torch.full(((M + 1) * (N + 3 * pad) + 1,), 77.0, dtype=dt, device="cuda")
    c = buf[pad:].as_strided((M, N), (N + 3 * pad, 1))
    tsm.matmul_mx4(a, sa, b.t(), sb, out=c, activation="leaky_relu", slope=0.25)
    check_product(c, *ref.product(va, vb, "leaky_relu", 0.25), K, out, 2.0 ** -24)
    c.fill_(77.0)
    assert (buf == 77.0).all()
    if (M, T) == (130, 64):  # enough tiles for the shorter ring
        M, N = 700, 520
    a3, sa3, _ = (t.reshape(5, M, -1) for t in operand(5 * M, K, 0, 0, g))
    b3, sb3, _ = (t.reshape(5, N, -1) for t in operand(5 * N, K, 0, 0, g, 112, 124))
    plain = tsm.matmul_mx4(a3, sa3, b3.transpose(1, 2), sb3, out_dtype=dt)
    for z in range(5):
        check_product(plain[z], *ref.product(ref.values(a3[z], sa3[z], K), ref.values(b3[z], sb3[z], K)), K, out)
    rows = torch.tensor([M, 0, M // 2, M + 5, -1], dtype=torch.int32, device="cuda")
    c = torch.full((5, M, N), 55.0, dtype=dt, device="cuda")
    tsm.matmul_mx4(a3, sa3, b3.transpose(1, 2), sb3, rows=rows, out=c)
    for z, m in enumerate([M, 0, M // 2, M, 0]):
        assert torch.equal(c[z, :m], plain[z, :m]) and (c[z, m:] == 55.0).all()


@pytest.mark.parametrize("out", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("M,N,K,pq,ps", [(1, 1, 1, 0, 0), (3, 70, 2, 1, 1), (65, 5, 31, 0, 3), (64, 64, 32, 2, 0),
                                         (10, 129, 33, 3, 2), (130, 7, 255, 0, 0), (70, 200, 256, 1, 1),
                                         (129, 65, 257, 2, 3), (33, 300, 511, 5, 0), (200, 100, 513, 0, 1),
                                         (257, 130, 769, 1, 2), (64, 128, 1000, 0, 0), (66, 67, 1023, 3, 1),
                                         (100, 31, 1281, 2, 2), (140, 260, 2047, 1, 0), (1, 500, 4097, 0, 3),
                                         (300, 33, 3333, 7, 5), (128, 64, 8190, 0, 0), (40, 40, 10001, 1, 1)])
@pytest.mark.parametrize("T", [64, 128])
def test_odd_rows(monkeypatch, T, M, N, K, pq, ps, out):
    """The general kernel, forced: rows at any address, K that ends anywhere in a slab, a batch and grouped counts;
    scales of NaN, and codes, behind the rows and in an odd K's last half byte."""
    import torch

    monkeypatch.setenv("TSM_GEMM_KERNEL", f"mx4_block_{T}x{T}x256")
    g = gen(M + N * 3 + K + T)
    dt = dtypes()[out]
    say(f"[gpu] mx4 odd rows {T} {M}x{N}x{K}+{pq},{ps} {out}")
    a, sa, va = operand(M, K, pq, ps, g)
    b, sb, vb = operand(N, K, pq + 1, ps + 2, g, 112, 124)
    buf = torch.full((M + 1, N + 3), 77.0, dtype=dt, device="cuda")
    tsm.matmul_mx4(a, sa, b.t(), sb, columns=K, out=buf[:M, :N], activation="leaky_relu", slope=0.25)
    check_product(buf[:M, :N], *ref.product(va, vb, "leaky_relu", 0.25), K, out, 2.0 ** -24)
    assert (buf[M] == 77.0).all() and (buf[:, N:] == 77.0).all()
    a3, sa3, va3 = (t.reshape(5, M, -1) for t in operand(5 * M, K, 0, 0, g))
    b3, sb3, vb3 = (t.reshape(5, N, -1) for t in operand(5 * N, K, 0, 0, g, 112, 124))
    plain = tsm.matmul_mx4(a3, sa3, b3.transpose(1, 2), sb3, columns=K, out_dtype=dt)
    for z in range(5):
        check_product(plain[z], *ref.product(va3[z], vb3[z]), K, out)
    rows = torch.tensor([M, 0, M // 2, M + 5, -1], dtype=torch.int32, device="cuda")
    c = torch.full((5, M, N), 55.0, dtype=dt, device="cuda")
    tsm.matmul_mx4(a3, sa3, b3.transpose(1, 2), sb3, columns=K, rows=rows, out=c)
    for z, m in enumerate([M, 0, M // 2, M, 0]):
        assert torch.equal(c[z, :m], plain[z, :m]) and (c[z, m:] == 55.0).all()


@pytest.mark.parametrize("M,N,K", [(4352, 4096, 256), (4100, 4360, 512), (2200, 2304, 768)])
def test_tiles_past_whole_rounds(M, N, K):
    """A few 256-tiles more than one per CU (272, 306), or fewer than a round: the two launches together write every
    element once."""
    import torch

    g = gen(M)
    a, sa, va = operand(M, K, 0, 0, g)
    b, sb, vb = operand(N, K, 0, 0, g, 112, 124)
    buf = torch.full((M + 1, N + 8), 77.0, dtype=torch.float16, device="cuda")
    say(f"[gpu] mx4 tiles past whole rounds {M}x{N}x{K}")
    assert tsm.tsm_gemm_mx4_kernel_name(M, N, K, a, K // 2, 0, sa, K // 32, 0, b, K // 2, 0, sb, K // 32, 0, buf, N + 8,
                                        0, 1, None, 1) == "mx4_tile_256x256x256"
    tsm.matmul_mx4(a, sa, b.t(), sb, out=buf[:M, :N])
    check_product(buf[:M, :N], *ref.product(va, vb), K, "f16")
    assert (buf[M] == 77.0).all() and (buf[:, N:] == 77.0).all()


@pytest.mark.parametrize("act", [None, "relu", "leaky_relu"])
@pytest.mark.parametrize("M,N,K", [(5, 200, 512), (64, 512, 4096), (300, 520, 777), (2304, 2304, 512)])
def test_nan_blocks_and_activations(M, N, K, act):
    """A block of scale 255 makes its row (column) NaN with every activation, whatever its codes; others are sound."""
    import torch

    g = gen(M + K)
    a, sa, _ = operand(M, K, 0, 0, g)
    b, sb, _ = operand(N, K, 0, 0, g, 112, 124)
    sa[M // 2, -1] = 255
    sb[N - 1, 0] = 255
    a[M // 2] = 0  # codes of 0, as the quantisation leaves them
    say(f"[gpu] mx4 NaN blocks {M}x{N}x{K} {act}")
    c = tsm.matmul_mx4(a, sa, b.t(), sb, columns=K, activation=act, slope=-0.5)
    want, mag = ref.product(ref.values(a, sa, K), ref.values(b, sb, K), act, -0.5)
    bad = torch.isnan(want)
    assert bad[M // 2].all() and bad[:, N - 1].all() and int(bad.sum()) == M + N - 1
    assert torch.equal(torch.isnan(c), bad)
    check_product(c[~bad], want[~bad], mag[~bad], K, "f32", 2.0 ** -24)


def test_scales_at_the_ends_of_their_range():
    """Scales whose product passes float32's range on either side: infinities where the sum is one, no NaN."""
    import torch

    g = gen(3)
    for lo, hi in ((0, 3), (250, 255), (0, 255), (60, 190)):
        a, sa, va = operand(40, 512, 0, 0, g, lo, hi)
        b, sb, vb = operand(64, 512, 0, 0, g, lo, hi)
        say(f"[gpu] mx4 scales {lo}..{hi}")
        c = tsm.matmul_mx4(a, sa, b.t(), sb)
        want, mag = ref.product(va, vb)
        ok = mag < 2.0 ** 127
        assert not torch.isnan(c[ok]).any()
        check_product(c[ok], want[ok], mag[ok], 512, "f32")
        far = want.abs() > 2.0 ** 129
        assert not torch.isfinite(c[far]).any()


@pytest.mark.parametrize("M,N,K", [(1, 64, 512), (16, 256, 1024), (40, 100, 333), (128, 512, 256), (600, 512, 768)])
def test_batches_and_groups(M, N, K):
    """Strided batches, a shared operand either side, and counts: rows past them are neither read nor written."""
    import torch

    g = gen(M + N + K)
    G = 5
    a, sa, va = operand(G * M, K, 0, 0, g)
    b, sb, vb = operand(G * N, K, 0, 0, g, 112, 124)
    a3, sa3, va3 = (t.reshape(G, M, -1) for t in (a, sa, va))
    b3, sb3, vb3 = (t.reshape(G, N, -1) for t in (b, sb, vb))
    say(f"[gpu] mx4 batches {M}x{N}x{K}")
    plain = tsm.matmul_mx4(a3, sa3, b3.transpose(1, 2), sb3, columns=K)
    for z in range(G):
        check_product(plain[z], *ref.product(va3[z], vb3[z]), K, "f32")
    shared_b = tsm.matmul_mx4(a3, sa3, b3[0].t(), sb3[0], columns=K)
    shared_a = tsm.matmul_mx4(a3[0], sa3[0], b3.transpose(1, 2), sb3, columns=K)
    for z in range(G):
        check_product(shared_b[z], *ref.product(va3[z], vb3[0]), K, "f32")
        check_product(shared_a[z], *ref.product(va3[0], vb3[z]), K, "f32")
    counts = [M, 0, (M + 1) // 2, M + 5, -1]
    rows = torch.tensor(counts, dtype=torch.int32, device="cuda")
    stale = torch.arange(M, device="cuda")[None, :] >= rows[:, None]
    sa3 = torch.where(stale[..., None], 255, sa3.long()).to(torch.uint8)  # scales of NaN where nothing may be read
    c = torch.full((G, M, N), 55.0, device="cuda")
    tsm.matmul_mx4(a3, sa3, b3.transpose(1, 2), sb3, columns=K, rows=rows, out=c)
    assert torch.equal(c[~stale], plain[~stale]) and (c[stale] == 55.0).all()


@pytest.mark.parametrize("fmt", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("M,N,K", [(1, 300, 4096), (1, 64, 33), (5, 100, 777), (16, 512, 2048), (64, 256, 512),
                                   (500, 512, 1024)])
def test_product_of_activations(M, N, K, fmt):
    """Activations quantised within the call: the products of their codes, with and without a workspace, in a batch,
    with a shared operand and with counts."""
    import torch

    g = gen(M + N + K)
    x = torch.randn((3, M, K), generator=g, device="cuda").to(dtypes()[fmt])
    w, ws = tsm.quantize_mx4(torch.randn((3, N, K), generator=g, device="cuda"))
    say(f"[gpu] mx4 product of activations {M}x{N}x{K} {fmt}")
    q, s = tsm.quantize_mx4(x)
    # the codes in rows that the call would use: the same kernel multiplies them
    want = torch.stack([tsm.matmul_mx4(x[z], None, w[z].t(), ws[z]) for z in range(3)])
    for z in range(3):
        check_product(want[z], *ref.product(ref.values(q[z], s[z], K), ref.values(w[z], ws[z], K)), K, "f32")
    got = tsm.matmul_mx4(x, None, w.transpose(1, 2), ws, workspace=tsm.mx4_workspace_for(x))
    for z in range(3):
        check_product(got[z], *ref.product(ref.values(q[z], s[z], K), ref.values(w[z], ws[z], K)), K, "f32")
    shared = tsm.matmul_mx4(x[0], None, w.transpose(1, 2), ws)
    for z in range(3):
        check_product(shared[z], *ref.product(ref.values(q[0], s[0], K), ref.values(w[z], ws[z], K)), K, "f32")
    counts = [M, 0, (M + 1) // 2]
    rows = torch.tensor(counts, dtype=torch.int32, device="cuda")
    stale = torch.arange(M, device="cuda")[None, :] >= rows[:, None]
    c = torch.full((3, M, N), 55.0, device="cuda")
    tsm.matmul_mx4(torch.where(stale[..., None], math.nan, x), None, w.transpose(1, 2), ws, rows=rows, out=c)
    for z, m in enumerate(counts):
        check_product(c[z, :m], *ref.product(ref.values(q[z, :m], s[z, :m], K), ref.values(w[z], ws[z], K)), K, "f32")
        assert (c[z, m:] == 55.0).all()


@pytest.mark.parametrize("fmt", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("K,pad", [(128, 0), (640, 3), (4096, 0), (8192, 8), (8320, 0), (16384, 1), (16512, 0)])
@pytest.mark.parametrize("M", [1, 2, 3])
def test_activations_of_few_rows(M, K, pad, fmt):
    """Activations in padded rows with NaN behind them, blocks of NaN, zeros and infinities among theirs; more columns
    than the kernels hold at once, an odd number of them; counts that leave rows as they are."""
    import torch

    g = gen(M * 31 + K)
    N = 16 * 512 * 2 + 37
    say(f"[gpu] mx4 activations of few rows {M}x{N}x{K}+{pad} {fmt}")
    x, _ = strided(M, K, K + pad, math.nan, dtypes()[fmt])
    x.copy_(torch.randn((M, K), generator=g, device="cuda"))
    x[:, 32:64] = 0
    w, ws = tsm.quantize_mx4(torch.randn((N, K), generator=g, device="cuda"))
    vw = ref.values(w, ws, K)
    for rows in (None, *range(M + 1)):
        if rows == M:
            x[0, 96 + K // 256 * 7] = math.nan
        if rows == 0 and M == 2:
            x[1, 5] = math.inf
        m = M if rows is None else rows
        count = None if rows is None else torch.tensor([rows], dtype=torch.int32, device="cuda")
        c = torch.full((1, M, N), 55.0, device="cuda", dtype=dtypes()[fmt])
        tsm.matmul_mx4(x[None], None, w[None].transpose(1, 2), ws[None], rows=count, out=c)
        assert (c[:, m:] == 55.0).all()
        if m:
            q, s = tsm.quantize_mx4(x[:m])
            want, mag = ref.product(ref.values(q, s, K), vw)
            nan = want.isnan()
            assert torch.equal(c[0, :m].isnan(), nan)
            check_product(c[0, :m].masked_fill(nan, 0), want.masked_fill(nan, 0), mag.masked_fill(nan, 0), K, fmt)


@pytest.mark.parametrize("out", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("M,N,K,pad", [(1, 16, 128, 0), (7, 33, 1024, 1), (15, 4099, 1152, 0), (16, 20011, 2048, 0),
                                       (16, 16400, 4224, 1), (17, 32, 1024, 0), (31, 10001, 1152, 1),
                                       (32, 4100, 8320, 0), (33, 31, 128, 1), (48, 9000, 1280, 0), (63, 1, 4096, 0),
                                       (64, 8193, 640, 1)])
def test_few_rows(monkeypatch, M, N, K, pad, out):
    """The streaming kernel, forced: every width of its tiles, more tiles than workgroups, rows that end inside a tile,
    K that ends inside a step or a turn of the ring; codes and scales of NaN behind the operands' rows."""
    import torch

    monkeypatch.setenv("TSM_GEMM_KERNEL", "mx4_stream")
    g = gen(M * 5 + N + K)
    say(f"[gpu] mx4 few rows {M}x{N}x{K}+{pad} {out}")
    a, sa, va = operand(M, K, 16 * pad, 4 * pad, g)
    b, sb, vb = operand(N, K, 48 * pad, 8 * pad, g, 112, 124)
    buf = torch.full((M + 1, N + 3 * pad), 77.0, dtype=dtypes()[out], device="cuda")
    tsm.matmul_mx4(a, sa, b.t(), sb, out=buf[:M, :N], activation="relu")
    check_product(buf[:M, :N], *ref.product(va, vb, "relu"), K, out)
    assert (buf[M] == 77.0).all() and (buf[:, N:] == 77.0).all()


@pytest.mark.parametrize("G,M,N,K", [(1, 4, 70, 256), (65, 5, 40, 384), (600, 3, 48, 256), (1100, 1, 16, 128),
                                     (70, 20, 64, 1152), (9, 64, 100, 2048)])
def test_few_rows_in_many_groups(G, M, N, K):
    """Groups in several launches of the streaming kernel, many of them without rows, counts below 0 and above M, rows
    past the counts left as they are; and the same problems as a batch."""
    import torch

    g = gen(G + M)
    say(f"[gpu] mx4 few rows in {G} groups {M}x{N}x{K}")
    a, sa, va = (t.reshape(G, M, -1) for t in operand(G * M, K, 0, 0, g))
    b, sb, vb = (t.reshape(G, N, -1) for t in operand(G * N, K, 0, 0, g, 112, 124))
    plain = tsm.matmul_mx4(a, sa, b.transpose(1, 2), sb)
    assert tsm.tsm_gemm_mx4_kernel_name(M, N, K, a, K // 2, M * K // 2, sa, K // 32, M * K // 32, b, K // 2,
                                        N * K // 2, sb, K // 32, N * K // 32, plain, N, M * N, G, None,
                                        0) == "mx4_stream"
    for z in range(G):
        check_product(plain[z], *ref.product(va[z], vb[z]), K, "f32")
    for share in (0.0, 0.3, 1.0):
        n = torch.randint(-1, M + 2, (G,), generator=g, device="cuda", dtype=torch.int32)
        rows = torch.where(torch.rand(G, generator=g, device="cuda") < share, n, 0).to(torch.int32)
        c = torch.full((G, M, N), 55.0, device="cuda")
        tsm.matmul_mx4(a, sa, b.transpose(1, 2), sb, rows=rows, out=c)
        own = torch.arange(M, device="cuda")[None, :] < rows[:, None]
        assert torch.equal(c[own], plain[own]) and (c[~own] == 55.0).all()


@pytest.mark.parametrize("G,M,N,K", [(2, 1, 300, 1024), (5, 1, 64, 512), (3, 7, 130, 640), (40, 16, 256, 256),
                                     (9, 5, 33, 77)])
def test_a_weight_that_problems_share(G, M, N, K):
    """Problems of one weight, whose rows follow each other or not: codes and activations, padded, with counts, and
    one matrix of activations for all."""
    import torch

    g = gen(G * M + N)
    say(f"[gpu] mx4 shared weight {G} {M}x{N}x{K}")
    kb, nb = (K + 1) // 2, (K + 31) // 32
    a, sa, va = operand(G * M, K, 0, 0, g)
    b, sb, vb = operand(N, K, 0, 0, g, 112, 124)
    want, mag = ref.product(va, vb)
    far = torch.full((G, M + 1, kb + 16), 0xFF, dtype=torch.uint8, device="cuda")
    far[:, :M, :kb] = a.view(G, M, kb)
    far_s = torch.full((G, M + 2, nb + 4), 0xFF, dtype=torch.uint8, device="cuda")
    far_s[:, :M, :nb] = sa.view(G, M, nb)
    buf = torch.full((G, M + 1, N + 5), 77.0, device="cuda")
    for q in (a.view(G, M, kb), far[:, :M, :kb]):
        for s in (sa.view(G, M, nb), far_s[:, :M, :nb]):
            for c in (torch.full((G, M, N), 9.0, device="cuda"), buf[:, :M, :N]):
                c.fill_(9.0)
                tsm.matmul_mx4(q, s, b.t(), sb, columns=K, out=c)
                check_product(c.reshape(G * M, N), want, mag, K, "f32")
    assert (buf[:, M] == 77.0).all() and (buf[:, :, N:] == 77.0).all()
    rows = torch.tensor([M - 1] + [M] * (G - 1), dtype=torch.int32, device="cuda")
    c = torch.full((G, M, N), 55.0, device="cuda")
    tsm.matmul_mx4(a.view(G, M, kb), sa.view(G, M, nb), b.t(), sb, columns=K, rows=rows, out=c)
    assert (c[0, M - 1] == 55.0).all()
    own = torch.arange(M, device="cuda")[None, :] < rows[:, None]
    check_product(c[own], want[own.view(-1)], mag[own.view(-1)], K, "f32")
    x = torch.randn((G, M + 1, K + 3), generator=g, device="cuda")
    for v in (x[:, :M, :K].contiguous(), x[:, :M, :K], x[:1, :M, :K].expand(G, M, K)):
        want, mag = ref.product(ref.values(*tsm.quantize_mx4(v.reshape(G * M, K)), K), vb)
        check_product(tsm.matmul_mx4(v, None, b.t(), sb).view(G * M, N), want, mag, K, "f32")


def test_two_calls_at_once():
    """Calls on two streams at once, of one weight, each with its own workspace, and quantisations beside them."""
    import torch

    g = gen(21)
    N, K = 4096, 4096
    w, ws = tsm.quantize_mx4(torch.randn((N, K), generator=g, device="cuda"))
    xs = [torch.randn((m, K), generator=g, device="cuda") for m in (2, 300, 700, 1)]
    say("[gpu] mx4 two calls at once")
    want = [tsm.matmul_mx4(x, None, w.t(), ws) for x in xs]
    codes = [tsm.quantize_mx4(x) for x in xs]
    rooms = [tsm.mx4_workspace_for(x) for x in xs]
    outs = [torch.empty_like(t) for t in want]
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    torch.cuda.synchronize()
    got = []
    for turn in range(6):
        for i, x in enumerate(xs):
            tsm.matmul_mx4(x, None, w.t(), ws, out=outs[i], workspace=rooms[i], stream=streams[i % 2])
            got.append((i, tsm.quantize_mx4(x, stream=streams[(i + 1) % 2])))
    torch.cuda.synchronize()
    for o, t in zip(outs, want):
        assert torch.equal(o, t)
    for i, (q, s) in got:
        assert torch.equal(q, codes[i][0]) and torch.equal(s, codes[i][1])


def test_empty_sums_and_sizes():
    import torch

    a, b = torch.empty((3, 0), dtype=torch.uint8, device="cuda"), torch.empty((0, 5), dtype=torch.uint8, device="cuda")
    s, t = torch.empty((3, 0), dtype=torch.uint8, device="cuda"), torch.empty((5, 0), dtype=torch.uint8, device="cuda")
    say("[gpu] mx4 empty")
    c = torch.full((3, 5), 9.0, device="cuda")
    assert (tsm.matmul_mx4(a, s, b, t, out=c) == 0).all()
    c.fill_(9.0)
    assert (tsm.matmul_mx4(torch.empty((3, 0), device="cuda"), None, b, t, out=c) == 0).all()
    q, e = tsm.quantize_mx4(torch.empty((0, 40), device="cuda"))
    assert q.shape == (0, 20) and e.shape == (0, 2)
    assert tsm.matmul_mx4(q, e, b.new_empty((20, 5)).t().contiguous().t(), t.new_empty((5, 2))).shape == (0, 5)


def test_operands_past_4_gib():
    """Codes, scales, results and activations whose offsets pass 32 bits."""
    import torch

    g = gen(8)
    K, N, M = 256, 64, 96
    step = (1 << 32) + 4096
    say("[gpu] mx4 operands past 4 GiB")
    big = torch.zeros(step + (1 << 20), dtype=torch.uint8, device="cuda")

    def far(rows, cols):
        return big.as_strided((2, rows, cols), (step, cols, 1))

    b, sb = tsm.quantize_mx4(torch.randn((2, N, K), generator=g, device="cuda"))
    x = torch.randn((2, M, K), generator=g, device="cuda")
    a, sa = tsm.quantize_mx4(x)
    want = tsm.matmul_mx4(a, sa, b.transpose(1, 2), sb)
    for what, t in (("b", b), ("sb", sb), ("a", a), ("sa", sa)):
        v = far(t.shape[1], t.shape[2])
        v.copy_(t)
        p = {"a": a, "sa": sa, "b": b, "sb": sb, what: v}
        assert torch.equal(tsm.matmul_mx4(p["a"], p["sa"], p["b"].transpose(1, 2), p["sb"]), want), what
    c = big.view(torch.float32).as_strided((2, M, N), (step // 4, N, 1))
    tsm.matmul_mx4(a, sa, b.transpose(1, 2), sb, out=c)
    assert torch.equal(c, want)
    xs = big.view(torch.float32).as_strided((2, M, K), (step // 4, K, 1))
    xs.copy_(x)
    q, s = tsm.quantize_mx4(xs)
    assert torch.equal(q, a) and torch.equal(s, sa)
    # rows that lie a GiB apart
    wide = big.as_strided((3, K // 2), (step // 3 // 16 * 16, 1))
    wide.copy_(a[0, :3])
    assert torch.equal(tsm.matmul_mx4(wide, sa[0, :3].contiguous(), b[0].t(), sb[0]),
                       tsm.matmul_mx4(a[0, :3].contiguous(), sa[0, :3].contiguous(), b[0].t(), sb[0]))


def test_calls_on_another_stream_and_captured():
    """On a stream of their own, with the memory that they allocate there; captured, and replayed over new inputs."""
    import torch

    g = gen(11)
    M, N, K = 24, 512, 1024
    w, ws = tsm.quantize_mx4(torch.randn((N, K), generator=g, device="cuda"))
    x = torch.randn((M, K), generator=g, device="cuda")
    want = tsm.matmul_mx4(x, None, w.t(), ws)
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    say("[gpu] mx4 streams")
    busy = torch.randn((4096, 4096), device="cuda")
    for _ in range(8):
        busy = busy @ busy * 1e-3  # the current stream is busy; the side stream does not wait for it
    got = tsm.matmul_mx4(x, None, w.t(), ws, stream=side)
    q, s = tsm.quantize_mx4(x, stream=side)
    y = tsm.dequantize_mx4(q, s, stream=side)
    side.synchronize()
    assert torch.equal(got, want) and torch.equal(y.double(), ref.values(q, s, K))
    torch.cuda.synchronize()
    room, c = tsm.mx4_workspace_for(x), torch.empty((M, N), device="cuda")
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        tsm.matmul_mx4(x, None, w.t(), ws, out=c, workspace=room)
    for k in range(4):
        x.copy_(torch.randn((M, K), generator=g, device="cuda"))
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(c, tsm.matmul_mx4(x, None, w.t(), ws)), k
