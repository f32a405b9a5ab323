"""Int8 products with scales and the row quantisation on the GPU, against float64.

Sums of int8 products are exact, so a float32 result acc * sa * sb carries three
roundings (the sum's conversion and two products), each at most 2^-24 relative;
a leaky ReLU adds one, a 16-bit output one of half a step of its format.  Codes
and scales of the quantisation are compared bit for bit.
"""

import numpy as np
import pytest

from gpu_util import say

import tiled_shared_memory_amd as tsm

pytestmark = pytest.mark.gpu

HALF_STEP = {"f32": 2.0 ** -24, "f16": 2.0 ** -11, "bf16": 2.0 ** -8}
TINY = {"f32": 0.0, "f16": 2.0 ** -25, "bf16": 0.0}  # half the spacing of f16 subnormals


def dtypes():
    import torch

    return {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}


def padded(rows, cols, ld, gen, lo=-128, hi=128):
    """An int8 (rows, cols) view with leading dimension ld, starting one byte into its buffer when ld is odd."""
    import torch

    off = ld % 2
    buf = torch.randint(lo, hi, (rows * ld + off,), generator=gen, device="cuda", dtype=torch.int8)
    return buf[off:].as_strided((rows, cols), (ld, 1)) if rows else buf.new_empty((0, cols))


def reference(a, sa, b, sb, act=None, slope=0.0):
    """float64 result from the codes (M, K), (N, K) and scales."""
    import torch

    c = torch.mm(a.double(), b.double().t().contiguous())  # exact: |sums| < 2^31
    c = c * (sa.double()[:, None] if sa is not None else 1.0) * (sb.double()[None, :] if sb is not None else 1.0)
    if act == "relu":
        c = c.clamp(min=0)
    elif act == "leaky_relu":
        c = torch.where(c > 0, c, c * float(np.float32(slope)))
    return c


def check(got, ref, out, roundings=3):
    import torch

    assert torch.isfinite(got).all()
    bound = ref.abs() * (roundings * 2.0 ** -24 * (1 + 2.0 ** -20))
    if out != "f32":
        bound = bound + (ref.abs() + bound) * HALF_STEP[out] + TINY[out]
    err = (got.double() - ref).abs()
    bad = err > bound
    assert not bad.any(), f"{int(bad.sum())} cells, first {bad.nonzero()[0].tolist()}: {float(err.max())}"


def scales(n, gen):
    import torch

    return torch.rand(n, generator=gen, device="cuda") * 0.02 + 1e-4


SHAPES = [  # M, N, K, lda - K, ldb - K, ldc - N
    (1, 1, 1, 0, 0, 0), (1, 8192, 8192, 0, 0, 0), (1, 130, 4096, 0, 0, 0), (1, 33, 15, 0, 0, 0), (3, 100, 17, 1, 2, 3),
    (16, 512, 2048, 0, 0, 0), (16, 1000, 777, 0, 0, 0), (7, 640, 1024, 16, 16, 0), (33, 65, 129, 0, 0, 0),
    (64, 128, 128, 0, 0, 0), (48, 4096, 512, 0, 0, 0), (100, 300, 4099, 5, 3, 1), (128, 256, 16384, 0, 0, 0),
    (256, 256, 8192, 0, 0, 0), (1000, 1500, 777, 0, 0, 0), (513, 770, 1024, 0, 0, 6), (2048, 2560, 1280, 0, 0, 0),
    (2300, 4104, 640, 16, 0, 8), (2049, 4090, 384, 0, 0, 0), (3000, 5000, 100, 0, 0, 0), (5, 70000, 64, 0, 0, 0),
    (70000, 5, 64, 0, 0, 0), (40, 40, 131071, 0, 0, 0)]


@pytest.mark.parametrize("shape", SHAPES, ids=lambda s: "x".join(map(str, s[:3])) + ("" if not any(s[3:]) else "_ld"))
@pytest.mark.parametrize("out", ["f32", "f16", "bf16"])
def test_product(shape, out):
    """Every kernel's shapes; C's padding and the rows behind it stay as they were."""
    import torch

    M, N, K, pa, pb, pc = shape
    g = torch.Generator(device="cuda").manual_seed(M * 7 + N * 3 + K)
    a, b = padded(M, K, K + pa, g), padded(N, K, K + pb, g)
    sa, sb = scales(M, g), scales(N, g) / K ** 0.5
    buf = torch.full((M + 1, N + pc), 77.0, dtype=dtypes()[out], device="cuda")
    c = buf[:M, :N]
    say(f"[gpu] i8 product {shape} {out} "
        f"{tsm.tsm_gemm_i8_kernel_name(M, N, K, a, K + pa, 0, b, K + pb, 0, c, N + pc, 0, 1, None, 0)}")
    tsm.matmul_i8(a, sa, b.t(), sb, out=c)
    check(c, reference(a, sa, b, sb), out)
    assert (buf[M] == 77.0).all() and (buf[:, N:] == 77.0).all()


@pytest.mark.parametrize("out", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("M,N,K,pad", [(256, 256, 128 * n, 0) for n in range(1, 15)]
                         + [(1, 8, 256, 0), (257, 264, 384, 16), (700, 520, 128, 32), (255, 1032, 1664, 0)])
def test_large_tiles(monkeypatch, M, N, K, pad, out):
    """The 256 x 256 kernel, forced: every count of slabs in and after its loop, ragged M and N, padded rows, an
    activation, a batch, and grouped counts."""
    import torch

    monkeypatch.setenv("TSM_GEMM_KERNEL", "i8_tile_256x256x128")
    g = torch.Generator(device="cuda").manual_seed(M + N + K)
    a, b = padded(M, K, K + pad, g), padded(N, K, K + pad, g)
    sa, sb = scales(M, g), scales(N, g) / K ** 0.5
    buf = torch.full((M + 1, N + 8), 77.0, dtype=dtypes()[out], device="cuda")
    say(f"[gpu] i8 large tiles {M}x{N}x{K} {out}")
    tsm.matmul_i8(a, sa, b.t(), sb, out=buf[:M, :N], activation="leaky_relu", slope=0.5)
    check(buf[:M, :N], reference(a, sa, b, sb, "leaky_relu", 0.5), out, 4)
    assert (buf[M] == 77.0).all() and (buf[:, N:] == 77.0).all()
    rows = torch.tensor([M, 0, M // 2, M + 5, 1], dtype=torch.int32, device="cuda")
    a3 = torch.randint(-128, 128, (5, M, K), generator=g, device="cuda", dtype=torch.int8)
    b3 = torch.randint(-128, 128, (5, N, K), generator=g, device="cuda", dtype=torch.int8)
    s3, t3 = scales((5, M), g), scales((5, N), g) / K ** 0.5
    plain = tsm.matmul_i8(a3, s3, b3.transpose(1, 2), t3, out_dtype=dtypes()[out])
    c = torch.full((5, M, N), 55.0, dtype=dtypes()[out], device="cuda")
    tsm.matmul_i8(a3, s3, b3.transpose(1, 2), t3, rows=rows, out=c)
    for z, m in enumerate([M, 0, M // 2, M, 1]):
        check(plain[z], reference(a3[z], s3[z], b3[z], t3[z]), out)
        assert torch.equal(c[z, :m], plain[z, :m]) and (c[z, m:] == 55.0).all()


@pytest.mark.parametrize("M,N,K", [(4352, 4096, 128), (4100, 4360, 256), (2200, 2304, 384)])
def test_tiles_past_whole_rounds(M, N, K):
    """A few 256-tiles more than one per CU (272, 306), or fewer than a round: the two launches together write every
    element once, plain and with a batch."""
    import torch

    g = torch.Generator(device="cuda").manual_seed(M)
    a, b = padded(M, K, K, g), padded(N, K, K, g)
    sa, sb = scales(M, g), scales(N, g) / K ** 0.5
    buf = torch.full((M + 1, N + 8), 77.0, dtype=torch.float16, device="cuda")
    say(f"[gpu] i8 tiles past whole rounds {M}x{N}x{K}")
    assert tsm.tsm_gemm_i8_kernel_name(M, N, K, a, K, 0, b, K, 0, buf, N + 8, 0, 1, None, 1) == "i8_tile_256x256x128"
    tsm.matmul_i8(a, sa, b.t(), sb, out=buf[:M, :N])
    check(buf[:M, :N], reference(a, sa, b, sb), "f16")
    assert (buf[M] == 77.0).all() and (buf[:, N:] == 77.0).all()


@pytest.mark.parametrize("rows", [[2048] * 4 + [100] * 2, [600, 0, 300, 1, 0, 0], [0] * 6, [2048, 2048, 2048, 2048, 257, 513],
                                  [2048] * 6])
def test_grouped_rounds(rows):
    """6 groups of up to 2048 rows, 2048 columns: 48 to 384 tiles of which the device leaves some to the second launch."""
    import torch

    M, N, K = 2048, 2048, 128
    g = torch.Generator(device="cuda").manual_seed(sum(rows))
    a = torch.randint(-128, 128, (6, M, K), generator=g, device="cuda", dtype=torch.int8)
    b = torch.randint(-128, 128, (6, N, K), generator=g, device="cuda", dtype=torch.int8)
    sa, sb = scales((6, M), g), scales((6, N), g)
    c = torch.full((6, M, N), 55.0, dtype=torch.bfloat16, device="cuda")
    r = torch.tensor(rows, dtype=torch.int32, device="cuda")
    say(f"[gpu] i8 grouped rounds {rows}")
    tsm.matmul_i8(a, sa, b.transpose(1, 2), sb, rows=r, out=c)
    for z, m in enumerate(rows):
        check(c[z, :m], reference(a[z, :m], sa[z, :m], b[z], sb[z]), "bf16")
        assert (c[z, m:] == 55.0).all()


@pytest.mark.parametrize("kernel", ["i8_skinny", "i8_stream"])
@pytest.mark.parametrize("M", [1, 3, 4, 5, 16, 17, 32, 33, 64])
@pytest.mark.parametrize("N,K", [(40, 16), (16, 256), (4200, 272), (20000, 1040), (100, 5120), (8208, 4112)])
def test_few_rows(monkeypatch, kernel, M, N, K):
    """The streaming and the register kernel on the same problems: K inside one step, in several, and past the ring;
    more columns than one round of workgroups holds; padded rows; a grouped call."""
    import torch

    monkeypatch.setenv("TSM_GEMM_KERNEL", kernel)
    g = torch.Generator(device="cuda").manual_seed(M + N + K)
    a, b = padded(M, K, K + 16, g), padded(N, K, K + 48, g)
    sa, sb = scales(M, g), scales(N, g) / K ** 0.5
    say(f"[gpu] {kernel} {M}x{N}x{K}")
    buf = torch.full((M + 1, N + 3), 77.0, dtype=torch.bfloat16, device="cuda")
    tsm.matmul_i8(a, sa, b.t(), sb, out=buf[:M, :N], activation="relu")
    check(buf[:M, :N], reference(a, sa, b, sb, "relu"), "bf16")
    assert (buf[M] == 77.0).all() and (buf[:, N:] == 77.0).all()
    if N > 5000:
        return
    rows = torch.tensor([0, M, 1, M // 2, -1, M + 1], dtype=torch.int32, device="cuda")
    a3 = torch.randint(-128, 128, (6, M, K), generator=g, device="cuda", dtype=torch.int8)
    b3 = torch.randint(-128, 128, (6, N, K), generator=g, device="cuda", dtype=torch.int8)
    c = torch.full((6, M, N), 55.0, device="cuda")
    tsm.matmul_i8(a3, None, b3.transpose(1, 2), None, rows=rows, out=c)
    for z, m in enumerate([0, M, 1, M // 2, 0, M]):
        check(c[z, :m], reference(a3[z, :m], None, b3[z], None), "f32")
        assert (c[z, m:] == 55.0).all()


@pytest.mark.parametrize("shape", [(1, 512, 512), (16, 300, 1000), (300, 200, 100), (2304, 2304, 512)])
@pytest.mark.parametrize("act", ["relu", "leaky_relu"])
def test_activation(shape, act):
    import torch

    M, N, K = shape
    g = torch.Generator(device="cuda").manual_seed(1)
    a, b = padded(M, K, K, g), padded(N, K, K, g)
    sa, sb = scales(M, g), scales(N, g)
    say(f"[gpu] i8 {act} {shape}")
    for out in ("f32", "bf16"):
        c = tsm.matmul_i8(a, sa, b.t(), sb, out_dtype=dtypes()[out], activation=act, slope=0.3)
        check(c, reference(a, sa, b, sb, act, 0.3), out, 4)


@pytest.mark.parametrize("shape", [(1, 64, 131071), (130, 140, 131071), (2304, 2304, 128)])
def test_extreme_codes_are_exact(shape):
    """All codes -128, without scales: sums of K * 16384, at K = 131071 the largest below 2^31."""
    import torch

    M, N, K = shape
    a = torch.full((M, K), -128, dtype=torch.int8, device="cuda")
    b = torch.full((N, K), -128, dtype=torch.int8, device="cuda")
    say(f"[gpu] i8 extremes {shape}")
    c = tsm.matmul_i8(a, None, b.t(), None)
    assert (c == float(np.float32(K * 16384))).all()


@pytest.mark.parametrize("M", [3, 20, 70, 2600])
def test_weights_past_4_gib(M):
    """A weight of 4.9e9 bytes: its last columns."""
    import torch

    N, K = (37600, 131056) if M < 100 else (37632, 130944)
    g = torch.Generator(device="cuda").manual_seed(M)
    b = torch.randint(-128, 128, (N, K), generator=g, device="cuda", dtype=torch.int8)
    a = torch.randint(-128, 128, (M, K), generator=g, device="cuda", dtype=torch.int8)
    sa, sb = scales(M, g), scales(N, g)
    say(f"[gpu] i8 weights past 4 GiB, {M} rows")
    c = tsm.matmul_i8(a, sa, b.t(), sb)
    for lo in (0, N - 100):
        check(c[:, lo:lo + 100], reference(a, sa, b[lo:lo + 100], sb[lo:lo + 100]), "f32")


def test_zero_k_and_scales_of_nan():
    import torch

    a = torch.zeros((3, 0), dtype=torch.int8, device="cuda")
    b = torch.zeros((5, 0), dtype=torch.int8, device="cuda")
    say("[gpu] i8 K = 0")
    assert (tsm.matmul_i8(a, torch.ones(3, device="cuda"), b.t(), None) == 0).all()
    for M in (2, 200):
        a = torch.ones((M, 40), dtype=torch.int8, device="cuda")
        b = torch.ones((70, 40), dtype=torch.int8, device="cuda")
        sa = torch.ones(M, device="cuda")
        sa[1] = float("nan")
        c = tsm.matmul_i8(a, sa, b.t(), None)
        assert torch.isnan(c[1]).all() and (c[0] == 40).all() and (c[2:] == 40).all()


@pytest.mark.parametrize("batch,M,N,K", [(3, 1, 256, 512), (5, 20, 130, 333), (4, 300, 260, 256), (9, 1024, 768, 512)])
def test_batches_and_broadcast(batch, M, N, K):
    import torch

    g = torch.Generator(device="cuda").manual_seed(3)
    a = torch.randint(-128, 128, (batch, M, K), generator=g, device="cuda", dtype=torch.int8)
    b = torch.randint(-128, 128, (batch, N, K), generator=g, device="cuda", dtype=torch.int8)
    sa, sb = scales((batch, M), g), scales((batch, N), g)
    say(f"[gpu] i8 batch {batch} {M}x{N}x{K}")
    c = tsm.matmul_i8(a, sa, b.transpose(1, 2), sb)
    d = tsm.matmul_i8(a, sa, b[:1].transpose(1, 2), sb[:1])  # one weight for all
    e = tsm.matmul_i8(a[0], sa[0], b.transpose(1, 2), sb)    # one token block for all
    for z in range(batch):
        check(c[z], reference(a[z], sa[z], b[z], sb[z]), "f32")
        check(d[z], reference(a[z], sa[z], b[0], sb[0]), "f32")
        check(e[z], reference(a[0], sa[0], b[z], sb[z]), "f32")


@pytest.mark.parametrize("M,N,K", [(8, 256, 512), (40, 130, 100), (300, 384, 256), (700, 1024, 512)])
def test_grouped(M, N, K):
    """Counts below zero, zero, one, odd, the capacity and above it; the other rows untouched and unread."""
    import torch

    rows = [M, 0, 1, -5, M + 9, M // 2 + 1, M - 1, 2] * 3
    G = len(rows)
    g = torch.Generator(device="cuda").manual_seed(M)
    x = torch.randn((G, M, K), generator=g, device="cuda", dtype=torch.float32).to(torch.bfloat16)
    w = torch.randint(-128, 128, (G, N, K), generator=g, device="cuda", dtype=torch.int8)
    sw = scales((G, N), g)
    r = torch.tensor(rows, dtype=torch.int32, device="cuda")
    held = [min(max(m, 0), M) for m in rows]
    for z, m in enumerate(held):
        x[z, m:] = float("nan")  # neither quantised nor multiplied
    say(f"[gpu] i8 grouped {M}x{N}x{K}")
    codes = torch.full((G, M, K), 99, dtype=torch.int8, device="cuda")
    sx = torch.full((G, M), 55.0, device="cuda")
    tsm.quantize(x, rows=r, out=codes, scale=sx)
    c = torch.full((G, M, N), float("nan"), device="cuda")
    tsm.matmul_i8(codes, sx, w.transpose(1, 2), sw, rows=r, out=c)
    for z, m in enumerate(held):
        assert (codes[z, m:] == 99).all() and (sx[z, m:] == 55.0).all()
        assert torch.isnan(c[z, m:]).all()
        check(c[z, :m], reference(codes[z, :m], sx[z, :m], w[z], sw[z]), "f32")


def plain_quantize(x):
    """float64: codes of the exact quotient, ties to even, and the float32 scales."""
    m = np.abs(x).max(axis=-1) if x.shape[-1] else np.zeros(x.shape[:-1])
    scale = (m.astype(np.float32) / np.float32(127)).astype(np.float32)
    with np.errstate(invalid="ignore", divide="ignore"):
        q = np.rint(127.0 * x / m[..., None])  # correctly rounded: distinct from a tie by more than 2^-25
    return np.where(m[..., None] > 0, q, 0.0).astype(np.int8), scale


@pytest.mark.parametrize("R,C", [(1, 1), (3, 7), (5, 64), (9, 512), (2, 513), (3, 777), (4, 2048), (2, 4100), (1, 8192),
                                 (2, 16384), (2, 16391), (1, 40000), (3000, 96)])
@pytest.mark.parametrize("fmt", ["f32", "f16", "bf16"])
def test_quantize(R, C, fmt):
    import torch

    g = torch.Generator(device="cuda").manual_seed(R + C)
    pad = 3 if C % 2 else 0
    buf = torch.randn((R, C + pad), generator=g, device="cuda").to(dtypes()[fmt])
    x = buf[:, :C]
    if C > 4:
        x[0, 1], x[0, 2], x[0, 3] = x[0].abs().max() * 2, x[0].abs().max() / 4, 0  # halves, quarters of the largest
    say(f"[gpu] quantize {R}x{C} {fmt}")
    qbuf = torch.full((R, C + 5), 77, dtype=torch.int8, device="cuda")
    q, s = tsm.quantize(x, out=qbuf[:, :C])
    ref_q, ref_s = plain_quantize(x.double().cpu().numpy())
    assert np.array_equal(s.cpu().numpy(), ref_s)
    assert np.array_equal(q.cpu().numpy(), ref_q)
    assert (qbuf[:, C:] == 77).all()


def test_quantize_borders():
    """Every tie n + 1/2 of a largest magnitude of 127 (x = n + 1/2), its float32 neighbours, and the same scaled to
    the ends of the range: the codes of the exact quotient."""
    import torch

    n = np.arange(0, 127, dtype=np.float32) + np.float32(0.5)
    row = np.concatenate([[127.0], n, -n, np.nextafter(n, np.float32(0)), np.nextafter(n, np.float32(200))])
    row = row.astype(np.float32)
    rows = [row, row * np.float32(2.0 ** 120), row * np.float32(2.0 ** -100), row * np.float32(2.0 ** -126),
            row * np.float32(3.0)]
    x = np.stack(rows)
    say("[gpu] quantize borders")
    q, s = tsm.quantize(torch.from_numpy(x).cuda())
    ref_q, ref_s = plain_quantize(x.astype(np.float64))
    assert np.array_equal(s.cpu().numpy(), ref_s)
    assert np.array_equal(q.cpu().numpy(), ref_q)


@pytest.mark.parametrize("fmt", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("C", [40, 3000, 20000])
def test_quantize_zeros_and_non_finite(fmt, C):
    import torch

    x = torch.ones((5, C), dtype=dtypes()[fmt], device="cuda")
    x[0] = 0
    x[1, C - 1] = float("nan")
    x[2, C // 2] = float("inf")
    x[3, 0] = float("-inf")
    x[3, 1] = float("nan")
    say(f"[gpu] quantize non-finite {fmt} {C}")
    q, s = tsm.quantize(x)
    assert s[0] == 0 and (q[:4] == 0).all() and torch.isnan(s[1:4]).all()
    assert (q[4] == 127).all() and s[4] == np.float32(1) / np.float32(127)


def test_quantize_empty_and_repeated_rows():
    import torch

    say("[gpu] quantize empty")
    q, s = tsm.quantize(torch.ones((4, 0), device="cuda"))
    assert q.shape == (4, 0) and (s == 0).all()
    q, s = tsm.quantize(torch.ones((0, 8), device="cuda"))
    assert q.shape == (0, 8)
    x = torch.arange(1, 9, device="cuda", dtype=torch.float32)
    q, s = tsm.quantize(x.expand(3, 8))
    assert (q == q[0]).all() and q[0, 7] == 127


def test_linear_layer_on_a_side_stream_and_replayed():
    """quantize + matmul_i8 captured into a graph and replayed on new inputs, against eager calls."""
    import torch

    g = torch.Generator(device="cuda").manual_seed(5)
    for M in (1, 16, 300):
        w = torch.randint(-128, 128, (512, 1024), generator=g, device="cuda", dtype=torch.int8)
        sw = scales(512, g)
        x = torch.randn((M, 1024), generator=g, device="cuda")
        q = torch.empty((M, 1024), dtype=torch.int8, device="cuda")
        s = torch.empty(M, device="cuda")
        c = torch.empty((M, 512), device="cuda")
        say(f"[gpu] i8 linear captured M={M}")
        side = torch.cuda.Stream()
        side.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(side):
            tsm.quantize(x, out=q, scale=s)
            tsm.matmul_i8(q, s, w.t(), sw, out=c)
        torch.cuda.current_stream().wait_stream(side)
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            tsm.quantize(x, out=q, scale=s)
            tsm.matmul_i8(q, s, w.t(), sw, out=c)
        for i in range(4):
            x.copy_(torch.randn((M, 1024), generator=g, device="cuda") * (i + 1))
            graph.replay()
            torch.cuda.synchronize()
            eq, es = tsm.quantize(x)
            e = tsm.matmul_i8(eq, es, w.t(), sw)
            assert torch.equal(q, eq) and torch.equal(s, es) and torch.equal(c, e)


@pytest.mark.parametrize("out", ["f32", "bf16"])
@pytest.mark.parametrize("M,N,K,pad", [
    (33, 12304, 1040, 0), (64, 14000, 272, 16), (16, 4096, 2047, 0), (9, 8200, 1023, 3), (40, 520, 4096, 0),
    (128, 200, 4224, 0), (65, 136, 4352, 1), (50, 100, 4480 + 77, 0), (100, 70, 8191, 0), (65, 18500, 256, 0),
    (128, 32700, 128, 0)])
def test_borders_of_the_selection(M, N, K, pad, out):
    """Few rows of many columns on 64-tiles, odd addresses, every phase of the deeper loop, 128-tiles half as wide as
    a 256-tile; plain, as two batches, and grouped."""
    import torch

    g = torch.Generator(device="cuda").manual_seed(M + N + K)
    a, b = padded(M, K, K + pad, g), padded(N, K, K + pad, g)
    sa, sb = scales(M, g), scales(N, g) / K ** 0.5
    say(f"[gpu] i8 borders {M}x{N}x{K} {out}")
    buf = torch.full((M + 1, N + 3), 77.0, dtype=dtypes()[out], device="cuda")
    tsm.matmul_i8(a, sa, b.t(), sb, out=buf[:M, :N])
    check(buf[:M, :N], reference(a, sa, b, sb), out)
    assert (buf[M] == 77.0).all() and (buf[:, N:] == 77.0).all()
    a2 = torch.randint(-128, 128, (2, M, K), generator=g, device="cuda", dtype=torch.int8)
    b2 = torch.stack([b, b.flip(0)])
    s2 = scales((2, M), g)
    plain = tsm.matmul_i8(a2, s2, b2.transpose(1, 2), None, out_dtype=dtypes()[out])
    c = torch.full((2, M, N), 55.0, dtype=dtypes()[out], device="cuda")
    tsm.matmul_i8(a2, s2, b2.transpose(1, 2), None, rows=torch.tensor([M - 1, M + 9], dtype=torch.int32, device="cuda"),
                  out=c)
    for z, m in enumerate([M - 1, M]):
        check(plain[z], reference(a2[z], s2[z], b2[z], None), out)
        assert torch.equal(c[z, :m], plain[z, :m]) and (c[z, m:] == 55.0).all()


@pytest.mark.parametrize("act", ["relu", "leaky_relu"])
@pytest.mark.parametrize("kernel,M,N,K", [("i8_skinny", 4, 40, 272), ("i8_stream", 20, 130, 272),
                                          ("i8_block_64x64x128", 70, 100, 133), ("i8_block_128x128x128", 150, 140, 256),
                                          ("i8_tile_256x256x128", 300, 264, 256)])
@pytest.mark.parametrize("out", ["f32", "bf16"])
def test_nan_scales_pass_the_activation(monkeypatch, kernel, act, M, N, K, out):
    """A token (or channel) whose scale is NaN gives NaN results with an activation too, in every kernel; the others
    are as they were."""
    import torch

    monkeypatch.setenv("TSM_GEMM_KERNEL", kernel)
    g = torch.Generator(device="cuda").manual_seed(M)
    a, b = padded(M, K, (K + 15) // 16 * 16, g), padded(N, K, (K + 15) // 16 * 16, g)
    sa, sb = scales(M, g), scales(N, g)
    sa[1], sb[N - 2] = float("nan"), float("nan")
    say(f"[gpu] {kernel} {act} of NaN scales {out}")
    c = tsm.matmul_i8(a, sa, b.t(), sb, out_dtype=dtypes()[out], activation=act, slope=0.5)
    rows = torch.arange(M, device="cuda") != 1
    cols = torch.arange(N, device="cuda") != N - 2
    assert torch.isnan(c[~rows]).all() and torch.isnan(c[:, ~cols]).all()
    check(c[rows][:, cols], reference(a[rows], sa[rows], b[cols], sb[cols], act, 0.5), out, 4)


def test_a_token_of_nan_shows_in_an_expert_layers_hidden_rows():
    """quantize, product with ReLU, quantize, product: the token's result is NaN, its neighbours' are not."""
    import torch

    g = torch.Generator(device="cuda").manual_seed(3)
    x = torch.randn((5, 96), generator=g, device="cuda")
    x[2, 7] = float("nan")
    up, down = (tsm.quantize(torch.randn(s, generator=g, device="cuda")) for s in ((128, 96), (96, 128)))
    say("[gpu] i8 layer of a NaN token")
    h = tsm.matmul_i8(*tsm.quantize(x), up[0].t(), up[1], activation="relu", out_dtype=torch.bfloat16)
    y = tsm.matmul_i8(*tsm.quantize(h), down[0].t(), down[1])
    bad = torch.isnan(y)
    assert bad[2].all() and not bad[[0, 1, 3, 4]].any()


def many_counts(G, M, kind):
    """Row counts of G groups: mixed ones, long runs of empty groups, or the last group alone."""
    rng = np.random.default_rng(G + M)
    if kind == "last":
        rows = np.zeros(G, np.int64)
        rows[-1] = M
        return rows
    rows = rng.choice([0, 1, M // 2, M - 1, M, M + 3, -2], G)
    if kind == "runs":
        for z in range(0, G, 64):
            if z // 64 % 2 == 0:
                rows[z:z + 64] = 0  # whole trips of the search over 64 counts without a row
        rows[-1] = max(1, M // 3)
    return rows


@pytest.mark.parametrize("kind", ["mixed", "runs", "last"])
@pytest.mark.parametrize("G", [65, 200, 513, 600])
@pytest.mark.parametrize("kernel,M,N,K", [
    ("i8_stream", 3, 40, 272), ("i8_stream", 16, 100, 528), ("i8_stream", 20, 40, 272), ("i8_stream", 40, 72, 272),
    ("i8_skinny", 5, 40, 100), ("i8_block_64x64x128", 70, 72, 133), ("i8_block_128x128x128", 130, 136, 133),
    ("i8_tile_256x256x128", 260, 264, 128), (None, 130, 264, 128)], ids=str)
def test_many_groups(monkeypatch, kernel, M, N, K, G, kind):
    """More groups than one trip of the search over the counts (64), than the streaming kernel takes in a launch (512),
    and (without a forced kernel) the 256-tiles with their second launch; rows past the counts untouched."""
    import torch

    if kernel:
        monkeypatch.setenv("TSM_GEMM_KERNEL", kernel)
    rows = many_counts(G, M, kind)
    g = torch.Generator(device="cuda").manual_seed(G + M)
    a = torch.randint(-128, 128, (G, M, K), generator=g, device="cuda", dtype=torch.int8)
    b = torch.randint(-128, 128, (G, N, K), generator=g, device="cuda", dtype=torch.int8)
    sa, sb = scales((G, M), g), scales((G, N), g)
    r = torch.from_numpy(rows.astype(np.int32)).cuda()
    c = torch.full((G, M, N), 55.0, dtype=torch.float16, device="cuda")
    name = tsm.tsm_gemm_i8_kernel_name(M, N, K, a, K, M * K, b, K, N * K, c, N, M * N, G, r, 1)
    say(f"[gpu] i8 {G} groups {kind} {M}x{N}x{K} {name}")
    assert name == (kernel or "i8_tile_256x256x128")
    tsm.matmul_i8(a, sa, b.transpose(1, 2), sb, rows=r, out=c)
    held = torch.arange(M, device="cuda")[None, :] < r[:, None]
    ref = torch.bmm(a.double(), b.double().transpose(1, 2).contiguous()) * sa.double()[..., None] * sb.double()[:, None]
    check(c[held], ref[held], "f16")
    assert (c[~held] == 55.0).all()
