"""Refusals of the microscaled 4-bit and router entry points: host-side checks, no GPU needed."""

import contextlib
import math

import pytest

import tiled_shared_memory_amd as tsm

# fake, suitably aligned device addresses: never dereferenced by these calls
A0, B0, C0, SA0, SB0, W0, P0 = (0x7F0000000000 + i * 0x1000000000 for i in range(7))


def refused(fn, kw, status, needle):
    with pytest.raises(tsm.TsmError) as ei:
        fn(**kw)
    assert ei.value.status == status
    assert needle in ei.value.detail


def gemm(**kw):
    a = dict(M=64, N=128, K=128, A=A0, lda=64, sA=0, sa=SA0, ldsa=4, ssa=0, B=B0, ldb=64, sB=0, sb=SB0, ldsb=4, ssb=0,
             C=C0, ldc=128, sC=0, batch=1, dt=0, act=0, slope=0.0)
    a.update(kw)
    return tsm.gemm_mx4_strided_batched(a["M"], a["N"], a["K"], a["A"], a["lda"], a["sA"], a["sa"], a["ldsa"], a["ssa"],
                                        a["B"], a["ldb"], a["sB"], a["sb"], a["ldsb"], a["ssb"], a["C"], a["ldc"],
                                        a["sC"], a["batch"], a["dt"], a["act"], a["slope"], 0)


@pytest.mark.parametrize("kw,status,needle", [
    (dict(M=-1), 1, "negative size"), (dict(K=-1), 1, "negative size"), (dict(batch=-1), 1, "negative batch"),
    (dict(dt=3), 1, "out_dtype"), (dict(act=3), 1, "activation"), (dict(act=2, slope=math.inf), 1, "slope"),
    (dict(A=0), 1, "A is NULL"), (dict(B=0), 1, "B is NULL"), (dict(sa=0), 1, "scale_a is NULL"),
    (dict(sb=0), 1, "scale_b is NULL"), (dict(C=0), 1, "C is NULL"), (dict(C=C0 + 2), 1, "aligned"),
    (dict(lda=63), 1, "lda=63"), (dict(K=127, lda=63), 1, "lda=63"), (dict(ldb=63), 1, "ldb=63"),
    (dict(ldsa=3), 1, "ld_sa=3"), (dict(K=129, lda=65, ldb=65), 1, "ld_sa=4"), (dict(ldsb=3), 1, "ld_sb=3"),
    (dict(ldc=127), 1, "ldc"), (dict(C=A0 + 2048), 1, "overlaps A"), (dict(C=B0), 1, "overlaps B"),
    (dict(C=SA0 + 64), 1, "overlaps scale_a"), (dict(sb=C0 + 64), 1, "overlaps scale_b"),
    (dict(batch=2, sC=1), 1, "strideC"), (dict(batch=2, sC=64 * 128, ssb=-1), 1, "negative stride"),
    (dict(M=1 << 31), 2, "2^31"), (dict(K=1 << 31, lda=1 << 30, ldb=1 << 30), 2, "2^31"),
    (dict(M=(1 << 31) - 1, N=(1 << 31) - 1, ldc=(1 << 31) - 1, C=1 << 62), 2, "overflows"),
    (dict(batch=1 << 40, sA=1 << 40, sB=1 << 40, sC=1 << 40), 2, "overflows")])
def test_gemm_refusals(kw, status, needle):
    refused(gemm, kw, status, needle)


@pytest.mark.parametrize("kw", [dict(M=0), dict(N=0), dict(batch=0), dict(M=0, A=0, B=0, C=0)])
def test_gemm_empty(kw):
    assert gemm(**kw) == 0


@pytest.mark.parametrize("rows,needle", [(0, "rows is NULL"), (P0 + 2, "rows not 4-byte")])
def test_gemm_grouped_needs_counts(rows, needle):
    with pytest.raises(tsm.TsmError) as ei:
        tsm.gemm_mx4_grouped(64, 128, 128, A0, 64, 4096, SA0, 4, 256, B0, 64, 8192, SB0, 4, 512, C0, 128, 64 * 128,
                             rows, 2, 0, 0, 0.0, 0)
    assert needle in ei.value.detail


def test_an_unknown_variant_is_refused(monkeypatch):
    monkeypatch.setenv("TSM_GEMM_KERNEL", "mx4_nothing")
    refused(gemm, {}, 1, "mx4_nothing")


BLOCK64, BLOCK128, RING64, RING128, TILE, STREAM = (
    "mx4_block_64x64x256", "mx4_block_128x128x256", "mx4_ring_64x64x256", "mx4_ring_128x128x256",
    "mx4_tile_256x256x256", "mx4_stream")


def name_of(M, N, K, batch=1, lda=None, ldb=None, a=1 << 20, fmt=tsm.TSM_BF16, ldc=None, lds=None, rows=None,
            shared=False):
    kb, nb = (K + 1) // 2, (K + 31) // 32
    lda, ldb, lds, ldc = lda or kb, ldb or kb, lds or nb, ldc or N
    return tsm.tsm_gemm_mx4_kernel_name(M, N, K, a, lda, M * lda, 1 << 21, lds, M * lds, 1 << 22, ldb, 0 if shared else N * ldb,
                                        1 << 23, lds, 0 if shared else N * lds, 1 << 45, ldc, M * ldc, batch, rows, fmt)


@pytest.mark.parametrize("M,N,K,kw,want", [
    (1, 8192, 8192, {}, STREAM), (32, 128000, 4096, {}, STREAM), (33, 8192, 8192, {}, STREAM),
    (64, 8192, 8192, {}, STREAM), (64, 8256, 8192, {}, RING64), (64, 512, 8192, dict(batch=16), STREAM),
    (64, 512, 8192, dict(batch=17), RING64), (16, 64, 128, dict(batch=600, rows=1 << 24), STREAM),
    (16, 8192, 8160, {}, BLOCK64), (16, 8192, 8192, dict(a=(1 << 20) + 8), BLOCK64),
    (16, 8192, 8192, dict(lda=4104), BLOCK64), (16, 8192, 8192, dict(lds=258), BLOCK64),
    (65, 8192, 8192, {}, RING64), (1024, 2048, 4096, {}, RING64), (1025, 2048, 4096, {}, RING128),
    (1024, 2048, 4064, {}, BLOCK64), (1025, 2048, 4096, dict(lds=130), BLOCK128), (65, 8192, 8192, dict(a=1048577), BLOCK64),
    (2048, 2048, 4096, {}, RING128), (2049, 2048, 4096, {}, TILE), (256, 16384, 4096, {}, RING128),
    (257, 16384, 4096, {}, TILE), (2304, 2048, 4224, {}, TILE), (2304, 2048, 4097, {}, BLOCK128),
    (2304, 2047, 4096, dict(ldc=2051), TILE), (2304, 2048, 4096, dict(lda=2056), BLOCK128),
    (256, 256, 4096, dict(batch=65), TILE), (256, 256, 4096, dict(batch=64), RING128),
    (1 << 21, 1 << 12, 256, {}, TILE), (2304, 2048, 4096, dict(lda=1 << 22), TILE),  # 255 * 2^22 + 2048 bytes are below 2^30
    (2304, 2048, 4096, dict(lda=1 << 23), BLOCK128),
    (2304, 2048, 4096, dict(ldc=1 << 23), BLOCK128), (5, 2**29, 256, {}, BLOCK128),
    (1, 4096, 4096, dict(batch=65, shared=True), RING64), (1, 4096, 4096, dict(batch=64, shared=True), STREAM),
    (16, 4096, 4096, dict(batch=256, shared=True), TILE), (16, 4096, 4096, dict(batch=256), STREAM),
    (16, 64, 128, dict(batch=600, rows=1 << 24, shared=True), STREAM),
    (5, 2**31 - 1, 256, {}, None)])  # more tiles than a grid may have work-items
def test_variants(M, N, K, kw, want):
    """Which kernel multiplies what: few rows, the borders of the tiles' sizes, what the large tiles and the streaming
    kernel need, and that nothing needs more than the general kernels."""
    assert name_of(M, N, K, **kw) == want


@pytest.mark.parametrize("name,M,N,K,kw", [
    (STREAM, 65, 512, 512, {}), (STREAM, 16, 512, 520, {}), (STREAM, 16, 512, 512, dict(lda=264)),
    (RING64, 300, 300, 320, {}), (RING128, 300, 300, 512, dict(ldb=1 << 23)), (RING128, 30, 30, 512, dict(lds=18)),
    (TILE, 300, 300, 320, {}), (TILE, 300, 300, 512, dict(lds=18)), (TILE, 300, 300, 512, dict(a=(1 << 20) + 4)),
    (TILE, 300, 300, 512, dict(ldb=1 << 23))])
def test_a_variant_that_cannot_run_the_problem_is_refused(monkeypatch, name, M, N, K, kw):
    assert name_of(M, N, K, **kw) is not None
    monkeypatch.setenv("TSM_GEMM_KERNEL", name)
    assert name_of(M, N, K, **kw) is None
    assert "cannot run" in tsm.tsm_last_error_detail()
    monkeypatch.setenv("TSM_GEMM_KERNEL", BLOCK128)
    assert name_of(M, N, K, **kw) == BLOCK128


def float_a(**kw):
    a = dict(M=64, N=128, K=128, X=A0, ldx=128, sX=0, xdt=2, B=B0, ldb=64, sB=0, sb=SB0, ldsb=4, ssb=0, C=C0, ldc=128,
             sC=0, batch=1, rows=None, dt=0, act=0, ws=W0, wsb=1 << 20)
    a.update(kw)
    return tsm.gemm_mx4_float_a(a["M"], a["N"], a["K"], a["X"], a["ldx"], a["sX"], a["xdt"], a["B"], a["ldb"], a["sB"],
                                a["sb"], a["ldsb"], a["ssb"], a["C"], a["ldc"], a["sC"], a["batch"], a["rows"], a["dt"],
                                a["act"], 0.0, a["ws"], a["wsb"], 0)


@pytest.mark.parametrize("kw,status,needle", [
    (dict(xdt=3), 1, "xdtype"), (dict(X=0), 1, "X is NULL"), (dict(X=A0 + 1), 1, "X not"), (dict(ldx=-1), 1, "ldx"),
    (dict(ws=0), 1, "workspace is NULL"), (dict(ws=W0 + 8), 1, "workspace not"), (dict(wsb=100), 1, "needed"),
    (dict(wsb=-1), 1, "workspace_bytes"), (dict(ws=A0 + 256), 1, "workspace overlaps X"),
    (dict(ws=C0 + 256), 1, "workspace overlaps C"), (dict(ws=B0), 1, "workspace overlaps B"),
    (dict(ws=SB0), 1, "workspace overlaps scale_b"), (dict(C=A0), 1, "C overlaps X"), (dict(B=0), 1, "B is NULL"),
    (dict(ldb=63), 1, "ldb"), (dict(rows=P0 + 1), 1, "rows"), (dict(batch=2, sC=1 << 20, sX=-4), 1, "negative stride"),
    (dict(dt=4), 1, "out_dtype")])
def test_float_a_refusals(kw, status, needle):
    refused(float_a, kw, status, needle)


def test_float_a_workspace_sizes():
    """Rows of codes in multiples of 16 bytes, of scales in multiples of 4."""
    f = tsm.gemm_mx4_float_a_workspace_bytes
    assert f(1, 8192, 1) == 4096 + 256 and f(10, 777, 3) == 30 * (400 + 28) and f(1, 1, 1) == 20
    for bad in ((0, 4, 1), (-1, 4, 1), (4, 0, 1), (4, 4, 0), ((1 << 31) - 1, (1 << 31) - 1, 1 << 40), (1 << 31, 4, 1)):
        assert f(*bad) == 0


def c_quantize(**kw):
    a = dict(R=8, C=64, X=A0, ldx=64, layout=0, sX=0, dt=0, Q=B0, ldq=32, sQ=0, s=SA0, lds=2, ss=0, rows=None, G=1)
    a.update(kw)
    return tsm.mx4_quantize(a["R"], a["C"], a["X"], a["ldx"], a["layout"], a["sX"], a["dt"], a["Q"], a["ldq"], a["sQ"],
                             a["s"], a["lds"], a["ss"], a["rows"], a["G"], 0)


QUANT = [
    (dict(dt=3), 1, "dtype"), (dict(R=-1), 1, "negative size"), (dict(G=-1), 1, "negative groups"),
    (dict(Q=0), 1, "Q is NULL"), (dict(s=0), 1, "scale is NULL"), (dict(ldq=31), 1, "ldq"), (dict(lds=1), 1, "ld_scale"),
    (dict(rows=P0 + 1), 1, "rows"), (dict(R=1 << 31), 2, "2^31"),
    (dict(G=2, sX=512, sQ=256, ss=-1), 1, "negative stride")]


@pytest.mark.parametrize("kw,status,needle", QUANT + [
    (dict(layout=2), 1, "layout"), (dict(X=0), 1, "X is NULL"), (dict(X=A0 + 2), 1, "X not"), (dict(ldx=-1), 1, "ldx"),
    (dict(Q=A0 + 100), 1, "Q overlaps X"), (dict(s=A0 + 16), 1, "scale overlaps X"),
    (dict(s=B0 + 16), 1, "scale overlaps Q"), (dict(G=2, sX=512, sQ=255, ss=16), 1, "strideQ"),
    (dict(G=2, sX=512, sQ=256, ss=15), 1, "stride_scale"), (dict(G=1 << 40, sX=0, sQ=1 << 40, ss=1 << 40), 2, "overflow")])
def test_quantize_refusals(kw, status, needle):
    refused(c_quantize, kw, status, needle)


def c_dequantize(**kw):
    a = dict(R=8, C=64, Q=B0, ldq=32, sQ=0, s=SA0, lds=2, ss=0, Y=C0, ldy=64, sX=0, dt=0, rows=None, G=1)
    a.update(kw)
    return tsm.mx4_dequantize(a["R"], a["C"], a["Q"], a["ldq"], a["sQ"], a["s"], a["lds"], a["ss"], a["Y"], a["ldy"],
                               a["sX"], a["dt"], a["rows"], a["G"], 0)


@pytest.mark.parametrize("kw,status,needle", QUANT + [
    (dict(Y=0), 1, "Y is NULL"), (dict(Y=C0 + 2), 1, "Y not"), (dict(ldy=63), 1, "ldy"), (dict(Y=B0), 1, "Y overlaps Q"),
    (dict(Y=SA0), 1, "Y overlaps scale"), (dict(G=2, sX=511, sQ=256, ss=16), 1, "strideY")])
def test_dequantize_refusals(kw, status, needle):
    refused(c_dequantize, kw, status, needle)


def route(**kw):
    a = dict(T=8, E=64, k=4, x=A0, ld=64, dt=0, score=0, bias=None, G=1, top=1, best=1, renorm=1, f=1.0, ids=P0, w=W0)
    a.update(kw)
    return tsm.moe_route(a["T"], a["E"], a["k"], a["x"], a["ld"], a["dt"], a["score"], a["bias"], a["G"], a["top"],
                         a["best"], a["renorm"], a["f"], a["ids"], a["w"], 0)


@pytest.mark.parametrize("kw,status,needle", [
    (dict(dt=3), 1, "dtype"), (dict(score=2), 1, "scores"), (dict(T=-1), 1, "negative size"),
    (dict(T=1 << 31), 2, "2^31"), (dict(E=513, ld=513), 2, "513"), (dict(k=65, E=128, ld=128), 2, "topk=65"),
    (dict(k=9, E=8), 1, "topk=9"), (dict(G=0), 1, "groups"), (dict(G=3), 1, "3 groups"), (dict(G=8, top=9), 1, "top_groups"),
    (dict(G=8, top=0), 1, "top_groups"), (dict(G=32, top=1), 1, "topk=4 of the 2"), (dict(best=3), 1, "group_best"),
    (dict(E=256, ld=256, G=128, top=127), 2, "groups=128"), (dict(f=math.nan), 1, "factor"),
    (dict(x=0), 1, "logits is NULL"), (dict(x=A0 + 2), 1, "logits not"), (dict(ld=63), 1, "logits: leading"),
    (dict(bias=B0 + 2), 1, "bias not"), (dict(ids=0), 1, "ids is NULL"), (dict(w=0), 1, "weights is NULL"),
    (dict(w=W0 + 2), 1, "weights not"), (dict(ids=A0 + 64), 1, "ids overlaps logits"),
    (dict(w=A0), 1, "weights overlaps logits"), (dict(ids=W0), 1, "weights overlaps ids"),
    (dict(bias=P0), 1, "ids overlaps bias"), (dict(T=(1 << 31) - 1, ld=1 << 40), 2, "overflows")])
def test_route_refusals(kw, status, needle):
    refused(route, kw, status, needle)


def route_backward(**kw):
    a = dict(T=8, E=64, k=4, dw=W0, x=A0, ld=64, dt=0, ids=P0, score=0, renorm=1, f=1.0, dx=C0, ldd=64)
    a.update(kw)
    return tsm.moe_route_backward(a["T"], a["E"], a["k"], a["dw"], a["x"], a["ld"], a["dt"], a["ids"], a["score"],
                                  a["renorm"], a["f"], a["dx"], a["ldd"], 0)


@pytest.mark.parametrize("kw,status,needle", [
    (dict(dt=3), 1, "dtype"), (dict(score=-1), 1, "scores"), (dict(k=-1), 1, "negative size"), (dict(f=math.inf), 1, "factor"),
    (dict(dw=0), 1, "dweights is NULL"), (dict(ids=0), 1, "ids is NULL"), (dict(x=0), 1, "logits is NULL"),
    (dict(dx=0), 1, "dlogits is NULL"), (dict(ldd=63), 1, "dlogits: leading"), (dict(dx=A0), 1, "dlogits overlaps logits"),
    (dict(dx=P0), 1, "dlogits overlaps ids"), (dict(dx=W0), 1, "dlogits overlaps dweights")])
def test_route_backward_refusals(kw, status, needle):
    refused(route_backward, kw, status, needle)


def test_empty_calls_launch_nothing():
    assert c_quantize(R=0) == 0 and c_quantize(C=0) == 0 and c_quantize(G=0) == 0
    assert c_dequantize(R=0) == 0 and c_dequantize(C=0) == 0 and c_dequantize(G=0) == 0
    assert float_a(M=0) == 0 and float_a(N=0) == 0 and float_a(batch=0) == 0
    assert route(T=0) == 0 and route(k=0) == 0 and route(T=0, E=0, k=0) == 0
    assert route_backward(T=0) == 0 and route_backward(E=0, k=0) == 0


def test_wrappers_refuse_tensors_they_cannot_read():
    import torch

    x = torch.zeros((4, 64))
    q, s = torch.zeros((4, 32), dtype=torch.uint8), torch.zeros((4, 2), dtype=torch.uint8)
    w = torch.zeros((4, 2))
    ids = torch.zeros((4, 2), dtype=torch.int32)
    for call, needle in [
        (lambda: tsm.quantize_mx4(x), "not on a GPU"), (lambda: tsm.quantize_mx4(x[0]), "2-D or 3-D"),
        (lambda: tsm.quantize_mx4(q), "dtype"), (lambda: tsm.quantize_mx4(x, out=q[:, :31]), "out has shape"),
        (lambda: tsm.quantize_mx4(x, scale=q), "scale has shape"),
        (lambda: tsm.quantize_mx4(torch.zeros((8, 4, 64))[::2, ::2, ::2]), "row- or column-major"),
        (lambda: tsm.quantize_mx4(x, rows=torch.zeros(2, dtype=torch.int32)), "rows has shape"),
        (lambda: tsm.dequantize_mx4(q, s), "not on a GPU"), (lambda: tsm.dequantize_mx4(q, s[:, :1]), "scales has shape"),
        (lambda: tsm.dequantize_mx4(q, s, columns=62), "codes has shape"),
        (lambda: tsm.dequantize_mx4(q, s, out=x, out_dtype=torch.float16), "out_dtype"),
        (lambda: tsm.matmul_mx4(q, s, q.t(), s), "not on a GPU"), (lambda: tsm.matmul_mx4(x, None, q.t(), s), "not on a GPU"),
        (lambda: tsm.matmul_mx4(x, s, q.t(), s), "a has dtype"), (lambda: tsm.matmul_mx4(q, None, q.t(), s), "a has dtype"),
        (lambda: tsm.matmul_mx4(q, s, x.t(), s), "b has dtype"), (lambda: tsm.matmul_mx4(q, s, q, s), "inner sizes"),
        (lambda: tsm.matmul_mx4(q, s, q.t().contiguous(), s), "column-major"),
        (lambda: tsm.matmul_mx4(q, s, q.t(), s[:3]), "scale_b has shape"),
        (lambda: tsm.matmul_mx4(q, s[:, :1], q.t(), s), "scale_a has shape"),
        (lambda: tsm.matmul_mx4(q, s, q.t(), s, columns=62), "a has shape"),
        (lambda: tsm.matmul_mx4(x, None, q.t(), s, columns=63), "columns is 63"),
        (lambda: tsm.matmul_mx4(q, s, q.t(), s, activation="gelu"), "activation"),
        (lambda: tsm.route_tokens(x, 2), "not on a GPU"), (lambda: tsm.route_tokens(x[0], 2), "2-D"),
        (lambda: tsm.route_tokens(x, 2, score="max"), "score"),
        (lambda: tsm.route_tokens(x, 2, bias=torch.zeros(63)), "bias has shape"),
        (lambda: tsm.route_tokens(x, 2, ids=ids[:, :1]), "ids has shape"),
        (lambda: tsm.route_tokens_backward(w, x, ids), "not on a GPU"),
        (lambda: tsm.route_tokens_backward(w, x, ids[:3]), "ids must be"),
        (lambda: tsm.route_tokens_backward(w[:, :1], x, ids), "dweights has shape"),
        (lambda: tsm.route_tokens_backward(w, x, ids, out=x.half()), "out has dtype")]:
        with pytest.raises(tsm.TsmError) as ei:
            call()
        assert ei.value.status == tsm.TSM_ERROR_INVALID_VALUE and needle in ei.value.detail, ei.value.detail


def test_allocations_are_made_on_the_stream_of_the_call(monkeypatch):
    """What a call on a stream of its own allocates, a workspace among it, is that stream's memory (the launch and the
    streams are stand-ins here)."""
    import torch

    class OnGpu(torch.Tensor):
        def get_device(self):
            return 0

    active, made = [], []

    @contextlib.contextmanager
    def under(stream):
        active.append(stream)
        yield
        active.pop()

    def recorded(make):
        def f(*a, **kw):
            made.append(active[-1] if active else None)
            return make(*a, **kw)

        return f

    def on_gpu(*shape, dtype=torch.float32):
        return torch.ones(shape, dtype=dtype).as_subclass(OnGpu)

    x, q, s = on_gpu(4, 64), on_gpu(4, 32, dtype=torch.uint8), on_gpu(4, 2, dtype=torch.uint8)
    ids, w = on_gpu(4, 2, dtype=torch.int32), on_gpu(4, 2)
    monkeypatch.setattr(torch.cuda, "stream", under)
    monkeypatch.setattr(torch.cuda, "ExternalStream", lambda handle, device: (handle, device))
    monkeypatch.setattr(torch.cuda, "default_stream", lambda device: ("default", device))
    monkeypatch.setattr(tsm, "_launch", lambda *a: None)
    monkeypatch.setattr(torch, "empty", recorded(torch.empty))
    for handle, want in ((1234, (1234, 0)), (0, ("default", 0)), (None, None)):
        for n, call in [(2, lambda: tsm.quantize_mx4(x, stream=handle)), (1, lambda: tsm.dequantize_mx4(q, s, stream=handle)),
                        (1, lambda: tsm.matmul_mx4(q, s, q.t(), s, stream=handle)),
                        (2, lambda: tsm.matmul_mx4(x, None, q.t(), s, stream=handle)),
                        (2, lambda: tsm.route_tokens(x, 2, stream=handle)),
                        (1, lambda: tsm.route_tokens_backward(w, x, ids, stream=handle))]:
            made.clear()
            call()
            assert made == [want] * n


@pytest.mark.parametrize("M,N,K,batch", [(1024, 1, 32, (1 << 20) + 1), (1, 1, 32, (1 << 31) - 1), (1, 128, 128, (1 << 30) + 1),
                                         (16, 2000, 64, 1 << 23)])
def test_problems_of_one_weight_that_one_grid_cannot_hold_stay_apart(M, N, K, batch):
    """Joined they would pass a launch's work-items, and be refused; one after another they run."""
    assert name_of(M * batch, N, K, shared=True) is None
    assert name_of(M, N, K, batch=batch, shared=True) is not None


def test_problems_of_one_weight_up_to_the_limit_run_as_one():
    """(2^30 rows by 128 columns are 2^23 tiles of 512 work-items, 2^32 in all: one too many.)"""
    assert name_of(1 << 30, 128, 128) is None
    assert name_of(8, 128, 128, batch=(1 << 27) - 16, shared=True) == name_of((1 << 30) - 128, 128, 128) != "mx4_stream"
    assert name_of(8, 128, 128, batch=1 << 27, shared=True) == "mx4_stream"
