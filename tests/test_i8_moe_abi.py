"""Refusals of the int8 and expert-routing entry points: host-side checks, no GPU needed."""

import pytest

import tiled_shared_memory_amd as tsm

# fake, suitably aligned device addresses: never dereferenced by these calls
A0, B0, C0, S0, P0, W0 = (0x7F0000000000 + i * 0x1000000000 for i in range(6))


def gemm(**kw):
    a = dict(M=64, N=128, K=128, A=A0, lda=128, sA=0, sca=S0, ssa=0, B=B0, ldb=128, sB=0, scb=S0 + 4096, ssb=0, C=C0,
             ldc=128, sC=0, batch=1, dt=0, act=0, slope=0.0)
    a.update(kw)
    return tsm.gemm_i8_strided_batched(a["M"], a["N"], a["K"], a["A"], a["lda"], a["sA"], a["sca"], a["ssa"], a["B"],
                                       a["ldb"], a["sB"], a["scb"], a["ssb"], a["C"], a["ldc"], a["sC"], a["batch"],
                                       a["dt"], a["act"], a["slope"], 0)


def refused(fn, kw, status, needle):
    with pytest.raises(tsm.TsmError) as ei:
        fn(**kw)
    assert ei.value.status == status
    assert needle in ei.value.detail


@pytest.mark.parametrize("kw,status,needle", [
    (dict(M=-1), 1, "negative size"), (dict(K=-1), 1, "negative size"), (dict(batch=-1), 1, "negative batch"),
    (dict(dt=3), 1, "out_dtype"), (dict(dt=-1), 1, "out_dtype"), (dict(act=3), 1, "activation"),
    (dict(act=2, slope=float("inf")), 1, "slope"), (dict(A=0), 1, "A is NULL"), (dict(B=0), 1, "B is NULL"),
    (dict(C=0), 1, "C is NULL"), (dict(C=C0 + 2), 1, "aligned"), (dict(dt=1, C=C0 + 1), 1, "aligned"),
    (dict(lda=127), 1, "lda"), (dict(ldb=127), 1, "ldb"), (dict(ldc=127), 1, "ldc"),
    (dict(sca=S0 + 2), 1, "scale_a"), (dict(scb=S0 + 1), 1, "scale_b"), (dict(C=A0 + 4096), 1, "overlaps A"),
    (dict(C=B0), 1, "overlaps B"), (dict(C=S0 + 64), 1, "overlaps scale_a"), (dict(scb=C0 + 64), 1, "scale_b"),
    (dict(batch=2, sC=1), 1, "strideC"), (dict(batch=2, sC=64 * 128, sA=-1), 1, "negative stride"),
    (dict(K=131072, lda=131072, ldb=131072), 2, "int32"), (dict(M=1 << 31), 2, "2^31"),
    (dict(M=(1 << 31) - 1, N=(1 << 31) - 1, ldc=(1 << 31) - 1, C=1 << 62), 2, "overflows"),
    (dict(batch=1 << 40, sA=1 << 40, sB=1 << 40, sC=1 << 40), 2, "overflows")])
def test_gemm_i8_refusals(kw, status, needle):
    refused(gemm, kw, status, needle)


@pytest.mark.parametrize("kw", [dict(M=0), dict(N=0), dict(batch=0), dict(M=0, A=0, B=0, C=0)])
def test_gemm_i8_empty(kw):
    assert gemm(**kw) == 0


@pytest.mark.parametrize("name,kw,status", [("i8_nothing", {}, 1), ("i8_tile_256x256x128", dict(K=127), 2),
                                            ("i8_tile_256x256x128", dict(N=124), 2),
                                            ("i8_tile_256x256x128", dict(A=A0 + 8), 2),
                                            ("i8_tile_256x256x128", dict(lda=136), 2),
                                            ("i8_tile_256x256x128", dict(dt=2, ldc=132), 2)])
def test_forced_variants_that_cannot_run_are_refused(monkeypatch, name, kw, status):
    monkeypatch.setenv("TSM_GEMM_KERNEL", name)
    refused(gemm, kw, status, name)


def test_gemm_i8_grouped_needs_counts():
    for rows, needle in ((0, "rows is NULL"), (P0 + 2, "rows not 4-byte")):
        with pytest.raises(tsm.TsmError) as ei:
            tsm.gemm_i8_grouped(64, 128, 128, A0, 128, 64 * 128, S0, 64, B0, 128, 128 * 128, None, 0, C0, 128, 64 * 128,
                                rows, 2, 0, 0, 0.0, 0)
        assert needle in ei.value.detail


def quantize(**kw):
    a = dict(R=8, C=64, X=A0, ldx=64, sX=0, dt=0, Q=B0, ldq=64, sQ=0, scale=S0, ss=0, rows=None, groups=1)
    a.update(kw)
    return tsm.quantize_i8(a["R"], a["C"], a["X"], a["ldx"], a["sX"], a["dt"], a["Q"], a["ldq"], a["sQ"], a["scale"],
                           a["ss"], a["rows"], a["groups"], 0)


@pytest.mark.parametrize("kw,status,needle", [
    (dict(dt=3), 1, "xdtype"), (dict(R=-1), 1, "negative size"), (dict(groups=-2), 1, "negative groups"),
    (dict(scale=0), 1, "scale is NULL"), (dict(scale=S0 + 2), 1, "scale not"), (dict(X=0), 1, "X is NULL"),
    (dict(Q=0), 1, "Q is NULL"), (dict(X=A0 + 2), 1, "X not"), (dict(dt=1, X=A0 + 1), 1, "X not"),
    (dict(ldx=-1), 1, "ldx"), (dict(ldq=63), 1, "ldq"), (dict(Q=A0 + 100), 1, "Q overlaps X"),
    (dict(scale=A0 + 16), 1, "scale overlaps X"), (dict(scale=B0 + 16), 1, "scale overlaps Q"),
    (dict(rows=P0 + 1), 1, "rows"), (dict(groups=2, ss=7), 1, "stride_scale"),
    (dict(groups=2, ss=8, sX=512, sQ=100), 1, "strideQ"), (dict(groups=2, ss=8, sX=-1, sQ=512), 1, "negative stride"),
    (dict(R=1 << 31), 2, "2^31"), (dict(groups=1 << 40, ss=1 << 40, sX=0, sQ=1 << 40), 2, "overflow")])
def test_quantize_refusals(kw, status, needle):
    refused(quantize, kw, status, needle)


def sort(**kw):
    a = dict(T=64, k=2, ids=A0, ld=2, idt=4, E=8, cap=20, pos=P0, counts=C0, ws=None, wsb=0)
    a.update(kw)
    return tsm.moe_sort(a["T"], a["k"], a["ids"], a["ld"], a["idt"], a["E"], a["cap"], a["pos"], a["counts"], a["ws"],
                        a["wsb"], 0)


@pytest.mark.parametrize("kw,status,needle", [
    (dict(idt=0), 1, "idtype"), (dict(T=-1), 1, "negative size"), (dict(cap=-1), 1, "negative size"),
    (dict(E=513), 2, "513"), (dict(T=1 << 31), 2, "2^31"), (dict(cap=1 << 30), 2, "2^31"),
    (dict(ids=0), 1, "ids is NULL"), (dict(ids=A0 + 2), 1, "ids not"), (dict(idt=5, ids=A0 + 4), 1, "ids not"),
    (dict(ld=1), 1, "ids: leading"), (dict(pos=0), 1, "positions is NULL"), (dict(counts=0), 1, "counts is NULL"),
    (dict(counts=C0 + 1), 1, "counts not"), (dict(pos=A0 + 8), 1, "positions overlaps ids"),
    (dict(counts=P0 + 4), 1, "counts overlaps positions"), (dict(T=8192), 1, "workspace is NULL"),
    (dict(T=8192, ws=W0, wsb=100), 1, "needed"), (dict(T=8192, ws=W0 + 2, wsb=1 << 20), 1, "workspace not"),
    (dict(T=8192, ws=P0, wsb=1 << 20), 1, "workspace overlaps positions"), (dict(wsb=-1), 1, "workspace_bytes")])
def test_sort_refusals(kw, status, needle):
    refused(sort, kw, status, needle)


def test_sort_workspace_sizes():
    assert tsm.moe_sort_workspace_bytes(4096, 2, 8) == 0
    assert tsm.moe_sort_workspace_bytes(4097, 2, 8) > 0
    for bad in ((-1, 2, 8), (1 << 40, 1 << 40, 8), (1 << 20, 8, 513), (0, 0, 0)):
        assert tsm.moe_sort_workspace_bytes(*bad) == 0


def dispatch(**kw):
    a = dict(T=8, k=2, H=64, X=A0, ldx=64, dt=2, scale=None, pos=P0, slots=32, slabs=B0, lds=64, ss=None)
    a.update(kw)
    return tsm.moe_dispatch(a["T"], a["k"], a["H"], a["X"], a["ldx"], a["dt"], a["scale"], a["pos"], a["slots"],
                            a["slabs"], a["lds"], a["ss"], 0)


@pytest.mark.parametrize("kw,status,needle", [
    (dict(dt=4), 1, "dtype"), (dict(T=-1), 1, "negative size"), (dict(slots=1 << 31), 2, "2^31"),
    (dict(X=0), 1, "X is NULL"), (dict(X=A0 + 1), 1, "X not"), (dict(ldx=63), 1, "X: leading"),
    (dict(slabs=0), 1, "slabs is NULL"), (dict(lds=63), 1, "slabs: leading"), (dict(pos=0), 1, "positions is NULL"),
    (dict(pos=P0 + 2), 1, "positions not"), (dict(scale=S0), 1, "come together"), (dict(ss=S0), 1, "come together"),
    (dict(scale=S0 + 1, ss=W0), 1, "scale not"), (dict(slabs=A0 + 64), 1, "slabs overlaps X"),
    (dict(slabs=P0), 1, "slabs overlaps positions"), (dict(scale=S0, ss=B0 + 4), 1, "slab_scale overlaps slabs"),
    (dict(T=(1 << 31) - 1, k=1, ldx=1 << 40), 2, "overflows"), (dict(T=1 << 30), 2, "2^31")])
def test_dispatch_refusals(kw, status, needle):
    refused(dispatch, kw, status, needle)


def combine(**kw):
    a = dict(T=8, k=2, H=64, slabs=A0, lds=64, slots=32, dt=2, pos=P0, w=W0, Y=C0, ldy=64)
    a.update(kw)
    return tsm.moe_combine(a["T"], a["k"], a["H"], a["slabs"], a["lds"], a["slots"], a["dt"], a["pos"], a["w"], a["Y"],
                           a["ldy"], 0)


@pytest.mark.parametrize("kw,status,needle", [
    (dict(dt=3), 1, "dtype"), (dict(k=-1), 1, "negative size"), (dict(Y=0), 1, "Y is NULL"),
    (dict(Y=C0 + 1), 1, "Y not"), (dict(ldy=63), 1, "Y: leading"), (dict(slabs=0), 1, "slabs is NULL"),
    (dict(lds=1), 1, "slabs: leading"), (dict(pos=0), 1, "positions is NULL"), (dict(w=W0 + 2), 1, "weights not"),
    (dict(Y=A0 + 128), 1, "Y overlaps slabs"), (dict(Y=P0), 1, "Y overlaps positions"),
    (dict(Y=W0), 1, "Y overlaps weights")])
def test_combine_refusals(kw, status, needle):
    refused(combine, kw, status, needle)


def backward(**kw):
    a = dict(T=8, k=2, H=64, dY=C0, lddy=64, slabs=A0, lds=64, slots=32, dt=2, pos=P0, w=W0, ds=B0, ldd=64, dw=S0)
    a.update(kw)
    return tsm.moe_combine_backward(a["T"], a["k"], a["H"], a["dY"], a["lddy"], a["slabs"], a["lds"], a["slots"],
                                    a["dt"], a["pos"], a["w"], a["ds"], a["ldd"], a["dw"], 0)


@pytest.mark.parametrize("kw,status,needle", [
    (dict(dt=3), 1, "dtype"), (dict(H=-1), 1, "negative size"), (dict(dY=0), 1, "dY is NULL"),
    (dict(slabs=0), 1, "slabs is NULL"), (dict(ds=0), 1, "dslabs is NULL"), (dict(ldd=63), 1, "dslabs: leading"),
    (dict(lddy=63), 1, "dY: leading"), (dict(pos=0), 1, "positions is NULL"), (dict(dw=0), 1, "dweights is NULL"),
    (dict(w=W0 + 1), 1, "weights not"), (dict(ds=A0), 1, "dslabs overlaps slabs"), (dict(dw=B0), 1, "dweights overlaps dslabs"),
    (dict(dw=W0), 1, "dweights overlaps weights"), (dict(ds=C0), 1, "dslabs overlaps dY")])
def test_backward_refusals(kw, status, needle):
    refused(backward, kw, status, needle)


def test_empty_calls_launch_nothing():
    assert quantize(R=0) == 0 and quantize(groups=0) == 0
    assert dispatch(T=0) == 0 and dispatch(k=0) == 0 and dispatch(slots=0) == 0 and dispatch(H=0) == 0
    assert combine(T=0) == 0 and combine(H=0) == 0
    assert backward(T=0) == 0 and backward(k=0) == 0
    assert sort(T=0, E=0) == 0


def test_wrappers_refuse_tensors_they_cannot_read():
    import torch

    x = torch.zeros((4, 8))
    q = torch.zeros((4, 8), dtype=torch.int8)
    pos = torch.zeros((4, 2), dtype=torch.int32)
    for call, needle in [
        (lambda: tsm.quantize(x), "not on a GPU"), (lambda: tsm.quantize(x[0]), "2-D or 3-D"),
        (lambda: tsm.matmul_i8(q, None, q.t(), None), "not on a GPU"),
        (lambda: tsm.matmul_i8(q[0], None, q.t(), None), "2-D or 3-D"),
        (lambda: tsm.sort_tokens(pos, 4, 4), "not on a GPU"), (lambda: tsm.sort_tokens(pos[0], 4, 4), "2-D"),
        (lambda: tsm.dispatch_tokens(x, pos, slots=4), "not on a GPU"),
        (lambda: tsm.combine_tokens(x, pos), "not on a GPU"),
        (lambda: tsm.combine_tokens_backward(x, x, pos), "not on a GPU")]:
        with pytest.raises(tsm.TsmError) as ei:
            call()
        assert ei.value.status == tsm.TSM_ERROR_INVALID_VALUE and needle in ei.value.detail


@pytest.mark.parametrize("M,N,K,batch,grouped,off,want", [
    (1, 8192, 8192, 1, 0, 0, "i8_stream"), (4, 28672, 4096, 1, 0, 0, "i8_skinny"),
    (4, 28672, 4112, 1, 0, 0, "i8_stream"), (4, 1024, 4096, 4, 1, 0, "i8_stream"),
    (16, 4096, 4095, 1, 0, 0, "i8_skinny"), (16, 4112, 4095, 1, 0, 0, "i8_block_64x64x128"),
    (1, 4096, 4096, 2, 0, 1, "i8_block_64x64x128"), (17, 64, 256, 1, 0, 1, "i8_block_64x64x128"),
    (32, 65536, 4096, 1, 0, 0, "i8_stream"), (33, 12272, 4096, 1, 0, 0, "i8_stream"),
    (33, 12288, 4096, 1, 0, 0, "i8_block_64x64x128"), (64, 32768, 8192, 1, 0, 0, "i8_block_64x64x128"),
    (64, 1024, 2048, 64, 0, 0, "i8_block_64x64x128"), (64, 1024, 2048, 64, 1, 0, "i8_stream"),
    (128, 16384, 8192, 1, 0, 0, "i8_block_64x64x128"), (128, 32768, 8192, 1, 0, 0, "i8_block_128x128x128"),
    (128, 32896, 8192, 1, 0, 0, "i8_tile_256x256x128"), (129, 18432, 4096, 1, 0, 0, "i8_tile_256x256x128"),
    (129, 16384, 4096, 1, 0, 0, "i8_block_128x128x128"), (2304, 2304, 1024, 1, 0, 0, "i8_tile_256x256x128")])
def test_i8_routing(monkeypatch, M, N, K, batch, grouped, off, want):
    """The kernel on either side of each border of the selection's rule."""
    monkeypatch.delenv("TSM_GEMM_KERNEL", raising=False)
    rows = P0 if grouped else None
    assert tsm.tsm_gemm_i8_kernel_name(M, N, K, A0 + off, K, M * K, B0, K, N * K, C0, N, M * N, batch, rows, 0) == want


def test_i8_routing_of_very_wide_products(monkeypatch):
    """Past the columns that one launch of the few-row kernels or of 64-tiles holds: 128-tiles."""
    monkeypatch.delenv("TSM_GEMM_KERNEL", raising=False)

    def route(M, N, K=16):
        return tsm.tsm_gemm_i8_kernel_name(M, N, K, A0, K, 0, B0, K, 0, 1 << 60, N, 0, 1, None, 1)

    assert route(40, (1 << 28) + 64) == "i8_block_64x64x128"
    assert route(40, 1 << 29) == "i8_block_128x128x128"
    monkeypatch.setenv("TSM_GEMM_KERNEL", "i8_skinny")
    assert route(16, 1 << 27) == "i8_skinny"
    assert route(40, (1 << 28) - 64) is None  # 3 x 2^24 blocks: cannot run


def test_allocations_are_made_and_filled_on_the_stream_of_the_call(monkeypatch):
    """What a call on a stream of its own allocates is that stream's memory, and zeros are written there (the launch
    and the streams are stand-ins here)."""
    import contextlib

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

    x, q, pos = on_gpu(4, 8), on_gpu(4, 8, dtype=torch.int8), on_gpu(4, 2, dtype=torch.int32)
    s, b = on_gpu(4), on_gpu(6, 8, dtype=torch.int8)
    monkeypatch.setattr(torch.cuda, "stream", under)
    monkeypatch.setattr(torch.cuda, "ExternalStream", lambda handle, device: (handle, device))
    monkeypatch.setattr(torch.cuda, "default_stream", lambda device: ("default", device))
    monkeypatch.setattr(tsm, "_launch", lambda *a: None)
    monkeypatch.setattr(torch, "empty", recorded(torch.empty))
    monkeypatch.setattr(torch, "zeros", recorded(torch.zeros))
    for handle, want in ((1234, (1234, 0)), (0, ("default", 0)), (None, None)):
        for n, call in [
            (2, lambda: tsm.quantize(x, stream=handle)), (1, lambda: tsm.matmul_i8(q, s, b.t(), None, stream=handle)),
            (2, lambda: tsm.sort_tokens(pos, 3, 4, stream=handle)),
            (2, lambda: tsm.dispatch_tokens(q, pos, slots=9, scale=s, stream=handle)),
            (1, lambda: tsm.combine_tokens(x, pos, stream=handle)),
            (1, lambda: tsm.dispatch_tokens_backward(x, pos, stream=handle)),
            (2, lambda: tsm.combine_tokens_backward(x, x, pos, stream=handle))]:
            made.clear()
            call()
            assert made == [want] * n


def test_calls_on_a_stream_refuse_tensors_off_the_gpu():
    import torch

    x, pos = torch.zeros((4, 8)), torch.zeros((4, 2), dtype=torch.int32)
    for call in (lambda: tsm.quantize(x, stream=1234), lambda: tsm.combine_tokens_backward(x, x, pos, stream=1234)):
        with pytest.raises(tsm.TsmError) as ei:
            call()
        assert ei.value.status == tsm.TSM_ERROR_INVALID_VALUE and "not on a GPU" in ei.value.detail


def test_a_forced_variant_past_its_grid_is_refused(monkeypatch):
    """4096 x 2050 tiles of 64 x 64 on 512 threads pass 2^32 work-items, 2048 x 1025 of 128 x 128 do not."""
    args = (262144, 131200, 16, A0, 16, 0, B0, 16, 0, 1 << 60, 131200, 0, 1, None, 1)
    monkeypatch.setenv("TSM_GEMM_KERNEL", "i8_block_128x128x128")
    assert tsm.tsm_gemm_i8_kernel_name(*args) == "i8_block_128x128x128"
    monkeypatch.setenv("TSM_GEMM_KERNEL", "i8_block_64x64x128")
    assert tsm.tsm_gemm_i8_kernel_name(*args) is None
    refused(gemm, dict(M=262144, N=131200, K=16, lda=16, ldb=16, ldc=131200, C=1 << 60, dt=1, sca=None, scb=None), 2,
            "i8_block_64x64x128")
