"""ctypes binding of ``libtsm_gemm.so`` (the C ABI in ``include/tsm_gemm.h``).

Argument marshalling only: pointers, sizes and the stream handle go straight
to the C entry points of the same names, and a non-zero status becomes a
``TsmError``.  All arithmetic runs in the library's HIP kernels; there is no
fallback.  ``torch`` is imported first so the library binds to the HIP runtime
torch already loaded (both carry the soname ``libamdhip64.so.7``), which makes
torch's stream handles and device pointers valid inside the library.
"""

from __future__ import annotations

import ctypes
import os

PKG = os.path.dirname(os.path.abspath(__file__))
LIBRARY = os.path.join(PKG, "libtsm_gemm.so")

TSM_SUCCESS = 0
TSM_ERROR_INVALID_VALUE = 1
TSM_ERROR_NOT_SUPPORTED = 2
TSM_ERROR_LAUNCH = 3

TSM_F16_F32 = 0
TSM_F16_F16 = 1
TSM_BF16_F32 = 2
TSM_BF16_F16 = 3
TSM_F16_BF16 = 4
TSM_BF16_BF16 = 5

TSM_ACT_NONE = 0
TSM_ACT_RELU = 1
TSM_ACT_LEAKY_RELU = 2

TSM_ROW = 0
TSM_COL = 1

TSM_ROWSUM_F32 = 0
TSM_ROWSUM_F16 = 1
TSM_ROWSUM_BF16 = 2

TSM_F32 = 0
TSM_F16 = 1
TSM_BF16 = 2
TSM_I8 = 3
TSM_I32 = 4
TSM_I64 = 5

TSM_SCORE_SOFTMAX = 0
TSM_SCORE_SIGMOID = 1

# Every function the header declares, with its ctypes signature.
_I64, _PTR, _INT = ctypes.c_int64, ctypes.c_void_p, ctypes.c_int
SIGNATURES = {
    "gemm": ([_I64, _I64, _I64, _PTR, _I64, _PTR, _I64, _PTR, _I64, _INT, _PTR], _INT),
    "gemm_ex": ([_I64, _I64, _I64, _PTR, _I64, _INT, _PTR, _I64, _INT, _PTR, _I64, _INT, _PTR], _INT),
    "gemm_strided_batched": ([_I64, _I64, _I64, _PTR, _I64, _I64, _PTR, _I64, _I64, _PTR, _I64, _I64, _I64, _INT,
                              _PTR], _INT),
    "gemm_strided_batched_ex": ([_I64, _I64, _I64, _PTR, _I64, _INT, _I64, _PTR, _I64, _INT, _I64, _PTR, _I64, _I64,
                                 _I64, _INT, _PTR], _INT),
    "tsm_status_string": ([_INT], ctypes.c_char_p),
    "tsm_last_error_detail": ([], ctypes.c_char_p),
    "tsm_gemm_kernel_name": ([_I64, _I64, _I64, _PTR, _I64, _INT, _I64, _PTR, _I64, _INT, _I64, _PTR, _I64, _I64,
                              _I64, _INT], ctypes.c_char_p),
    "gemm_grouped": ([_I64, _I64, _I64, _PTR, _I64, _INT, _I64, _PTR, _I64, _INT, _I64, _PTR, _I64, _I64, _PTR, _I64,
                      _INT, _PTR], _INT),
    "tsm_gemm_grouped_kernel_name": ([_I64, _I64, _I64, _PTR, _I64, _INT, _I64, _PTR, _I64, _INT, _I64, _PTR, _I64,
                                      _I64, _PTR, _I64, _INT], ctypes.c_char_p),
    "rowsum": ([_I64, _I64, _PTR, _I64, _I64, _INT, _PTR, _PTR], _INT),
    "gemm_strided_batched_act": ([_I64, _I64, _I64, _PTR, _I64, _INT, _I64, _PTR, _I64, _INT, _I64, _PTR, _I64, _I64,
                                  _I64, _INT, _INT, ctypes.c_float, _PTR], _INT),
    "tsm_rowsum_kernel_name": ([_I64, _I64, _PTR, _I64, _I64, _INT, _PTR], ctypes.c_char_p),
    "gemm_workspace_bytes": ([_I64, _I64, _I64, _I64], _I64),
    "gemm_strided_batched_ws": ([_I64, _I64, _I64, _PTR, _I64, _INT, _I64, _PTR, _I64, _INT, _I64, _PTR, _I64, _I64,
                                 _I64, _INT, _INT, ctypes.c_float, _PTR, _I64, _PTR], _INT),
    "gemm_strided_batched_noalloc": ([_I64, _I64, _I64, _PTR, _I64, _INT, _I64, _PTR, _I64, _INT, _I64, _PTR, _I64,
                                      _I64, _I64, _INT, _INT, ctypes.c_float, _PTR], _INT),
    "gemm_noalloc_scratch_bytes": ([], _I64),
    "tsm_gemm_ws_kernel_name": ([_I64, _I64, _I64, _PTR, _I64, _INT, _I64, _PTR, _I64, _INT, _I64, _PTR, _I64, _I64,
                                 _I64, _INT, _PTR, _I64], ctypes.c_char_p),
    "quantize_i8": ([_I64, _I64, _PTR, _I64, _I64, _INT, _PTR, _I64, _I64, _PTR, _I64, _PTR, _I64, _PTR], _INT),
    "gemm_i8": ([_I64, _I64, _I64, _PTR, _I64, _PTR, _PTR, _I64, _PTR, _PTR, _I64, _INT, _PTR], _INT),
    "gemm_i8_strided_batched": ([_I64, _I64, _I64, _PTR, _I64, _I64, _PTR, _I64, _PTR, _I64, _I64, _PTR, _I64, _PTR,
                                 _I64, _I64, _I64, _INT, _INT, ctypes.c_float, _PTR], _INT),
    "gemm_i8_grouped": ([_I64, _I64, _I64, _PTR, _I64, _I64, _PTR, _I64, _PTR, _I64, _I64, _PTR, _I64, _PTR, _I64,
                         _I64, _PTR, _I64, _INT, _INT, ctypes.c_float, _PTR], _INT),
    "tsm_gemm_i8_kernel_name": ([_I64, _I64, _I64, _PTR, _I64, _I64, _PTR, _I64, _I64, _PTR, _I64, _I64, _I64, _PTR,
                                 _INT], ctypes.c_char_p),
    "moe_sort": ([_I64, _I64, _PTR, _I64, _INT, _I64, _I64, _PTR, _PTR, _PTR, _I64, _PTR], _INT),
    "moe_sort_workspace_bytes": ([_I64, _I64, _I64], _I64),
    "moe_dispatch": ([_I64, _I64, _I64, _PTR, _I64, _INT, _PTR, _PTR, _I64, _PTR, _I64, _PTR, _PTR], _INT),
    "moe_combine": ([_I64, _I64, _I64, _PTR, _I64, _I64, _INT, _PTR, _PTR, _PTR, _I64, _PTR], _INT),
    "moe_combine_backward": ([_I64, _I64, _I64, _PTR, _I64, _PTR, _I64, _I64, _INT, _PTR, _PTR, _PTR, _I64, _PTR,
                              _PTR], _INT),
    "mx4_quantize": ([_I64, _I64, _PTR, _I64, _INT, _I64, _INT, _PTR, _I64, _I64, _PTR, _I64, _I64, _PTR, _I64, _PTR],
                     _INT),
    "mx4_dequantize": ([_I64, _I64, _PTR, _I64, _I64, _PTR, _I64, _I64, _PTR, _I64, _I64, _INT, _PTR, _I64, _PTR],
                       _INT),
    "gemm_mx4": ([_I64, _I64, _I64, _PTR, _I64, _PTR, _I64, _PTR, _I64, _PTR, _I64, _PTR, _I64, _INT, _PTR], _INT),
    "gemm_mx4_strided_batched": ([_I64, _I64, _I64, _PTR, _I64, _I64, _PTR, _I64, _I64, _PTR, _I64, _I64, _PTR,
                                  _I64, _I64, _PTR, _I64, _I64, _I64, _INT, _INT, ctypes.c_float, _PTR], _INT),
    "gemm_mx4_grouped": ([_I64, _I64, _I64, _PTR, _I64, _I64, _PTR, _I64, _I64, _PTR, _I64, _I64, _PTR, _I64, _I64,
                          _PTR, _I64, _I64, _PTR, _I64, _INT, _INT, ctypes.c_float, _PTR], _INT),
    "gemm_mx4_float_a": ([_I64, _I64, _I64, _PTR, _I64, _I64, _INT, _PTR, _I64, _I64, _PTR, _I64, _I64, _PTR, _I64,
                          _I64, _I64, _PTR, _INT, _INT, ctypes.c_float, _PTR, _I64, _PTR], _INT),
    "gemm_mx4_float_a_workspace_bytes": ([_I64, _I64, _I64], _I64),
    "tsm_gemm_mx4_kernel_name": ([_I64, _I64, _I64, _PTR, _I64, _I64, _PTR, _I64, _I64, _PTR, _I64, _I64, _PTR,
                                  _I64, _I64, _PTR, _I64, _I64, _I64, _PTR, _INT], ctypes.c_char_p),
    "moe_route": ([_I64, _I64, _I64, _PTR, _I64, _INT, _INT, _PTR, _I64, _I64, _INT, _INT, ctypes.c_float, _PTR,
                   _PTR, _PTR], _INT),
    "moe_route_backward": ([_I64, _I64, _I64, _PTR, _PTR, _I64, _INT, _PTR, _INT, _INT, ctypes.c_float, _PTR, _I64,
                            _PTR], _INT),
}


class TsmError(RuntimeError):
    def __init__(self, status: int, detail: str):
        super().__init__(f"{_status_text(status)} ({status}): {detail}")
        self.status = status
        self.detail = detail


_LIB = None


def load(path: str = LIBRARY):
    """Load the HIP library (after torch's HIP runtime); raise if it is not built."""
    global _LIB
    if _LIB is not None and path == LIBRARY:
        return _LIB
    import torch  # noqa: F401  -- binds the library to torch's HIP runtime

    if not os.path.exists(path):
        raise RuntimeError(f"{path} is not built: run `python -c 'import __graft_entry__ as g; g.build()'` "
                           "(there is no CPU fallback)")
    lib = ctypes.CDLL(path)
    for name, (args, res) in SIGNATURES.items():
        fn = getattr(lib, name)
        fn.argtypes = args
        fn.restype = res
    if path == LIBRARY:
        _LIB = lib
    return lib


def _status_text(status: int) -> str:
    return {0: "success", 1: "invalid value", 2: "not supported", 3: "launch failure"}.get(status, "unknown status")


def _ptr(x):
    if x is None:
        return None
    if isinstance(x, int):
        return x
    return x.data_ptr()


_LOOKUPS = None  # torch's (current device index, current stream handle of a device)


def _lookups():
    global _LOOKUPS
    if _LOOKUPS is None:
        import torch

        torch.cuda.current_stream()  # initialises the device
        raw = getattr(torch._C, "_cuda_getCurrentRawStream", None)
        _LOOKUPS = (getattr(torch._C, "_cuda_getDevice", torch.cuda.current_device),
                    raw or (lambda device: torch.cuda.current_stream(device).cuda_stream))
    return _LOOKUPS


def _current_stream():
    """Handle of the current stream of the current GPU: torch's own lookup, without the Stream object that
    ``torch.cuda.current_stream()`` builds around it (2.6 us, as much as a launch)."""
    device, stream = _lookups()
    return stream(device())


def _stream(stream):
    if stream is None:
        return _current_stream()
    if isinstance(stream, int):
        return stream
    return stream.cuda_stream


def _check(lib, status: int):
    if status != TSM_SUCCESS:
        detail = lib.tsm_last_error_detail()
        raise TsmError(status, detail.decode() if detail else "")
    return status


def gemm(M, N, K, A, lda, B, ldb, C, ldc, dtype, stream=None):
    lib = load()
    return _check(lib, lib.gemm(M, N, K, _ptr(A), lda, _ptr(B), ldb, _ptr(C), ldc, dtype, _stream(stream)))


def gemm_ex(M, N, K, A, lda, layout_a, B, ldb, layout_b, C, ldc, dtype, stream=None):
    lib = load()
    return _check(lib, lib.gemm_ex(M, N, K, _ptr(A), lda, layout_a, _ptr(B), ldb, layout_b, _ptr(C), ldc, dtype,
                                   _stream(stream)))


def gemm_strided_batched(M, N, K, A, lda, strideA, B, ldb, strideB, C, ldc, strideC, batch, dtype, stream=None):
    lib = load()
    return _check(lib, lib.gemm_strided_batched(M, N, K, _ptr(A), lda, strideA, _ptr(B), ldb, strideB, _ptr(C), ldc,
                                                strideC, batch, dtype, _stream(stream)))


def gemm_strided_batched_ex(M, N, K, A, lda, layout_a, strideA, B, ldb, layout_b, strideB, C, ldc, strideC, batch,
                            dtype, stream=None):
    lib = load()
    return _check(lib, lib.gemm_strided_batched_ex(M, N, K, _ptr(A), lda, layout_a, strideA, _ptr(B), ldb, layout_b,
                                                   strideB, _ptr(C), ldc, strideC, batch, dtype, _stream(stream)))


def gemm_strided_batched_act(M, N, K, A, lda, layout_a, strideA, B, ldb, layout_b, strideB, C, ldc, strideC, batch,
                             dtype, activation, slope, stream=None):
    lib = load()
    return _check(lib, lib.gemm_strided_batched_act(M, N, K, _ptr(A), lda, layout_a, strideA, _ptr(B), ldb, layout_b,
                                                    strideB, _ptr(C), ldc, strideC, batch, dtype, activation, slope,
                                                    _stream(stream)))


def gemm_workspace_bytes(M, N, K, batch):
    return int(load().gemm_workspace_bytes(M, N, K, batch))


def gemm_strided_batched_ws(M, N, K, A, lda, layout_a, strideA, B, ldb, layout_b, strideB, C, ldc, strideC, batch,
                            dtype, activation, slope, workspace, workspace_bytes, stream=None):
    lib = load()
    return _check(lib, lib.gemm_strided_batched_ws(M, N, K, _ptr(A), lda, layout_a, strideA, _ptr(B), ldb, layout_b,
                                                   strideB, _ptr(C), ldc, strideC, batch, dtype, activation, slope,
                                                   _ptr(workspace), workspace_bytes, _stream(stream)))


def gemm_strided_batched_noalloc(M, N, K, A, lda, layout_a, strideA, B, ldb, layout_b, strideB, C, ldc, strideC,
                                 batch, dtype, activation, slope, stream=None):
    lib = load()
    return _check(lib, lib.gemm_strided_batched_noalloc(M, N, K, _ptr(A), lda, layout_a, strideA, _ptr(B), ldb,
                                                        layout_b, strideB, _ptr(C), ldc, strideC, batch, dtype,
                                                        activation, slope, _stream(stream)))


def gemm_noalloc_scratch_bytes():
    return int(load().gemm_noalloc_scratch_bytes())


def tsm_gemm_ws_kernel_name(M, N, K, A, lda, layout_a, strideA, B, ldb, layout_b, strideB, C, ldc, strideC, batch,
                            dtype, workspace, workspace_bytes):
    r = load().tsm_gemm_ws_kernel_name(M, N, K, _ptr(A), lda, layout_a, strideA, _ptr(B), ldb, layout_b, strideB,
                                       _ptr(C), ldc, strideC, batch, dtype, _ptr(workspace), workspace_bytes)
    return r.decode() if r else None


def gemm_grouped(M, N, K, A, lda, layout_a, strideA, B, ldb, layout_b, strideB, C, ldc, strideC, rows, groups, dtype,
                 stream=None):
    lib = load()
    return _check(lib, lib.gemm_grouped(M, N, K, _ptr(A), lda, layout_a, strideA, _ptr(B), ldb, layout_b, strideB,
                                        _ptr(C), ldc, strideC, _ptr(rows), groups, dtype, _stream(stream)))


def tsm_status_string(status: int) -> str:
    return load().tsm_status_string(status).decode()


def tsm_last_error_detail() -> str:
    return load().tsm_last_error_detail().decode()


def tsm_gemm_kernel_name(M, N, K, A, lda, layout_a, strideA, B, ldb, layout_b, strideB, C, ldc, strideC, batch,
                         dtype):
    r = load().tsm_gemm_kernel_name(M, N, K, _ptr(A), lda, layout_a, strideA, _ptr(B), ldb, layout_b, strideB,
                                    _ptr(C), ldc, strideC, batch, dtype)
    return r.decode() if r else None


def tsm_gemm_grouped_kernel_name(M, N, K, A, lda, layout_a, strideA, B, ldb, layout_b, strideB, C, ldc, strideC, rows,
                                 groups, dtype):
    r = load().tsm_gemm_grouped_kernel_name(M, N, K, _ptr(A), lda, layout_a, strideA, _ptr(B), ldb, layout_b, strideB,
                                            _ptr(C), ldc, strideC, _ptr(rows), groups, dtype)
    return r.decode() if r else None


def rowsum(R, C, X, row_stride, col_stride, xdtype, out, stream=None):
    lib = load()
    return _check(lib, lib.rowsum(R, C, _ptr(X), row_stride, col_stride, xdtype, _ptr(out), _stream(stream)))


def tsm_rowsum_kernel_name(R, C, X, row_stride, col_stride, xdtype, out):
    r = load().tsm_rowsum_kernel_name(R, C, _ptr(X), row_stride, col_stride, xdtype, _ptr(out))
    return r.decode() if r else None


def quantize_i8(R, C, X, ldx, strideX, xdtype, Q, ldq, strideQ, scale, stride_scale, rows, groups, stream=None):
    lib = load()
    return _check(lib, lib.quantize_i8(R, C, _ptr(X), ldx, strideX, xdtype, _ptr(Q), ldq, strideQ, _ptr(scale),
                                       stride_scale, _ptr(rows), groups, _stream(stream)))


def gemm_i8(M, N, K, A, lda, scale_a, B, ldb, scale_b, C, ldc, out_dtype, stream=None):
    lib = load()
    return _check(lib, lib.gemm_i8(M, N, K, _ptr(A), lda, _ptr(scale_a), _ptr(B), ldb, _ptr(scale_b), _ptr(C), ldc,
                                   out_dtype, _stream(stream)))


def gemm_i8_strided_batched(M, N, K, A, lda, strideA, scale_a, stride_sa, B, ldb, strideB, scale_b, stride_sb, C, ldc,
                            strideC, batch, out_dtype, activation, slope, stream=None):
    lib = load()
    return _check(lib, lib.gemm_i8_strided_batched(M, N, K, _ptr(A), lda, strideA, _ptr(scale_a), stride_sa, _ptr(B),
                                                   ldb, strideB, _ptr(scale_b), stride_sb, _ptr(C), ldc, strideC,
                                                   batch, out_dtype, activation, slope, _stream(stream)))


def gemm_i8_grouped(M, N, K, A, lda, strideA, scale_a, stride_sa, B, ldb, strideB, scale_b, stride_sb, C, ldc,
                    strideC, rows, groups, out_dtype, activation, slope, stream=None):
    lib = load()
    return _check(lib, lib.gemm_i8_grouped(M, N, K, _ptr(A), lda, strideA, _ptr(scale_a), stride_sa, _ptr(B), ldb,
                                           strideB, _ptr(scale_b), stride_sb, _ptr(C), ldc, strideC, _ptr(rows),
                                           groups, out_dtype, activation, slope, _stream(stream)))


def tsm_gemm_i8_kernel_name(M, N, K, A, lda, strideA, B, ldb, strideB, C, ldc, strideC, batch, rows, out_dtype):
    r = load().tsm_gemm_i8_kernel_name(M, N, K, _ptr(A), lda, strideA, _ptr(B), ldb, strideB, _ptr(C), ldc, strideC,
                                       batch, _ptr(rows), out_dtype)
    return r.decode() if r else None


def moe_sort(tokens, topk, ids, ld_ids, idtype, experts, capacity, positions, counts, workspace, workspace_bytes,
             stream=None):
    lib = load()
    return _check(lib, lib.moe_sort(tokens, topk, _ptr(ids), ld_ids, idtype, experts, capacity, _ptr(positions),
                                    _ptr(counts), _ptr(workspace), workspace_bytes, _stream(stream)))


def moe_sort_workspace_bytes(tokens, topk, experts):
    return int(load().moe_sort_workspace_bytes(tokens, topk, experts))


def moe_dispatch(tokens, topk, hidden, X, ldx, dtype, scale, positions, slots, slabs, ld_slabs, slab_scale,
                 stream=None):
    lib = load()
    return _check(lib, lib.moe_dispatch(tokens, topk, hidden, _ptr(X), ldx, dtype, _ptr(scale), _ptr(positions), slots,
                                        _ptr(slabs), ld_slabs, _ptr(slab_scale), _stream(stream)))


def moe_combine(tokens, topk, hidden, slabs, ld_slabs, slots, dtype, positions, weights, Y, ldy, stream=None):
    lib = load()
    return _check(lib, lib.moe_combine(tokens, topk, hidden, _ptr(slabs), ld_slabs, slots, dtype, _ptr(positions),
                                       _ptr(weights), _ptr(Y), ldy, _stream(stream)))


def moe_combine_backward(tokens, topk, hidden, dY, lddy, slabs, ld_slabs, slots, dtype, positions, weights, dslabs,
                         ld_dslabs, dweights, stream=None):
    lib = load()
    return _check(lib, lib.moe_combine_backward(tokens, topk, hidden, _ptr(dY), lddy, _ptr(slabs), ld_slabs, slots,
                                                dtype, _ptr(positions), _ptr(weights), _ptr(dslabs), ld_dslabs,
                                                _ptr(dweights), _stream(stream)))


def mx4_quantize(R, C, X, ldx, layout, strideX, xdtype, Q, ldq, strideQ, scale, ld_scale, stride_scale, rows, groups,
                 stream=None):
    lib = load()
    return _check(lib, lib.mx4_quantize(R, C, _ptr(X), ldx, layout, strideX, xdtype, _ptr(Q), ldq, strideQ,
                                        _ptr(scale), ld_scale, stride_scale, _ptr(rows), groups, _stream(stream)))


def mx4_dequantize(R, C, Q, ldq, strideQ, scale, ld_scale, stride_scale, Y, ldy, strideY, ydtype, rows, groups,
                   stream=None):
    lib = load()
    return _check(lib, lib.mx4_dequantize(R, C, _ptr(Q), ldq, strideQ, _ptr(scale), ld_scale, stride_scale, _ptr(Y),
                                          ldy, strideY, ydtype, _ptr(rows), groups, _stream(stream)))


def gemm_mx4(M, N, K, A, lda, scale_a, ld_sa, B, ldb, scale_b, ld_sb, C, ldc, out_dtype, stream=None):
    lib = load()
    return _check(lib, lib.gemm_mx4(M, N, K, _ptr(A), lda, _ptr(scale_a), ld_sa, _ptr(B), ldb, _ptr(scale_b), ld_sb,
                                    _ptr(C), ldc, out_dtype, _stream(stream)))


def gemm_mx4_strided_batched(M, N, K, A, lda, strideA, scale_a, ld_sa, stride_sa, B, ldb, strideB, scale_b, ld_sb,
                             stride_sb, C, ldc, strideC, batch, out_dtype, activation, slope, stream=None):
    lib = load()
    return _check(lib, lib.gemm_mx4_strided_batched(M, N, K, _ptr(A), lda, strideA, _ptr(scale_a), ld_sa, stride_sa,
                                                    _ptr(B), ldb, strideB, _ptr(scale_b), ld_sb, stride_sb, _ptr(C),
                                                    ldc, strideC, batch, out_dtype, activation, slope,
                                                    _stream(stream)))


def gemm_mx4_grouped(M, N, K, A, lda, strideA, scale_a, ld_sa, stride_sa, B, ldb, strideB, scale_b, ld_sb, stride_sb,
                     C, ldc, strideC, rows, groups, out_dtype, activation, slope, stream=None):
    lib = load()
    return _check(lib, lib.gemm_mx4_grouped(M, N, K, _ptr(A), lda, strideA, _ptr(scale_a), ld_sa, stride_sa, _ptr(B),
                                            ldb, strideB, _ptr(scale_b), ld_sb, stride_sb, _ptr(C), ldc, strideC,
                                            _ptr(rows), groups, out_dtype, activation, slope, _stream(stream)))


def gemm_mx4_float_a(M, N, K, X, ldx, strideX, xdtype, B, ldb, strideB, scale_b, ld_sb, stride_sb, C, ldc, strideC,
                     batch, rows, out_dtype, activation, slope, workspace, workspace_bytes, stream=None):
    lib = load()
    return _check(lib, lib.gemm_mx4_float_a(M, N, K, _ptr(X), ldx, strideX, xdtype, _ptr(B), ldb, strideB,
                                            _ptr(scale_b), ld_sb, stride_sb, _ptr(C), ldc, strideC, batch, _ptr(rows),
                                            out_dtype, activation, slope, _ptr(workspace), workspace_bytes,
                                            _stream(stream)))


def gemm_mx4_float_a_workspace_bytes(M, K, batch):
    return int(load().gemm_mx4_float_a_workspace_bytes(M, K, batch))


def tsm_gemm_mx4_kernel_name(M, N, K, A, lda, strideA, scale_a, ld_sa, stride_sa, B, ldb, strideB, scale_b, ld_sb,
                             stride_sb, C, ldc, strideC, batch, rows, out_dtype):
    r = load().tsm_gemm_mx4_kernel_name(M, N, K, _ptr(A), lda, strideA, _ptr(scale_a), ld_sa, stride_sa, _ptr(B), ldb,
                                        strideB, _ptr(scale_b), ld_sb, stride_sb, _ptr(C), ldc, strideC, batch,
                                        _ptr(rows), out_dtype)
    return r.decode() if r else None


def moe_route(tokens, experts, topk, logits, ld_logits, dtype, scores, bias, groups, top_groups, group_best,
              renormalize, factor, ids, weights, stream=None):
    lib = load()
    return _check(lib, lib.moe_route(tokens, experts, topk, _ptr(logits), ld_logits, dtype, scores, _ptr(bias), groups,
                                     top_groups, group_best, renormalize, factor, _ptr(ids), _ptr(weights),
                                     _stream(stream)))


def moe_route_backward(tokens, experts, topk, dweights, logits, ld_logits, dtype, ids, scores, renormalize, factor,
                       dlogits, ld_dlogits, stream=None):
    lib = load()
    return _check(lib, lib.moe_route_backward(tokens, experts, topk, _ptr(dweights), _ptr(logits), ld_logits, dtype,
                                              _ptr(ids), scores, renormalize, factor, _ptr(dlogits), ld_dlogits,
                                              _stream(stream)))
