"""Blocked GEMM for AMD MI355X (gfx950): C = A.B, f16/bf16 in, float32 accumulate.

The C entry points (``include/tsm_gemm.h``) are exposed under the same names
by ``_lib``; ``matmul`` is a convenience wrapper that reads sizes, strides and
layouts off torch tensors and allocates the output with torch.  torch serves
only as device memory and streams: every multiply-add runs in the library's
HIP kernels.
"""

from __future__ import annotations

from ._lib import (TSM_ACT_LEAKY_RELU, TSM_ACT_NONE, TSM_ACT_RELU, TSM_BF16, TSM_BF16_BF16,  # noqa: F401
                   TSM_BF16_F16, TSM_BF16_F32, TSM_COL, TSM_ERROR_INVALID_VALUE, TSM_ERROR_LAUNCH,
                   TSM_ERROR_NOT_SUPPORTED, TSM_F16, TSM_F16_BF16, TSM_F16_F16, TSM_F16_F32, TSM_F32, TSM_I8, TSM_I32,
                   TSM_I64, TSM_ROW, TSM_ROWSUM_BF16, TSM_ROWSUM_F16, TSM_ROWSUM_F32, TSM_SUCCESS, TsmError,
                   _check, _lookups, gemm, gemm_ex, gemm_grouped, gemm_i8, gemm_i8_grouped, gemm_i8_strided_batched,
                   gemm_noalloc_scratch_bytes, gemm_strided_batched, gemm_strided_batched_act, gemm_strided_batched_ex,
                   gemm_strided_batched_noalloc, gemm_strided_batched_ws, gemm_workspace_bytes, load, moe_combine,
                   moe_combine_backward, moe_dispatch, moe_sort, moe_sort_workspace_bytes, quantize_i8, rowsum,
                   tsm_gemm_grouped_kernel_name, tsm_gemm_i8_kernel_name, tsm_gemm_kernel_name,
                   tsm_gemm_ws_kernel_name, tsm_last_error_detail, tsm_rowsum_kernel_name, tsm_status_string)


def dtype_code(in_dtype, out_dtype) -> int:
    import torch

    table = {
        (torch.float16, torch.float32): TSM_F16_F32,
        (torch.float16, torch.float16): TSM_F16_F16,
        (torch.bfloat16, torch.float32): TSM_BF16_F32,
        (torch.bfloat16, torch.float16): TSM_BF16_F16,
        (torch.float16, torch.bfloat16): TSM_F16_BF16,
        (torch.bfloat16, torch.bfloat16): TSM_BF16_BF16,
    }
    try:
        return table[(in_dtype, out_dtype)]
    except KeyError:
        raise TsmError(TSM_ERROR_INVALID_VALUE, f"unsupported dtypes {in_dtype} -> {out_dtype}") from None


def _layout(t, rows_dim_size, cols_dim_size):
    """(layout, ld) of the last two dims of a logical rows x cols tensor view."""
    s_r, s_c = t.stride(-2), t.stride(-1)
    if s_c == 1 and (s_r >= max(1, cols_dim_size) or rows_dim_size <= 1):
        return TSM_ROW, max(s_r, max(1, cols_dim_size))
    if s_r == 1 and (s_c >= max(1, rows_dim_size) or cols_dim_size <= 1):
        return TSM_COL, max(s_c, max(1, rows_dim_size))
    raise TsmError(TSM_ERROR_INVALID_VALUE, "operand must be row- or column-major in its last two dims")


_ACTIVATIONS = {None: TSM_ACT_NONE, "relu": TSM_ACT_RELU, "leaky_relu": TSM_ACT_LEAKY_RELU}


def workspace_for(a, b):
    """A float32 CUDA tensor big enough for ``matmul(a, b, workspace=...)`` to split K, or None when the shape
    does not split.  Allocate it once and reuse it across calls of that shape on one stream."""
    import torch

    M, K, N = a.shape[-2], a.shape[-1], b.shape[-1]
    batch = max(a.shape[0] if a.dim() == 3 else 1, b.shape[0] if b.dim() == 3 else 1)
    nbytes = gemm_workspace_bytes(M, N, K, batch)
    return torch.empty((nbytes + 3) // 4, dtype=torch.float32, device=a.device) if nbytes else None


def matmul(a, b, *, out=None, out_dtype=None, activation=None, slope=0.01, workspace=None, stream=None):
    """C = act(A.B) for CUDA tensors ``a`` (..., M, K) and ``b`` (..., K, N) in float16 or bfloat16.

    2-D operands give one product, 3-D ones a strided batch (a batch dim of
    size 1 or stride 0 broadcasts).  Each operand may be row-major or
    column-major in its last two dims (e.g. ``w.t()``); the result is row-major
    float32 (default), float16 or bfloat16.  ``activation`` is None, "relu" or
    "leaky_relu" (with ``slope``), fused into the kernels' epilogue.  With a
    ``workspace`` (see ``workspace_for``) products with few output tiles and
    deep K split K through it.  On a ``stream`` other than the current one give
    ``out``: a result allocated here is memory of the current stream.
    """
    import torch

    if a.dtype != b.dtype:
        raise TsmError(TSM_ERROR_INVALID_VALUE, "a and b must share a dtype")
    out_dtype = out_dtype or (out.dtype if out is not None else torch.float32)
    code = dtype_code(a.dtype, out_dtype)
    M, K = a.shape[-2], a.shape[-1]
    K2, N = b.shape[-2], b.shape[-1]
    if K != K2:
        raise TsmError(TSM_ERROR_INVALID_VALUE, f"inner sizes differ: {K} vs {K2}")
    batched = a.dim() == 3 or b.dim() == 3
    batch = max(a.shape[0] if a.dim() == 3 else 1, b.shape[0] if b.dim() == 3 else 1)
    if out is None:
        out = torch.empty((batch, M, N) if batched else (M, N), dtype=out_dtype, device=a.device)
    la, lda = _layout(a, M, K)
    lb, ldb = _layout(b, K, N)
    if out.stride(-1) != 1:
        raise TsmError(TSM_ERROR_INVALID_VALUE, "out must be row-major")
    ldc = out.stride(-2) if M > 1 else max(1, N)

    def bstride(t):
        return 0 if t.dim() == 2 or t.shape[0] == 1 else t.stride(0)

    if activation not in _ACTIVATIONS:
        raise TsmError(TSM_ERROR_INVALID_VALUE, f"unknown activation {activation!r}")
    ws_bytes = workspace.numel() * workspace.element_size() if workspace is not None else 0
    gemm_strided_batched_ws(M, N, K, a, lda, la, bstride(a), b, ldb, lb, bstride(b), out, ldc,
                            out.stride(0) if out.dim() == 3 else 0, batch, code, _ACTIVATIONS[activation], slope,
                            workspace, ws_bytes, stream)
    return out


# ---- int8 products and expert routing --------------------------------------------------------------------------
#
# ``stream`` (a torch stream or its handle): None is the current stream of the tensors' GPU.  What a call given one
# allocates is memory of that stream, as inside ``torch.cuda.stream``: another stream waits for it before it uses the
# result, and ``record_stream`` tells torch of that use.
#
# No function here records anything for autograd: results never require a gradient, whatever the inputs do.  Training
# calls the ``_backward`` functions, for instance from a ``torch.autograd.Function`` of the model's own.


def _bad(text):
    raise TsmError(TSM_ERROR_INVALID_VALUE, text)


_FORMATS = {}


def _formats():
    """The library's codes (TSM_F32 .. TSM_I64) by torch dtype."""
    if not _FORMATS:
        import torch

        _FORMATS.update({torch.float32: TSM_F32, torch.float16: TSM_F16, torch.bfloat16: TSM_BF16, torch.int8: TSM_I8,
                         torch.int32: TSM_I32, torch.int64: TSM_I64})
    return _FORMATS


def _wants(what, t, formats, shape=None):
    """Check a tensor argument: of one of the formats, of the shape.  Returns its format."""
    f = (_FORMATS or _formats()).get(t.dtype)
    if f not in formats:
        _bad(f"{what} has dtype {t.dtype}")
    if shape is not None and t.shape != shape:
        _bad(f"{what} has shape {tuple(t.shape)}, {tuple(shape)} wanted")
    return f


def _rows_ld(what, t):
    """Leading dimension of the last two dims of a tensor whose rows are contiguous."""
    if t.numel() == 0:
        return max(1, t.shape[-1])
    if t.shape[-1] > 1 and t.stride(-1) != 1:
        _bad(f"{what}: rows must be contiguous")
    return t.stride(-2) if t.shape[-2] > 1 else max(1, t.shape[-1])


def _packed(what, t):
    if not t.is_contiguous():
        _bad(f"{what} must be contiguous")


def _under(stream, d):
    """Context in which torch allocates and fills for a call on ``stream`` (a torch stream or its handle) of GPU d."""
    import torch

    if isinstance(stream, torch.cuda.Stream):
        return torch.cuda.stream(stream)
    handle = stream if isinstance(stream, int) else stream.cuda_stream
    # (a handle of 0 would make ExternalStream take a stream of torch's pool)
    return torch.cuda.stream(torch.cuda.ExternalStream(handle, device=d) if handle else torch.cuda.default_stream(d))


def _new(like, shape, dtype, stream, fill=None):
    """A tensor of a dtype (torch's, or its name) on the GPU of ``like``, zeros with ``fill``.  With a stream it is that
    stream's memory, and the zeros are written there: on the current stream nothing would order them, or work that
    still uses the block's last tensor, before the call."""
    import torch

    dtype = getattr(torch, dtype) if isinstance(dtype, str) else dtype
    make = torch.zeros if fill else torch.empty
    if stream is None:
        return make(shape, dtype=dtype, device=like.device)
    d = like.get_device()
    if d < 0:
        _bad("tensors must be on a GPU (the first is not on a GPU)")
    with _under(stream, d):
        return make(shape, dtype=dtype, device=like.device)


def _at(t):
    return None if t is None else t.data_ptr()


def _launch(call, stream, tensors, args):
    """call(*args, stream) through the C interface, the GPU of the tensors (None among them: not given) current: they
    must all be on one.  Without a stream, its current one.  A small operator's time is this path (3.9 us are the
    launch itself), so it goes to the library without the checks and conversions of the functions in _lib."""
    d = tensors[0].get_device()
    if d < 0:
        _bad("tensors must be on a GPU (the first is not on a GPU)")
    for t in tensors:
        if t is not None and t.get_device() != d:
            _bad(f"tensors on {tensors[0].device} and {t.device}")
    lib = load()
    device, current_stream = _lookups()
    if stream is None:
        stream = current_stream(d)
    elif not isinstance(stream, int):
        stream = stream.cuda_stream
    if d == device():
        status = getattr(lib, call)(*args, stream)
    else:
        import torch

        with torch.cuda.device(d):
            status = getattr(lib, call)(*args, stream)
    if status:
        _check(lib, status)


_FLOATS = (TSM_F32, TSM_F16, TSM_BF16)


def quantize(x, *, rows=None, out=None, scale=None, stream=None):
    """(codes, scales) of the rows of ``x`` (..., R, C) in float32, float16 or bfloat16: int8 codes with
    ``x ~ codes * scales[..., None]``, the scales float32 of shape (..., R).

    2-D or 3-D.  With ``rows`` (int32, one count per matrix of a 3-D ``x``, on the GPU) only the first rows of each
    are read and written.
    """
    if x.dim() not in (2, 3):
        _bad("x must be 2-D or 3-D")
    f = _wants("x", x, _FLOATS)
    if out is None:
        out = _new(x, x.shape, "int8", stream)
    if scale is None:
        scale = _new(x, x.shape[:-1], "float32", stream)
    _wants("out", out, (TSM_I8,), x.shape)
    _wants("scale", scale, (TSM_F32,), x.shape[:-1])
    G = x.shape[0] if x.dim() == 3 else 1
    if rows is not None:
        _wants("rows", rows, (TSM_I32,), (G,))
        _packed("rows", rows)
    if scale.shape[-1] > 1 and scale.stride(-1) != 1:
        _bad("scale: rows must be contiguous")
    ldx, ldq = _rows_ld("x", x), _rows_ld("out", out)
    sx, sq, ss = (x.stride(0), out.stride(0), scale.stride(0)) if x.dim() == 3 else (0, 0, 0)
    _launch("quantize_i8", stream, (x, out, scale, rows),
            (x.shape[-2], x.shape[-1], x.data_ptr(), ldx, sx, f, out.data_ptr(), ldq, sq, scale.data_ptr(), ss,
             _at(rows), G))
    return out, scale


def matmul_i8(a, scale_a, b, scale_b, *, rows=None, out=None, out_dtype=None, activation=None, slope=0.01, stream=None):
    """C = act(scale_a[..., None] * scale_b * (A.B)) for int8 CUDA tensors ``a`` (..., M, K) and ``b`` (..., K, N).

    ``a`` has contiguous rows and ``b`` is column-major (``w.t()`` of a weight stored N x K).  ``scale_a`` (..., M) and
    ``scale_b`` (..., N) are float32 (None: ones).  2-D operands give one product, 3-D ones a strided batch (a batch
    dim of size 1 broadcasts); with ``rows`` (int32 counts on the GPU, one per problem) the grouped product over a
    mixture of experts' slabs.  The result is float32 (default), float16 or bfloat16; ``activation`` as for ``matmul``,
    but a NaN stays NaN.
    """
    if a.dim() not in (2, 3) or b.dim() not in (2, 3):
        _bad("a and b must be 2-D or 3-D")
    _wants("a", a, (TSM_I8,))
    _wants("b", b, (TSM_I8,))
    M, K = a.shape[-2], a.shape[-1]
    K2, N = b.shape[-2], b.shape[-1]
    if K != K2:
        _bad(f"inner sizes differ: {K} vs {K2}")
    batched = a.dim() == 3 or b.dim() == 3
    ba, bb = (a.shape[0] if a.dim() == 3 else 1), (b.shape[0] if b.dim() == 3 else 1)
    if ba != bb and ba != 1 and bb != 1:
        _bad(f"batch sizes differ: {ba} vs {bb}")
    batch = ba if bb == 1 else bb
    shape = (batch, M, N) if batched else (M, N)
    if out is None:
        out = _new(a, shape, out_dtype or "float32", stream)
    elif out_dtype is not None and out.dtype != out_dtype:
        _bad(f"out has dtype {out.dtype}, out_dtype is {out_dtype}")
    f = _wants("out", out, _FLOATS, shape)
    if activation not in _ACTIVATIONS:
        _bad(f"unknown activation {activation!r}")

    def scales(what, t, op, n):
        """Batch stride of an operand's scales."""
        if t is None:
            return 0
        _wants(what, t, (TSM_F32,), (*op.shape[:-2], n))
        if n > 1 and t.stride(-1) != 1:
            _bad(f"{what}: scales must be contiguous")
        return t.stride(0) if t.dim() == 2 and t.shape[0] > 1 else 0

    ssa, ssb = scales("scale_a", scale_a, a, M), scales("scale_b", scale_b, b, N)
    if N > 0 and K > 1 and b.stride(-2) != 1:
        _bad("b must be column-major (the transpose of a weight stored N x K)")
    lda, ldb, ldc = _rows_ld("a", a), _rows_ld("b", b.transpose(-1, -2)), _rows_ld("out", out)
    sa, sb = (a.stride(0) if ba > 1 else 0), (b.stride(0) if bb > 1 else 0)
    sc = out.stride(0) if batched else 0
    act = _ACTIVATIONS[activation]
    if rows is None:
        _launch("gemm_i8_strided_batched", stream, (a, b, out, scale_a, scale_b),
                (M, N, K, a.data_ptr(), lda, sa, _at(scale_a), ssa, b.data_ptr(), ldb, sb, _at(scale_b), ssb,
                 out.data_ptr(), ldc, sc, batch, f, act, slope))
    else:
        _wants("rows", rows, (TSM_I32,), (batch,))
        _packed("rows", rows)
        _launch("gemm_i8_grouped", stream, (a, b, out, scale_a, scale_b, rows),
                (M, N, K, a.data_ptr(), lda, sa, _at(scale_a), ssa, b.data_ptr(), ldb, sb, _at(scale_b), ssb,
                 out.data_ptr(), ldc, sc, rows.data_ptr(), batch, f, act, slope))
    return out


def sort_workspace_for(ids, experts):
    """A CUDA tensor for ``sort_tokens(..., workspace=...)``, or None when the sizes need none."""
    n = moe_sort_workspace_bytes(ids.shape[0], ids.shape[1], experts)
    return _new(ids, (n,), "uint8", None) if n else None


def sort_tokens(ids, experts, capacity, *, positions=None, counts=None, workspace=None, stream=None):
    """(positions, counts) of the experts' ids (tokens, topk), int32 or int64: the row of each choice in the slabs
    (experts * capacity rows, expert e's from e * capacity), in token order, -1 for an id outside [0, experts) or past
    the capacity; and how many choices each expert got (int32, those past the capacity among them).

    A workspace (see ``sort_workspace_for``) is allocated when the sizes need one and none is given, for calls on the
    current stream.
    """
    if ids.dim() != 2:
        _bad("ids must be 2-D")
    f = _wants("ids", ids, (TSM_I32, TSM_I64))
    if positions is None:
        positions = _new(ids, ids.shape, "int32", stream)
    if counts is None:
        counts = _new(ids, (experts,), "int32", stream)
    _wants("positions", positions, (TSM_I32,), ids.shape)
    _wants("counts", counts, (TSM_I32,), (experts,))
    _packed("positions", positions)
    _packed("counts", counts)
    if workspace is None:
        workspace = sort_workspace_for(ids, experts)
        if workspace is not None and stream is not None:
            # memory of the current stream, which would take it back before the other stream is done with it
            _bad("a call on a stream of its own needs its workspace (see sort_workspace_for)")
    nbytes = 0
    if workspace is not None:
        _packed("workspace", workspace)
        nbytes = workspace.numel() * workspace.element_size()
    _launch("moe_sort", stream, (ids, positions, counts, workspace),
            (ids.shape[0], ids.shape[1], ids.data_ptr(), _rows_ld("ids", ids), f, experts, capacity,
             positions.data_ptr(), counts.data_ptr(), _at(workspace), nbytes))
    return positions, counts


def _slab_args(what, slabs, positions, tokens, hidden):
    """Check 2-D slabs (slots, hidden) and the positions (tokens, topk)."""
    if slabs.dim() != 2 or (hidden is not None and slabs.shape[1] != hidden):
        _bad(f"{what} must be 2-D with {hidden} columns")
    if positions.dim() != 2 or (tokens is not None and positions.shape[0] != tokens):
        _bad(f"positions must be 2-D with {tokens} rows")
    _wants("positions", positions, (TSM_I32,))
    _packed("positions", positions)


def dispatch_tokens(x, positions, *, slots=None, out=None, scale=None, out_scale=None, stream=None):
    """Token rows ``x`` (tokens, hidden) at their ``positions`` (tokens, topk) in the slabs (slots, hidden), float32,
    float16, bfloat16 or int8.

    ``out`` keeps its other rows; without it the slabs are allocated with ``slots`` rows (the others unset).  With
    ``scale`` (float32, one per token) also the slab rows' scales: returns (slabs, scales).

    Not recorded for autograd: the gradient of ``x`` is ``dispatch_tokens_backward``.
    """
    if x.dim() != 2:
        _bad("x must be 2-D")
    f = _wants("x", x, _FLOATS + (TSM_I8,))
    if out is None:
        if slots is None:
            _bad("slots or out is needed")
        out = _new(x, (slots, x.shape[1]), x.dtype, stream)
    elif slots is not None and out.shape[0] != slots:
        _bad(f"out has {out.shape[0]} rows, slots is {slots}")
    _slab_args("out", out, positions, x.shape[0], x.shape[1])
    _wants("out", out, (f,))
    if scale is not None:
        _wants("scale", scale, (TSM_F32,), (x.shape[0],))
        _packed("scale", scale)
        if out_scale is None:
            out_scale = _new(x, (out.shape[0],), "float32", stream)
        _wants("out_scale", out_scale, (TSM_F32,), (out.shape[0],))
        _packed("out_scale", out_scale)
    elif out_scale is not None:
        _bad("out_scale without scale")
    _launch("moe_dispatch", stream, (x, out, positions, scale, out_scale),
            (x.shape[0], positions.shape[1], x.shape[1], x.data_ptr(), _rows_ld("x", x), f, _at(scale),
             positions.data_ptr(), out.shape[0], out.data_ptr(), _rows_ld("out", out), _at(out_scale)))
    return out if scale is None else (out, out_scale)


def combine_tokens(slabs, positions, weights=None, *, out=None, stream=None):
    """Y[t] = sum_j weights[t, j] * slabs[positions[t, j]] over the choices with a position, float32 sums in the order
    of j; ``weights`` float32 (tokens, topk), None for ones.  Y has the slabs' dtype (float32, float16 or bfloat16).

    Not recorded for autograd: the gradients of ``slabs`` and ``weights`` are ``combine_tokens_backward``.
    """
    _slab_args("slabs", slabs, positions, None, None)
    f = _wants("slabs", slabs, _FLOATS)
    tokens, hidden = positions.shape[0], slabs.shape[1]
    if out is None:
        out = _new(slabs, (tokens, hidden), slabs.dtype, stream)
    _wants("out", out, (f,), (tokens, hidden))
    if weights is not None:
        _wants("weights", weights, (TSM_F32,), positions.shape)
        _packed("weights", weights)
    _launch("moe_combine", stream, (slabs, out, positions, weights),
            (tokens, positions.shape[1], hidden, slabs.data_ptr(), _rows_ld("slabs", slabs), slabs.shape[0], f,
             positions.data_ptr(), _at(weights), out.data_ptr(), _rows_ld("out", out)))
    return out


def dispatch_tokens_backward(dslabs, positions, *, out=None, stream=None):
    """Gradient of ``dispatch_tokens`` with respect to ``x``: dX[t] = sum_j dslabs[positions[t, j]]."""
    return combine_tokens(dslabs, positions, None, out=out, stream=stream)


def combine_tokens_backward(dy, slabs, positions, weights=None, *, out=None, dweights=None, stream=None):
    """(dslabs, dweights) of ``combine_tokens`` from ``dy`` (tokens, hidden): dslabs[positions[t, j]] =
    weights[t, j] * dy[t] (``out``; its other rows are kept, or zeros where it is allocated here) and
    dweights[t, j] = <dy[t], slabs[positions[t, j]]> (float32, 0 without a position)."""
    if dy.dim() != 2:
        _bad("dy must be 2-D")
    f = _wants("dy", dy, _FLOATS)
    _slab_args("slabs", slabs, positions, dy.shape[0], dy.shape[1])
    _wants("slabs", slabs, (f,))
    if out is None:
        out = _new(slabs, slabs.shape, slabs.dtype, stream, fill=True)
    _wants("out", out, (f,), slabs.shape)
    if dweights is None:
        dweights = _new(dy, positions.shape, "float32", stream)
    _wants("dweights", dweights, (TSM_F32,), positions.shape)
    _packed("dweights", dweights)
    if weights is not None:
        _wants("weights", weights, (TSM_F32,), positions.shape)
        _packed("weights", weights)
    _launch("moe_combine_backward", stream, (dy, slabs, out, positions, weights, dweights),
            (dy.shape[0], positions.shape[1], dy.shape[1], dy.data_ptr(), _rows_ld("dy", dy), slabs.data_ptr(),
             _rows_ld("slabs", slabs), slabs.shape[0], f, positions.data_ptr(), _at(weights), out.data_ptr(),
             _rows_ld("out", out), dweights.data_ptr()))
    return out, dweights
