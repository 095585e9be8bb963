"""Operators of a transformer's feed-forward half layer, on torch tensors.

Layer norm, the gated projections h = act(x Wg^T) * (x Wu^T), both with their
backward passes, the quantisation of activations row by row and the 8-bit
integer product.  Argument checks and marshalling only: the work is done by the
kernels behind include/gemm_relu_ffn.h, and there is no CPU or PyTorch fallback.

Activations are matrices of rows: any shape whose last dimension is the row, if
contiguous, or 2-D with contiguous rows any distance apart.  Results are new
contiguous tensors.  The kernels run on ``stream`` (a torch.cuda.Stream, a raw
hipStream_t, or None for torch's current stream); results and workspaces are
allocated for that stream.  A tensor made on another stream has to be ready
before the call, as with any torch operation.
"""
import contextlib
import ctypes

ACTIVATIONS = {"silu": 0, "gelu": 1, "gelu_tanh": 2, "relu": 3}

_vp, _i64, _int, _u64 = ctypes.c_void_p, ctypes.c_int64, ctypes.c_int, ctypes.c_uint64
_SIGNATURES = {
    "gemm_relu_layer_norm": ([_vp, _i64, _vp, _vp, _vp, _vp, _vp, _i64, _i64, _int, _int,
                              ctypes.c_float, _vp], _int),
    "gemm_relu_layer_norm_backward_workspace": ([_i64, _i64], _i64),
    "gemm_relu_layer_norm_backward": ([_vp, _i64, _vp, _i64, _vp, _vp, _vp, _vp, _vp, _vp, _i64,
                                       _i64, _int, _int, _vp, _u64, _vp], _int),
    "gemm_relu_gated": ([_vp, _i64, _vp, _i64, _vp, _vp, _i64, _i64, _i64, _int, _int, _vp], _int),
    "gemm_relu_gated_plan": ([_i64, _i64, _i64, _int], ctypes.c_char_p),
    "gemm_relu_gated_backward_workspace": ([_i64, _i64, _i64], _i64),
    "gemm_relu_gated_backward": ([_vp, _i64, _vp, _vp, _i64, _vp, _i64, _vp, _vp, _i64, _i64,
                                  _i64, _int, _int, _vp, _u64, _vp], _int),
    "gemm_relu_gated_backward_plan": ([_i64, _i64, _i64, _int], ctypes.c_char_p),
    "gemm_relu_quantize_rows": ([_vp, _i64, _vp, _vp, _i64, _i64, _int, _vp], _int),
    "gemm_relu_i8": ([_vp, _i64, _vp, _vp, _i64, _vp, _vp, _i64, _i64, _i64, _int, _vp], _int),
    "gemm_relu_i8_plan": ([_i64, _i64, _i64, _int], ctypes.c_char_p),
}


def declare(lib):
    """Argument and result types of the functions of include/gemm_relu_ffn.h."""
    for name, (args, res) in _SIGNATURES.items():
        fn = getattr(lib, name)
        fn.argtypes, fn.restype = args, res


def _library():
    from . import library
    return library()


def _codes():
    import torch
    return {torch.float16: 0, torch.bfloat16: 1, torch.float32: 2}


def _check(status):
    if status:
        from . import GemmReluError, gemm_relu_strerror
        raise GemmReluError(status, gemm_relu_strerror(status))


def _rows(t, name):
    """(rows, columns, elements from row to row) of an activation tensor."""
    if t.dim() < 1:
        raise ValueError("%s must have at least one dimension" % name)
    cols = t.shape[-1]
    if t.is_contiguous():
        rows = 1
        for n in t.shape[:-1]:
            rows *= n
        return rows, cols, cols
    if t.dim() == 2 and t.stride(1) == 1 and t.stride(0) >= cols:
        return t.shape[0], cols, t.stride(0)
    raise ValueError("%s must be contiguous, or 2-D with contiguous rows" % name)


def _weight(t, name):
    if t.dim() != 2:
        raise ValueError("%s must be 2-D" % name)
    return _rows(t, name)


def _vector(t, name, n, dtypes):
    if t.dtype not in dtypes:
        raise TypeError("%s must be %s, not %s" % (name, " or ".join(map(str, dtypes)), t.dtype))
    if t.numel() != n or not t.is_contiguous():
        raise ValueError("%s must be contiguous with %d elements" % (name, n))


def _one_gpu(first, *others):
    if not first.is_cuda or any(t is not None and t.device != first.device for t in others):
        raise ValueError("all tensors must be on the same GPU")


@contextlib.contextmanager
def _on(device, stream):
    """Makes `device` and `stream` current for the allocations and the launch
    inside; gives the raw stream."""
    import torch
    with torch.cuda.device(device):
        if stream is None:
            yield torch.cuda.current_stream().cuda_stream
            return
        if isinstance(stream, int):
            stream = torch.cuda.ExternalStream(stream, device=device)
        with torch.cuda.stream(stream):
            yield stream.cuda_stream


def _workspace(nbytes, device):
    import torch
    return torch.empty(nbytes, dtype=torch.uint8, device=device)


def layer_norm(x, weight, bias=None, eps=1e-5, stats=False, stream=None):
    """Layer norm over the last dimension: (x - mean) * rstd * weight + bias.

    x: float16, bfloat16 or float32; weight and bias (or None): x's type or
    float32.  Returns y, or with ``stats`` (y, mean, rstd), the fp32 statistics
    of each row that the backward pass takes.
    """
    import torch
    codes = _codes()
    if x.dtype not in codes:
        raise TypeError("x must be float16, bfloat16 or float32, not %s" % x.dtype)
    rows, cols, ld = _rows(x, "x")
    _vector(weight, "weight", cols, (x.dtype, torch.float32))
    if bias is not None:
        _vector(bias, "bias", cols, (weight.dtype,))
    _one_gpu(x, weight, bias)
    with _on(x.device, stream) as st:
        y = torch.empty(x.shape, dtype=x.dtype, device=x.device)
        mean = rstd = None
        if stats:
            mean, rstd = (torch.empty(x.shape[:-1], dtype=torch.float32, device=x.device) for _ in range(2))
        _check(_library().gemm_relu_layer_norm(
            x.data_ptr(), ld, weight.data_ptr(), None if bias is None else bias.data_ptr(), y.data_ptr(),
            mean.data_ptr() if stats else None, rstd.data_ptr() if stats else None, rows, cols,
            codes[x.dtype], codes[weight.dtype], eps, st))
    return (y, mean, rstd) if stats else y


def layer_norm_backward(dy, x, weight, mean, rstd, stream=None):
    """Gradients (dx, dweight, dbias) of layer_norm, given dy and the statistics
    of the forward call.  dx has x's type, dweight and dbias weight's."""
    import torch
    codes = _codes()
    if x.dtype not in codes:
        raise TypeError("x must be float16, bfloat16 or float32, not %s" % x.dtype)
    if dy.dtype != x.dtype:
        raise TypeError("dy must have x's type")
    if dy.shape != x.shape:
        raise ValueError("dy and x must have the same shape")
    rows, cols, ld = _rows(x, "x")
    dy_ld = _rows(dy, "dy")[2]
    _vector(weight, "weight", cols, (x.dtype, torch.float32))
    _vector(mean, "mean", rows, (torch.float32,))
    _vector(rstd, "rstd", rows, (torch.float32,))
    _one_gpu(x, dy, weight, mean, rstd)
    lib = _library()
    with _on(x.device, stream) as st:
        dx = torch.empty(x.shape, dtype=x.dtype, device=x.device)
        dw, db = torch.empty_like(weight), torch.empty_like(weight)
        ws = _workspace(lib.gemm_relu_layer_norm_backward_workspace(rows, cols), x.device)
        _check(lib.gemm_relu_layer_norm_backward(
            dy.data_ptr(), dy_ld, x.data_ptr(), ld, weight.data_ptr(), mean.data_ptr(), rstd.data_ptr(),
            dx.data_ptr(), dw.data_ptr(), db.data_ptr(), rows, cols, codes[x.dtype], codes[weight.dtype],
            ws.data_ptr(), ws.numel(), st))
    return dx, dw, db


def _gated_args(x, weight, act):
    import torch
    if act not in ACTIVATIONS:
        raise ValueError("act must be one of %s" % ", ".join(sorted(ACTIVATIONS)))
    if x.dtype not in (torch.float16, torch.bfloat16) or weight.dtype != x.dtype:
        raise TypeError("x and weight must share dtype float16 or bfloat16")
    rows, cols, ld = _rows(x, "x")
    wrows, wcols, wld = _weight(weight, "weight")
    if wcols != cols or wrows % 2:
        raise ValueError("weight must be (2 * hidden, %d), gate rows first" % cols)
    return rows, cols, ld, wrows // 2, wld


def matmul_gated(x, weight, act="silu", save=False, stream=None):
    """Gated projections h = act(x Wg^T) * (x Wu^T).

    x: (..., cols) float16 or bfloat16; weight: (2 * hidden, cols), the gate's
    rows Wg first, then Wu.  act: "silu", "gelu", "gelu_tanh" or "relu".  Returns
    h (..., hidden), or with ``save`` (h, gu): gu (..., 2 * hidden) holds the
    fp32 sums x Wg^T and x Wu^T for matmul_gated_backward (in 16 bits their
    rounding would be as large as that of the gradients themselves).
    """
    import torch
    rows, cols, ld, hidden, wld = _gated_args(x, weight, act)
    _one_gpu(x, weight)
    with _on(x.device, stream) as st:
        h = torch.empty(x.shape[:-1] + (hidden,), dtype=x.dtype, device=x.device)
        gu = torch.empty(x.shape[:-1] + (2 * hidden,), dtype=torch.float32, device=x.device) if save else None
        _check(_library().gemm_relu_gated(x.data_ptr(), ld, weight.data_ptr(), wld, h.data_ptr(),
                                          gu.data_ptr() if save else None, rows, hidden, cols,
                                          _codes()[x.dtype], ACTIVATIONS[act], st))
    return (h, gu) if save else h


def matmul_gated_backward(dh, gu, x, weight, act="silu", stream=None):
    """Gradients (dx, dweight) of matmul_gated, given dh and the forward call's
    gu.  Both have x's type."""
    import torch
    rows, cols, ld, hidden, wld = _gated_args(x, weight, act)
    if dh.dtype != x.dtype:
        raise TypeError("dh must have x's type")
    if dh.shape != x.shape[:-1] + (hidden,):
        raise ValueError("dh must have matmul_gated's shape %s" % (tuple(x.shape[:-1]) + (hidden,),))
    dh_ld = _rows(dh, "dh")[2]
    _vector(gu, "gu", rows * 2 * hidden, (torch.float32,))
    _one_gpu(x, weight, dh, gu)
    lib = _library()
    with _on(x.device, stream) as st:
        dx = torch.empty(x.shape, dtype=x.dtype, device=x.device)
        dw = torch.empty(weight.shape, dtype=x.dtype, device=x.device)
        ws = _workspace(lib.gemm_relu_gated_backward_workspace(rows, hidden, cols), x.device)
        _check(lib.gemm_relu_gated_backward(
            dh.data_ptr(), dh_ld, gu.data_ptr(), x.data_ptr(), ld, weight.data_ptr(), wld, dx.data_ptr(),
            dw.data_ptr(), rows, hidden, cols, _codes()[x.dtype], ACTIVATIONS[act], ws.data_ptr(),
            ws.numel(), st))
    return dx, dw


def quantize_rows(x, stream=None):
    """Each row (last dimension) of x in 8 bits: returns (q, scale), int8 q of x's
    shape and fp32 scale = max|row| / 127, with row ~ q * scale.  A row that holds
    an infinity or NaN has scale NaN."""
    import torch
    codes = _codes()
    if x.dtype not in codes:
        raise TypeError("x must be float16, bfloat16 or float32, not %s" % x.dtype)
    rows, cols, ld = _rows(x, "x")
    _one_gpu(x)
    with _on(x.device, stream) as st:
        q = torch.empty(x.shape, dtype=torch.int8, device=x.device)
        scale = torch.empty(x.shape[:-1], dtype=torch.float32, device=x.device)
        _check(_library().gemm_relu_quantize_rows(x.data_ptr(), ld, q.data_ptr(), scale.data_ptr(), rows, cols,
                                                  codes[x.dtype], st))
    return q, scale


def matmul_i8(x, x_scale, weight, weight_scale, out_dtype=None, stream=None):
    """8-bit integer product y = (x weight^T) * x_scale[..., None] * weight_scale.

    x: (..., k) int8 with one fp32 scale per row; weight: (n, k) int8 with one
    fp32 scale per row (output channel).  Sums are exact (k <= 131071).  Returns
    y (..., n) of out_dtype (float16, bfloat16 or float32; default bfloat16).
    """
    import torch
    codes = _codes()
    out_dtype = torch.bfloat16 if out_dtype is None else out_dtype
    if x.dtype != torch.int8 or weight.dtype != torch.int8:
        raise TypeError("x and weight must be int8")
    if out_dtype not in codes:
        raise TypeError("out_dtype must be float16, bfloat16 or float32, not %s" % out_dtype)
    rows, k, ld = _rows(x, "x")
    n, wk, wld = _weight(weight, "weight")
    if wk != k:
        raise ValueError("inner dimensions differ: %d vs %d" % (k, wk))
    _vector(x_scale, "x_scale", rows, (torch.float32,))
    _vector(weight_scale, "weight_scale", n, (torch.float32,))
    _one_gpu(x, x_scale, weight, weight_scale)
    with _on(x.device, stream) as st:
        y = torch.empty(x.shape[:-1] + (n,), dtype=out_dtype, device=x.device)
        _check(_library().gemm_relu_i8(x.data_ptr(), ld, x_scale.data_ptr(), weight.data_ptr(), wld,
                                       weight_scale.data_ptr(), y.data_ptr(), rows, n, k, codes[out_dtype], st))
    return y
