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


class _Env:
    """What every call needs of torch and the library, looked up once: a call's
    own cost on the host is that of a short kernel."""

    def __init__(self):
        import torch
        from . import library
        self.codes = {torch.float16: 0, torch.bfloat16: 1, torch.float32: 2}
        self.torch, self.lib = torch, library()
        self.empty_like, self.f32, self.i8, self.u8 = torch.empty_like, torch.float32, torch.int8, torch.uint8
        self.current_device = torch._C._cuda_getDevice
        self.raw_stream = torch._C._cuda_getCurrentRawStream


_env = None


def _get_env():
    global _env
    if _env is None:
        _env = _Env()
    return _env


def _check(status):
    if status:
        from . import GemmReluError, gemm_relu_strerror
        raise GemmReluError(status, gemm_relu_strerror(status))


def _rows(t, name):
    """(rows, columns, elements from row to row) of an activation tensor."""
    shape = t.shape
    if len(shape) == 2:
        rows, cols = shape
        if t.is_contiguous():
            return rows, cols, cols
        ld, one = t.stride()
        if one == 1 and ld >= cols:
            return rows, cols, ld
    elif len(shape) == 0:
        raise ValueError("%s must have at least one dimension" % name)
    elif t.is_contiguous():
        cols = shape[-1]
        rows = 1
        for n in shape[:-1]:
            rows *= n
        return rows, cols, cols
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


def _one_gpu(*tensors):
    """The index of the GPU that holds all of the tensors."""
    index = tensors[0].get_device()
    for t in tensors:
        if t.get_device() != index or index < 0:
            raise ValueError("all tensors must be on the same GPU")
    return index


def _elsewhere(index, stream, inputs, fn, *args):
    """fn(*args) with GPU `index` and `stream` current, for its allocations and
    its launches."""
    cuda = _get_env().torch.cuda
    with cuda.device(index):
        if stream is None:
            return fn(*args)
        if isinstance(stream, int):
            stream = cuda.ExternalStream(stream, device=index)
        with cuda.stream(stream):
            out = fn(*args)
        # the caller may drop an input while the stream still reads it
        for t in inputs:
            t.record_stream(stream)
        return out


def layer_norm(x, weight, bias=None, eps=1e-5, stats=False, stream=None):
    """Layer norm over the last dimension: (x - mean) * rstd * weight + bias.

    x: float16, bfloat16 or float32; weight and bias (or None): x's type or
    float32.  Returns y, or with ``stats`` (y, mean, rstd), the fp32 statistics
    of each row that the backward pass takes.
    """
    env = _get_env()
    codes, dt = env.codes, x.dtype
    if dt not in codes:
        raise TypeError("x must be float16, bfloat16 or float32, not %s" % dt)
    rows, cols, ld = _rows(x, "x")
    wdt = weight.dtype
    _vector(weight, "weight", cols, (dt, env.f32))
    if bias is None:
        inputs = (x, weight)
    else:
        _vector(bias, "bias", cols, (wdt,))
        inputs = (x, weight, bias)
    index = _one_gpu(*inputs)
    if stream is not None or env.current_device() != index:
        return _elsewhere(index, stream, inputs, layer_norm, x, weight, bias, eps, stats)
    y = env.empty_like(x) if ld == cols else x.new_empty(x.shape)
    mean = rstd = None
    if stats:
        mean, rstd = x.new_empty((2,) + x.shape[:-1], dtype=env.f32).unbind(0)
    _check(env.lib.gemm_relu_layer_norm(
        x.data_ptr(), ld, weight.data_ptr(), None if bias is None else bias.data_ptr(), y.data_ptr(),
        mean.data_ptr() if stats else None, rstd.data_ptr() if stats else None, rows, cols,
        codes[dt], codes[wdt], eps, env.raw_stream(index)))
    return (y, mean, rstd) if stats else y


def layer_norm_backward(dy, x, weight, mean, rstd, stream=None):
    """Gradients (dx, dweight, dbias) of layer_norm, given dy and the statistics
    of the forward call.  dx has x's type, dweight and dbias weight's."""
    env = _get_env()
    codes, dt, f32 = env.codes, x.dtype, env.f32
    if dt not in codes:
        raise TypeError("x must be float16, bfloat16 or float32, not %s" % dt)
    if dy.dtype != dt:
        raise TypeError("dy must have x's type")
    if dy.shape != x.shape:
        raise ValueError("dy and x must have the same shape")
    rows, cols, ld = _rows(x, "x")
    dy_ld = _rows(dy, "dy")[2]
    _vector(weight, "weight", cols, (dt, f32))
    _vector(mean, "mean", rows, (f32,))
    _vector(rstd, "rstd", rows, (f32,))
    inputs = (x, dy, weight, mean, rstd)
    index = _one_gpu(*inputs)
    if stream is not None or env.current_device() != index:
        return _elsewhere(index, stream, inputs, layer_norm_backward, dy, x, weight, mean, rstd)
    lib = env.lib
    dx = env.empty_like(x) if ld == cols else x.new_empty(x.shape)
    dw, db = weight.new_empty((2,) + weight.shape).unbind(0)
    nbytes = lib.gemm_relu_layer_norm_backward_workspace(rows, cols)
    ws = x.new_empty(nbytes, dtype=env.u8)
    _check(lib.gemm_relu_layer_norm_backward(
        dy.data_ptr(), dy_ld, x.data_ptr(), ld, weight.data_ptr(), mean.data_ptr(), rstd.data_ptr(),
        dx.data_ptr(), dw.data_ptr(), db.data_ptr(), rows, cols, codes[dt], codes[weight.dtype],
        ws.data_ptr(), nbytes, env.raw_stream(index)))
    return dx, dw, db


def _gated_args(env, x, weight, act):
    code = ACTIVATIONS.get(act)
    if code is None:
        raise ValueError("act must be one of %s" % ", ".join(sorted(ACTIVATIONS)))
    dt = x.dtype
    if dt == env.f32 or dt not in env.codes or weight.dtype != dt:
        raise TypeError("x and weight must share dtype float16 or bfloat16")
    rows, cols, ld = _rows(x, "x")
    wrows, wcols, wld = _weight(weight, "weight")
    if wcols != cols or wrows % 2:
        raise ValueError("weight must be (2 * hidden, %d), gate rows first" % cols)
    return rows, cols, ld, wrows // 2, wld, code


def matmul_gated(x, weight, act="silu", save=False, stream=None):
    """Gated projections h = act(x Wg^T) * (x Wu^T).

    x: (..., cols) float16 or bfloat16; weight: (2 * hidden, cols), the gate's
    rows Wg first, then Wu.  act: "silu", "gelu", "gelu_tanh" or "relu".  Returns
    h (..., hidden), or with ``save`` (h, gu): gu (..., 2 * hidden) holds the
    fp32 sums x Wg^T and x Wu^T for matmul_gated_backward (in 16 bits their
    rounding would be as large as that of the gradients themselves).
    """
    env = _get_env()
    rows, cols, ld, hidden, wld, code = _gated_args(env, x, weight, act)
    index = _one_gpu(x, weight)
    if stream is not None or env.current_device() != index:
        return _elsewhere(index, stream, (x, weight), matmul_gated, x, weight, act, save)
    lead = x.shape[:-1]
    h = x.new_empty(lead + (hidden,))
    gu = x.new_empty(lead + (2 * hidden,), dtype=env.f32) if save else None
    _check(env.lib.gemm_relu_gated(x.data_ptr(), ld, weight.data_ptr(), wld, h.data_ptr(),
                                   gu.data_ptr() if save else None, rows, hidden, cols, env.codes[x.dtype],
                                   code, env.raw_stream(index)))
    return (h, gu) if save else h


def matmul_gated_backward(dh, gu, x, weight, act="silu", stream=None):
    """Gradients (dx, dweight) of matmul_gated, given dh and the forward call's
    gu.  Both have x's type."""
    env = _get_env()
    rows, cols, ld, hidden, wld, code = _gated_args(env, x, weight, act)
    if dh.dtype != x.dtype:
        raise TypeError("dh must have x's type")
    if dh.shape != x.shape[:-1] + (hidden,):
        raise ValueError("dh must have matmul_gated's shape %s" % (tuple(x.shape[:-1]) + (hidden,),))
    dh_ld = _rows(dh, "dh")[2]
    _vector(gu, "gu", rows * 2 * hidden, (env.f32,))
    inputs = (x, weight, dh, gu)
    index = _one_gpu(*inputs)
    if stream is not None or env.current_device() != index:
        return _elsewhere(index, stream, inputs, matmul_gated_backward, dh, gu, x, weight, act)
    lib = env.lib
    dx = env.empty_like(x) if ld == cols else x.new_empty(x.shape)
    dw = env.empty_like(weight) if wld == cols else weight.new_empty(weight.shape)
    nbytes = lib.gemm_relu_gated_backward_workspace(rows, hidden, cols)
    ws = x.new_empty(nbytes, dtype=env.u8)
    _check(lib.gemm_relu_gated_backward(
        dh.data_ptr(), dh_ld, gu.data_ptr(), x.data_ptr(), ld, weight.data_ptr(), wld, dx.data_ptr(),
        dw.data_ptr(), rows, hidden, cols, env.codes[x.dtype], code, ws.data_ptr(), nbytes,
        env.raw_stream(index)))
    return dx, dw


def quantize_rows(x, stream=None):
    """Each row (last dimension) of x in 8 bits: returns (q, scale), int8 q of x's
    shape and fp32 scale = max|row| / 127, with row ~ q * scale.  A row that holds
    an infinity or NaN has scale NaN."""
    env = _get_env()
    code = env.codes.get(x.dtype)
    if code is None:
        raise TypeError("x must be float16, bfloat16 or float32, not %s" % x.dtype)
    rows, cols, ld = _rows(x, "x")
    index = _one_gpu(x)
    if stream is not None or env.current_device() != index:
        return _elsewhere(index, stream, (x,), quantize_rows, x)
    q = x.new_empty(x.shape, dtype=env.i8)
    scale = x.new_empty(x.shape[:-1], dtype=env.f32)
    _check(env.lib.gemm_relu_quantize_rows(x.data_ptr(), ld, q.data_ptr(), scale.data_ptr(), rows, cols, code,
                                           env.raw_stream(index)))
    return q, scale


def matmul_i8(x, x_scale, weight, weight_scale, out_dtype=None, stream=None):
    """8-bit integer product y = (x weight^T) * x_scale[..., None] * weight_scale.

    x: (..., k) int8 with one fp32 scale per row; weight: (n, k) int8 with one
    fp32 scale per row (output channel).  Sums are exact (k <= 131071).  Returns
    y (..., n) of out_dtype (float16, bfloat16 or float32; default bfloat16).
    """
    env = _get_env()
    out_dtype = env.torch.bfloat16 if out_dtype is None else out_dtype
    if x.dtype != env.i8 or weight.dtype != env.i8:
        raise TypeError("x and weight must be int8")
    code = env.codes.get(out_dtype)
    if code is None:
        raise TypeError("out_dtype must be float16, bfloat16 or float32, not %s" % out_dtype)
    rows, k, ld = _rows(x, "x")
    n, wk, wld = _weight(weight, "weight")
    if wk != k:
        raise ValueError("inner dimensions differ: %d vs %d" % (k, wk))
    _vector(x_scale, "x_scale", rows, (env.f32,))
    _vector(weight_scale, "weight_scale", n, (env.f32,))
    inputs = (x, x_scale, weight, weight_scale)
    index = _one_gpu(*inputs)
    if stream is not None or env.current_device() != index:
        return _elsewhere(index, stream, inputs, matmul_i8, x, x_scale, weight, weight_scale, out_dtype)
    y = x.new_empty(x.shape[:-1] + (n,), dtype=out_dtype)
    _check(env.lib.gemm_relu_i8(x.data_ptr(), ld, x_scale.data_ptr(), weight.data_ptr(), wld,
                                weight_scale.data_ptr(), y.data_ptr(), rows, n, k, code, env.raw_stream(index)))
    return y
