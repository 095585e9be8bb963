"""Operators of a transformer's feed-forward half layer, on torch tensors.

Layer norm, the gated projections h = act(x Wg^T) * (x Wu^T), both with their
backward passes, the quantisation of activations row by row and the 8-bit
integer product.  The work is done by the kernels behind
include/gemm_relu_ffn.h, called through a small C++ module (csrc/ffn_torch.cpp)
that checks the arguments and allocates; there is no CPU or PyTorch fallback.

Activations are matrices of rows: any shape whose last dimension is the row, if
contiguous, or 2-D with contiguous rows any distance apart.  Results are new
contiguous tensors.  The kernels run on ``stream`` (a torch.cuda.Stream, a raw
hipStream_t, or None for torch's current stream); results and workspaces are
allocated for that stream.  A tensor made on another stream has to be ready
before the call, as with any torch operation.  Results carry no autograd graph: a
backward function is a call of its own.  An input that requires a gradient, where
gradients are recorded, gives a UserWarning.
"""
import ctypes
import importlib.machinery
import importlib.util
import os

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


MODULE_PATH = os.path.join(os.path.dirname(os.path.abspath(__file__)), "_ffn.so")
# the C functions the front end calls, in the order it takes them
_BOUND = ("gemm_relu_layer_norm", "gemm_relu_layer_norm_backward_workspace", "gemm_relu_layer_norm_backward",
          "gemm_relu_gated", "gemm_relu_gated_backward_workspace", "gemm_relu_gated_backward",
          "gemm_relu_quantize_rows", "gemm_relu_i8")


def _status_error(status):
    from . import GemmReluError, gemm_relu_strerror
    return GemmReluError(status, gemm_relu_strerror(status))


_ops = _current_device = _raw_stream = _tensor = None


def load_module(name, path, bound):
    """The front end module `name`, bound to the `bound` functions of the loaded
    library; raises if either has not been built."""
    from . import library
    lib = library()
    if not os.path.exists(path):
        raise RuntimeError("front end %s is not built; run __graft_entry__.build()" % path)
    loader = importlib.machinery.ExtensionFileLoader(name, path)
    ops = importlib.util.module_from_spec(importlib.util.spec_from_loader(name, loader))
    loader.exec_module(ops)
    ops.bind(_status_error, *(ctypes.cast(getattr(lib, fn), _vp).value for fn in bound))
    return ops


def _load():
    global _ops, _current_device, _raw_stream, _tensor
    import torch
    ops = load_module("_ffn", MODULE_PATH, _BOUND)
    _current_device, _raw_stream = torch._C._cuda_getDevice, torch._C._cuda_getCurrentRawStream
    _tensor = torch.Tensor
    _ops = ops
    return ops


def _as_torch_stream(stream, index):
    """`stream` as a torch stream of GPU `index`.  0 is the handle of the default
    stream; ExternalStream would take it for "none given" and hand out a stream of
    torch's pool, which waits for nothing."""
    import torch
    if not isinstance(stream, int):
        return stream
    return torch.cuda.ExternalStream(stream, device=index) if stream else torch.cuda.default_stream(index)


def _call(name, stream, *args):
    return call_on(_ops or _load(), name, stream, args)


def call_on(ops, name, stream, args):
    """One call of the front end `ops`: on the tensors' GPU and `stream`, both made
    current for the allocations and the launches."""
    first = next((a for a in args if hasattr(a, "get_device")), None)
    index = -1 if first is None else first.get_device()
    if index < 0:                                     # refused there, with the reason
        return getattr(ops, name)(*args, 0)
    import torch
    with torch.cuda.device(index):
        if stream is None:
            return getattr(ops, name)(*args, torch._C._cuda_getCurrentRawStream(index))
        stream = _as_torch_stream(stream, index)
        with torch.cuda.stream(stream):
            out = getattr(ops, name)(*args, stream.cuda_stream)
        # the caller may drop an input while the stream still reads it
        for t in args:
            if isinstance(t, torch.Tensor):
                t.record_stream(stream)
        return out


def layer_norm(x, weight, bias=None, eps=1e-5, stats=False, stream=None):
    """Layer norm over the last dimension: (x - mean) * rstd * weight + bias.

    x: float16, bfloat16 or float32; weight and bias (or None): x's type or
    float32.  Returns y, or with ``stats`` (y, mean, rstd), the fp32 statistics
    of each row that the backward pass takes.
    """
    if stream is None and _ops is not None and isinstance(x, _tensor):
        index = x.get_device()
        if index >= 0 and _current_device() == index:
            return _ops.layer_norm(x, weight, bias, eps, stats, _raw_stream(index))
    return _call("layer_norm", stream, x, weight, bias, eps, stats)


def layer_norm_backward(dy, x, weight, mean, rstd, stream=None):
    """Gradients (dx, dweight, dbias) of layer_norm, given dy and the statistics
    of the forward call.  dx has x's type, dweight and dbias weight's."""
    if stream is None and _ops is not None and isinstance(x, _tensor):
        index = x.get_device()
        if index >= 0 and _current_device() == index:
            return _ops.layer_norm_backward(dy, x, weight, mean, rstd, _raw_stream(index))
    return _call("layer_norm_backward", stream, dy, x, weight, mean, rstd)


def _activation(act):
    code = ACTIVATIONS.get(act)
    if code is None:
        raise ValueError("act must be one of %s" % ", ".join(sorted(ACTIVATIONS)))
    return code


def matmul_gated(x, weight, act="silu", save=False, stream=None):
    """Gated projections h = act(x Wg^T) * (x Wu^T).

    x: (..., cols) float16 or bfloat16; weight: (2 * hidden, cols), the gate's
    rows Wg first, then Wu.  act: "silu", "gelu", "gelu_tanh" or "relu".  Returns
    h (..., hidden), or with ``save`` (h, gu): gu (..., 2 * hidden) holds the
    fp32 sums x Wg^T and x Wu^T for matmul_gated_backward (in 16 bits their
    rounding would be as large as that of the gradients themselves).
    """
    code = _activation(act)
    if stream is None and _ops is not None and isinstance(x, _tensor):
        index = x.get_device()
        if index >= 0 and _current_device() == index:
            return _ops.matmul_gated(x, weight, code, save, _raw_stream(index))
    return _call("matmul_gated", stream, x, weight, code, save)


def matmul_gated_backward(dh, gu, x, weight, act="silu", stream=None):
    """Gradients (dx, dweight) of matmul_gated, given dh and the forward call's
    gu.  Both have x's type."""
    code = _activation(act)
    if stream is None and _ops is not None and isinstance(x, _tensor):
        index = x.get_device()
        if index >= 0 and _current_device() == index:
            return _ops.matmul_gated_backward(dh, gu, x, weight, code, _raw_stream(index))
    return _call("matmul_gated_backward", stream, dh, gu, x, weight, code)


def quantize_rows(x, stream=None):
    """Each row (last dimension) of x in 8 bits: returns (q, scale), int8 q of x's
    shape and fp32 scale = max|row| / 127, with row ~ q * scale.  A row that holds
    an infinity or NaN has scale NaN."""
    if stream is None and _ops is not None and isinstance(x, _tensor):
        index = x.get_device()
        if index >= 0 and _current_device() == index:
            return _ops.quantize_rows(x, _raw_stream(index))
    return _call("quantize_rows", stream, x)


def matmul_i8(x, x_scale, weight, weight_scale, out_dtype=None, stream=None):
    """8-bit integer product y = (x weight^T) * x_scale[..., None] * weight_scale.

    x: (..., k) int8 with one fp32 scale per row; weight: (n, k) int8 with one
    fp32 scale per row (output channel).  Sums are exact (k <= 131071).  Returns
    y (..., n) of out_dtype (float16, bfloat16 or float32; default bfloat16).
    """
    if stream is None and _ops is not None and isinstance(x, _tensor):
        index = x.get_device()
        if index >= 0 and _current_device() == index:
            return _ops.matmul_i8(x, x_scale, weight, weight_scale, out_dtype, _raw_stream(index))
    return _call("matmul_i8", stream, x, x_scale, weight, weight_scale, out_dtype)
