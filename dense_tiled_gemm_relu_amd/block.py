"""Operators around a transformer's feed-forward half layer, on torch tensors.

The product with bias, activation and residual in its epilogue and the step from one
block to the next (residual sum and norms), both with their backward passes, and the
orthogonalisation of a weight's update.  The work is done by the kernels behind include/gemm_relu_block.h, called
through a small C++ module (csrc/block_torch.cpp); there is no CPU or PyTorch
fallback.  Rows, strides, streams, results without autograd graphs: as in ffn.py.
"""
import ctypes
import numbers
import os

from . import ffn

ACTIVATIONS = {"none": 4, **ffn.ACTIVATIONS}
NORMS = {"rms": 0, "layer": 1}

_vp, _i64, _int, _u64 = ctypes.c_void_p, ctypes.c_int64, ctypes.c_int, ctypes.c_uint64
_SIGNATURES = {
    "gemm_relu_act": ([_vp, _i64, _vp, _i64, _vp, _vp, _i64, _vp, _vp, _i64, _i64, _i64, _int, _int, _int, _vp], _int),
    "gemm_relu_act_plan": ([_i64, _i64, _i64, _int], ctypes.c_char_p),
    "gemm_relu_act_backward_workspace": ([_i64, _i64, _i64], _i64),
    "gemm_relu_act_backward": ([_vp, _i64, _vp, _vp, _i64, _vp, _i64, _vp, _vp, _vp, _i64, _i64, _i64, _int, _int,
                                _int, _vp, _u64, _vp], _int),
    "gemm_relu_act_backward_plan": ([_i64, _i64, _i64, _int], ctypes.c_char_p),
    "gemm_relu_add_norm": ([_vp, _i64, _vp, _i64, _vp, _i64] + [_vp] * 6 + [_i64, _i64, _int, _int, _int, ctypes.c_float,
                           ctypes.c_float, _vp], _int),
    "gemm_relu_add_norm_backward_workspace": ([_i64, _i64], _i64),
    "gemm_relu_orthogonalize_workspace": ([_i64, _i64, _i64], _i64),
    "gemm_relu_orthogonalize_plan": ([_i64, _i64, _i64], ctypes.c_char_p),
    "gemm_relu_orthogonalize": ([_vp, _i64, _i64, _vp, _i64, _i64, _i64, _int, _vp, _int, ctypes.c_float, _vp, _u64, _vp], _int),
    "gemm_relu_add_norm_backward": ([_vp, _i64] * 5 + [_vp] * 9 + [_i64, _i64, _int, _int, _int, ctypes.c_float, _vp, _u64,
                                    _vp], _int),
}


def declare(lib):
    """Argument and result types of the functions of include/gemm_relu_block.h."""
    for name, (args, res) in _SIGNATURES.items():
        fn = getattr(lib, name)
        fn.argtypes, fn.restype = args, res


MODULE_PATH = os.path.join(os.path.dirname(os.path.abspath(__file__)), "_block.so")
# the C functions the front end calls, in the order it takes them
_BOUND = ("gemm_relu_act", "gemm_relu_act_backward_workspace", "gemm_relu_act_backward", "gemm_relu_add_norm",
          "gemm_relu_add_norm_backward_workspace", "gemm_relu_add_norm_backward", "gemm_relu_orthogonalize_workspace",
          "gemm_relu_orthogonalize")

_ops = _current_device = _raw_stream = _tensor = None


def _load():
    """The front end module, bound to the loaded library; raises if either has
    not been built."""
    global _ops, _current_device, _raw_stream, _tensor
    import torch
    ops = ffn.load_module("_block", MODULE_PATH, _BOUND)
    _current_device, _raw_stream = torch._C._cuda_getDevice, torch._C._cuda_getCurrentRawStream
    _tensor = torch.Tensor
    _ops = ops
    return ops


def _call(name, stream, *args):
    return ffn.call_on(_ops or _load(), name, stream, args)


def _activation(act):
    code = ACTIVATIONS.get(act)
    if code is None:
        raise ValueError("act must be one of %s" % ", ".join(sorted(ACTIVATIONS)))
    return code


def matmul_act(x, weight, bias=None, act="none", residual=None, save=False, stream=None):
    """Product with bias, activation and residual: y = act(x weight^T + bias) + residual.

    x: (..., k) float16 or bfloat16; weight: (n, k); bias (n) of x's type or float32;
    residual: (..., n), of x's type.  act: "none", "silu", "gelu", "gelu_tanh" or
    "relu".  Returns y (..., n), or with ``save`` (y, z): z (..., n) holds the fp32
    sums x weight^T + bias for matmul_act_backward (None without an activation, whose
    gradient takes none).
    """
    code = _activation(act)
    if stream is None and _ops is not None and isinstance(x, _tensor):
        index = x.get_device()
        if index >= 0 and _current_device() == index:
            return _ops.matmul_act(x, weight, bias, code, residual, save, _raw_stream(index))
    return _call("matmul_act", stream, x, weight, bias, code, residual, save)


def matmul_act_backward(dy, z, x, weight, act="none", bias=None, stream=None):
    """Gradients (dx, dweight, dbias) of matmul_act, given dy and the forward call's z
    (None without an activation).  dx and dweight have x's type; dbias has the bias's,
    and is None without one.  The residual's gradient is dy."""
    code = _activation(act)
    if stream is None and _ops is not None and isinstance(x, _tensor):
        index = x.get_device()
        if index >= 0 and _current_device() == index:
            return _ops.matmul_act_backward(dy, z, x, weight, code, bias, _raw_stream(index))
    return _call("matmul_act_backward", stream, dy, z, x, weight, code, bias)


def _norm(norm):
    code = NORMS.get(norm)
    if code is None:
        raise ValueError("norm must be one of %s" % ", ".join(sorted(NORMS)))
    return code


def add_norm(x, residual, weight=None, bias=None, gate=None, scale=1.0, post_weight=None, norm="rms", eps=1e-5, stats=False,
             stream=None):
    """From one block to the next: the residual sum s = residual + scale * gate * t, where
    t is x, the block's output, or with ``post_weight`` norm(x) * post_weight; and the
    next block's input y = norm(s) * weight + bias (y is None without a weight).

    norm: "rms", v / sqrt(mean v^2 + eps), or "layer", which also takes the mean out.
    x, residual and a gate of x's shape: float16, bfloat16 or float32, one type; weight,
    bias, post_weight and a gate of one row (1-D, the same for all rows): x's type or
    float32, one type.  Returns (s, y), or with ``stats`` (s, y, stats), the fp32
    statistics (..., 4) of each row that the backward pass takes.
    """
    code = _norm(norm)
    if stream is None and _ops is not None and isinstance(x, _tensor):
        index = x.get_device()
        if index >= 0 and _current_device() == index:
            return _ops.add_norm(x, residual, weight, bias, gate, scale, post_weight, code, eps, stats, _raw_stream(index))
    return _call("add_norm", stream, x, residual, weight, bias, gate, scale, post_weight, code, eps, stats)


def add_norm_backward(dy, ds, x, residual, stats, weight=None, bias=None, gate=None, scale=1.0, post_weight=None, norm="rms",
                      stream=None):
    """Gradients (dx, dresidual, dweight, dbias, dgate, dpost_weight) of add_norm; those of
    what was not given are None.  dy is the gradient of y (None without a weight), ds the
    one that reaches s from elsewhere (or None).  Without gate and post_weight and with
    scale 1, dx and dresidual are one tensor; without a weight dresidual is ds."""
    code = _norm(norm)
    if stream is None and _ops is not None and isinstance(x, _tensor):
        index = x.get_device()
        if index >= 0 and _current_device() == index:
            return _ops.add_norm_backward(dy, ds, x, residual, stats, weight, bias, gate, scale, post_weight, code,
                                          _raw_stream(index))
    return _call("add_norm_backward", stream, dy, ds, x, residual, stats, weight, bias, gate, scale, post_weight, code)


# of a step whose slope at 0 is large: five of them bring singular values from 1e-3 of the
# matrix's norm into 0.7 .. 1.2
NEWTON_SCHULZ = (3.4445, -4.7750, 2.0315)


def _coefficients(steps, coefficients):
    c = tuple(coefficients)
    if len(c) == 3 and all(isinstance(v, numbers.Real) for v in c):
        return c * steps
    if len(c) != steps or any(not hasattr(v, "__len__") or len(v) != 3 for v in c):
        raise ValueError("coefficients must be (a, b, c), or one such triple for each of the %d steps" % steps)
    return tuple(v for triple in c for v in triple)


def orthogonalize(g, steps=5, coefficients=NEWTON_SCHULZ, eps=1e-7, stream=None):
    """A matrix's update orthogonalised by Newton-Schulz steps: X = g / (|g| + eps), then
    ``steps`` times X <- a X + (b A + c A^2) X with A = X X^T.  g's singular vectors stay,
    its singular values tend to 1 (as far as the coefficients take them).

    g: (m, n), or a batch (b, m, n) of matrices each on its own; float16, bfloat16 or
    float32, with contiguous rows.  coefficients: (a, b, c), or a triple for each step.
    Returns bfloat16 of g's shape.  Before that rounding it is within 3e-3 of its norm for up
    to 6 steps of the default coefficients where the shorter side is at least 16 (1e-2 for
    up to 5 below that), whatever g's singular values; include/gemm_relu_block.h says more.
    """
    steps = int(steps)
    if not 0 <= steps <= 64:
        raise ValueError("steps must be from 0 to 64")
    c = _coefficients(steps, coefficients)
    if stream is None and _ops is not None and isinstance(g, _tensor):
        index = g.get_device()
        if index >= 0 and _current_device() == index:
            return _ops.orthogonalize(g, c, eps, _raw_stream(index))
    return _call("orthogonalize", stream, g, c, eps)
