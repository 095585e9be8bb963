"""The feed-forward operators on the host: what they refuse, before any GPU call."""
import pytest
import torch

import dense_tiled_gemm_relu_amd as gr

# fake, well-aligned and disjoint addresses: validation inspects, never dereferences
P = [i << 40 for i in range(1, 12)]
X, W, B, Y, S0, S1, DY, DX, DW, DB, WS = P
F16, BF16, F32 = gr.F16, gr.BF16, gr.F32
BIG = 2 ** 31


def call(name, args, **over):
    """The C function's status for `args` (a dict in argument order) with some replaced."""
    assert set(over) <= set(args)
    return getattr(gr.library(), name)(*{**args, **over}.values(), 0)


NORM = dict(x=X, x_stride=8, w=W, b=B, y=Y, mean=S0, rstd=S1, rows=4, cols=8, dtype=F16, wdtype=F16, eps=1e-5)
NORM_BWD = dict(dy=DY, dy_stride=8, x=X, x_stride=8, w=W, mean=S0, rstd=S1, dx=DX, dw=DW, db=DB, rows=4, cols=8,
                dtype=BF16, wdtype=F32, ws=WS, ws_bytes=1 << 20)
GATED = dict(x=X, x_stride=8, w=W, w_stride=8, h=Y, gu=S0, rows=4, hidden=6, cols=8, dtype=F16, act=0)
GATED_BWD = dict(dh=DY, dh_stride=6, gu=S0, x=X, x_stride=8, w=W, w_stride=8, dx=DX, dw=DW, rows=4, hidden=6, cols=8,
                 dtype=F16, act=0, ws=WS, ws_bytes=1 << 20)
QUANT = dict(x=X, x_stride=8, q=Y, scale=S0, rows=4, cols=8, dtype=F16)
I8 = dict(x=X, x_stride=8, xs=S0, w=W, w_stride=8, ws=S1, y=Y, rows=4, n=6, k=8, out=F16)

CASES = [("gemm_relu_layer_norm", NORM, o) for o in (
    dict(rows=-1), dict(cols=-1), dict(cols=0), dict(rows=BIG), dict(dtype=3), dict(dtype=F32), dict(wdtype=BF16),
    dict(x_stride=7), dict(x_stride=BIG), dict(x=0), dict(w=0), dict(y=0), dict(x=X + 1), dict(w=W + 1), dict(y=Y + 1),
    dict(mean=S0 + 2), dict(rstd=S0), dict(y=X), dict(y=X + 62), dict(mean=W), dict(eps=-1.0), dict(eps=float("nan")))]
CASES += [("gemm_relu_layer_norm_backward", NORM_BWD, o) for o in (
    dict(rows=-1), dict(cols=0), dict(dtype=8), dict(wdtype=F16), dict(dy_stride=4), dict(dy=0), dict(mean=0),
    dict(rstd=0), dict(dw=0), dict(dx=X), dict(dx=DY), dict(dw=W), dict(db=DW), dict(ws=0), dict(ws=WS + 128),
    dict(ws_bytes=8), dict(ws=X), dict(dw=DW + 2))]
CASES += [("gemm_relu_gated", GATED, o) for o in (
    dict(rows=-1), dict(hidden=-1), dict(cols=-1), dict(hidden=2 ** 30), dict(dtype=F32), dict(dtype=3), dict(act=-1),
    dict(act=4), dict(x_stride=7), dict(w_stride=7), dict(x=0), dict(w=0), dict(h=0), dict(x=X + 1), dict(h=Y + 1),
    dict(gu=S0 + 2), dict(h=X), dict(h=W + 100), dict(gu=W), dict(gu=Y))]
CASES += [("gemm_relu_gated_backward", GATED_BWD, o) for o in (
    dict(rows=-1), dict(hidden=BIG), dict(dtype=F32), dict(act=9), dict(dh_stride=5), dict(x_stride=1), dict(dh=0),
    dict(gu=0), dict(x=0), dict(w=0), dict(dx=0), dict(dw=0), dict(dx=X), dict(dw=W), dict(dx=DW), dict(dx=DY),
    dict(ws=0), dict(ws=WS + 64), dict(ws_bytes=100), dict(ws=W))]
CASES += [("gemm_relu_quantize_rows", QUANT, o) for o in (
    dict(rows=-1), dict(cols=BIG), dict(dtype=3), dict(x_stride=7), dict(x=0), dict(q=0), dict(scale=0), dict(x=X + 1),
    dict(scale=S0 + 2), dict(q=X + 8), dict(scale=Y))]
CASES += [("gemm_relu_i8", I8, o) for o in (
    dict(rows=-1), dict(n=-1), dict(k=-1), dict(out=3), dict(x_stride=7), dict(w_stride=7), dict(x=0), dict(w=0),
    dict(xs=0), dict(ws=0), dict(y=0), dict(y=Y + 1), dict(xs=S0 + 1), dict(y=X), dict(y=W), dict(y=S0))]


@pytest.mark.parametrize("name,args,over", CASES)
def test_invalid_arguments_fail_before_the_device(name, args, over):
    assert call(name, args, **over) == gr.EINVAL


def test_sums_that_could_overflow_are_refused():
    assert call("gemm_relu_i8", I8, k=131072, x_stride=131072, w_stride=131072) == gr.EUNSUPPORTED


@pytest.mark.parametrize("name,args,over", [
    ("gemm_relu_layer_norm", NORM, dict(rows=0, x=0, y=0, mean=0, rstd=0)),
    ("gemm_relu_layer_norm_backward", NORM_BWD, dict(rows=0, cols=0)),
    ("gemm_relu_gated", GATED, dict(rows=0, x=0, h=0, gu=0)), ("gemm_relu_gated", GATED, dict(hidden=0)),
    ("gemm_relu_gated_backward", GATED_BWD, dict(cols=0, x_stride=0, w_stride=0)),
    ("gemm_relu_gated_backward", GATED_BWD, dict(rows=0, hidden=0)),
    ("gemm_relu_quantize_rows", QUANT, dict(rows=0)),
    ("gemm_relu_i8", I8, dict(rows=0)), ("gemm_relu_i8", I8, dict(n=0)),
])
def test_calls_without_outputs_are_a_no_op(name, args, over):
    assert call(name, args, **over) == gr.OK


def test_workspace_sizes():
    lib = gr.library()
    assert lib.gemm_relu_layer_norm_backward_workspace(0, 100) == 0
    assert lib.gemm_relu_layer_norm_backward_workspace(1, 100) >= 2 * 100 * 4
    assert lib.gemm_relu_layer_norm_backward_workspace(-1, 100) == gr.EINVAL
    # both layouts of dg and du
    assert lib.gemm_relu_gated_backward_workspace(10, 20, 30) >= 2 * 2 * 10 * 40
    assert lib.gemm_relu_gated_backward_workspace(10, -20, 30) == gr.EINVAL
    # grows without wrapping
    assert lib.gemm_relu_gated_backward_workspace(2 ** 20, 2 ** 20, 8) >= 2 ** 43


def test_plans():
    lib = gr.library()
    assert lib.gemm_relu_gated_plan(4, 6, 8, F32) is None
    assert lib.gemm_relu_gated_plan(0, 6, 8, F16) == b"none"
    assert lib.gemm_relu_gated_plan(4, 6, 8, F16)
    assert lib.gemm_relu_gated_backward_plan(4, 6, 8, F32) is None
    assert lib.gemm_relu_gated_backward_plan(4, 6, 0, F16) == b"none"
    assert lib.gemm_relu_gated_backward_plan(4, 6, 8, F16).count(b",") == 1
    assert lib.gemm_relu_i8_plan(4, 6, 8, 3) is None
    assert lib.gemm_relu_i8_plan(4, 0, 8, F16) == b"none"
    assert lib.gemm_relu_i8_plan(4, 6, 131072, F16) == b"unsupported"
    assert lib.gemm_relu_i8_plan(4, 6, 8, F16)


# ---- the tensor front ends (CPU tensors: every refusal comes before the device is looked at, the last one is it)
def t(*shape, dtype=torch.float16):
    return torch.zeros(shape, dtype=dtype)


F = torch.float32
H = torch.bfloat16


@pytest.mark.parametrize("error,fn", [
    (ValueError, lambda: gr.layer_norm(t(4, 8), t(8), t(8))),                          # not on a GPU
    (TypeError, lambda: gr.layer_norm(t(4, 8, dtype=torch.int8), t(8))),
    (TypeError, lambda: gr.layer_norm(t(4, 8), t(8, dtype=H))),
    (TypeError, lambda: gr.layer_norm(t(4, 8), t(8), t(8, dtype=F))),
    (ValueError, lambda: gr.layer_norm(t(4, 8), t(7))),
    (ValueError, lambda: gr.layer_norm(t(8, 4).t(), t(8))),                            # rows not contiguous
    (ValueError, lambda: gr.layer_norm(t(1, 8).expand(4, 8), t(8))),                   # rows overlap
    (ValueError, lambda: gr.layer_norm(t(3, 4, 8)[:, ::2], t(8))),
    (ValueError, lambda: gr.layer_norm(t(), t(8))),
    (TypeError, lambda: gr.layer_norm_backward(t(4, 8, dtype=F), t(4, 8), t(8), t(4, dtype=F), t(4, dtype=F))),
    (ValueError, lambda: gr.layer_norm_backward(t(4, 7), t(4, 8), t(8), t(4, dtype=F), t(4, dtype=F))),
    (TypeError, lambda: gr.layer_norm_backward(t(4, 8), t(4, 8), t(8), t(4), t(4, dtype=F))),
    (ValueError, lambda: gr.layer_norm_backward(t(4, 8), t(4, 8), t(8), t(4, dtype=F), t(5, dtype=F))),
    (ValueError, lambda: gr.layer_norm_backward(t(4, 8), t(4, 8), t(8), t(4, dtype=F), t(4, dtype=F))),
    (ValueError, lambda: gr.matmul_gated(t(4, 8), t(6, 8), "swish")),
    (TypeError, lambda: gr.matmul_gated(t(4, 8, dtype=F), t(6, 8, dtype=F))),
    (TypeError, lambda: gr.matmul_gated(t(4, 8), t(6, 8, dtype=H))),
    (ValueError, lambda: gr.matmul_gated(t(4, 8), t(7, 8))),                           # an odd number of rows
    (ValueError, lambda: gr.matmul_gated(t(4, 8), t(6, 9))),
    (ValueError, lambda: gr.matmul_gated(t(4, 8), t(8, 6).t())),
    (ValueError, lambda: gr.matmul_gated(t(4, 8), t(2, 3, 8))),
    (ValueError, lambda: gr.matmul_gated(t(4, 8), t(6, 8))),
    (TypeError, lambda: gr.matmul_gated_backward(t(4, 3, dtype=H), t(4, 6, dtype=F), t(4, 8), t(6, 8))),
    (ValueError, lambda: gr.matmul_gated_backward(t(4, 6), t(4, 6, dtype=F), t(4, 8), t(6, 8))),
    (TypeError, lambda: gr.matmul_gated_backward(t(4, 3), t(4, 6), t(4, 8), t(6, 8))),
    (ValueError, lambda: gr.matmul_gated_backward(t(4, 3), t(4, 5, dtype=F), t(4, 8), t(6, 8))),
    (ValueError, lambda: gr.matmul_gated_backward(t(4, 3), t(4, 6, dtype=F), t(4, 8), t(6, 8))),
    (TypeError, lambda: gr.quantize_rows(t(4, 8, dtype=torch.int8))),
    (ValueError, lambda: gr.quantize_rows(t(8, 4).t())),
    (ValueError, lambda: gr.quantize_rows(t(4, 8))),
    (TypeError, lambda: gr.matmul_i8(t(4, 8), t(4, dtype=F), t(6, 8), t(6, dtype=F))),
    (TypeError, lambda: gr.matmul_i8(t(4, 8, dtype=torch.int8), t(4), t(6, 8, dtype=torch.int8), t(6, dtype=F))),
    (ValueError, lambda: gr.matmul_i8(t(4, 8, dtype=torch.int8), t(4, dtype=F), t(6, 9, dtype=torch.int8),
                                      t(6, dtype=F))),
    (ValueError, lambda: gr.matmul_i8(t(4, 8, dtype=torch.int8), t(3, dtype=F), t(6, 8, dtype=torch.int8),
                                      t(6, dtype=F))),
    (TypeError, lambda: gr.matmul_i8(t(4, 8, dtype=torch.int8), t(4, dtype=F), t(6, 8, dtype=torch.int8),
                                     t(6, dtype=F), torch.int8)),
    (ValueError, lambda: gr.matmul_i8(t(4, 8, dtype=torch.int8), t(4, dtype=F), t(6, 8, dtype=torch.int8),
                                      t(6, dtype=F))),
])
def test_front_ends_refuse(error, fn):
    with pytest.raises(error):
        fn()
