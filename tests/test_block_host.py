"""The operators around the half layer on the host: what they refuse, before any GPU call."""
import ctypes

import pytest
import torch

import dense_tiled_gemm_relu_amd as gr

# fake, well-aligned and disjoint addresses: validation inspects, never dereferences
P = [i << 40 for i in range(1, 16)]
X, W, B, R, Y, Z, DY, DX, DW, DB, WS, G, PW, S, ST = P
F16, BF16, F32 = gr.F16, gr.BF16, gr.F32
BIG = 2 ** 31


def call(name, args, **over):
    """The C function's status for `args` (a dict in argument order) with some replaced."""
    assert set(over) <= set(args)
    return getattr(gr.library(), name)(*{**args, **over}.values(), 0)


ACT = dict(x=X, x_stride=8, w=W, w_stride=8, b=B, r=R, r_stride=6, y=Y, z=Z, rows=4, n=6, k=8, dtype=F16, bdtype=F32, act=0)
ACT_BWD = dict(dy=DY, dy_stride=6, z=Z, x=X, x_stride=8, w=W, w_stride=8, dx=DX, dw=DW, db=DB, rows=4, n=6, k=8, dtype=F16,
               bdtype=F16, act=0, ws=WS, ws_bytes=1 << 20)

NORM = dict(x=X, x_stride=8, r=R, r_stride=8, gate=G, g_stride=0, pw=PW, w=W, b=B, s=S, y=Y, stats=ST, rows=4, cols=8,
            dtype=BF16, wdtype=F32, norm=0, scale=1.0, eps=1e-5)
NORM_BWD = dict(dy=DY, dy_stride=8, ds=Z, ds_stride=8, x=X, x_stride=8, r=R, r_stride=8, gate=G, g_stride=8, pw=PW, w=W,
                stats=ST, dx=DX, dr=1 << 50, dgate=DB, dpw=1 << 51, dw=DW, db=1 << 52, rows=4, cols=8, dtype=F16, wdtype=F16,
                norm=1, scale=1.0, ws=WS, ws_bytes=1 << 20)

CASES = [("gemm_relu_act", ACT, o) for o in (
    dict(rows=-1), dict(n=-1), dict(k=-1), dict(rows=BIG), dict(n=BIG), dict(dtype=F32), dict(dtype=3), dict(bdtype=BF16),
    dict(act=-1), dict(act=5), dict(x_stride=7), dict(w_stride=7), dict(r_stride=5), dict(x_stride=BIG), dict(x=0), dict(w=0),
    dict(y=0), dict(x=X + 1), dict(w=W + 1), dict(y=Y + 1), dict(b=B + 2), dict(r=R + 1), dict(z=Z + 2), dict(y=X), dict(y=W + 90),
    dict(y=R), dict(z=R), dict(z=Y), dict(z=B), dict(y=B))]
CASES += [("gemm_relu_act_backward", ACT_BWD, o) for o in (
    dict(rows=-1), dict(n=BIG), dict(k=-1), dict(dtype=F32), dict(bdtype=BF16), dict(act=5), dict(dy_stride=5), dict(x_stride=1),
    dict(dy=0), dict(z=0), dict(x=0), dict(w=0), dict(dx=0), dict(dw=0), dict(dx=X), dict(dw=W), dict(db=DW), dict(dx=DY),
    dict(db=DY), dict(ws=0), dict(ws=WS + 64), dict(ws_bytes=100), dict(ws=W), dict(db=DB + 1))]

NAN, INF = float("nan"), float("inf")
CASES += [("gemm_relu_add_norm", NORM, o) for o in (
    dict(rows=-1), dict(cols=-1), dict(cols=0), dict(rows=BIG), dict(dtype=3), dict(wdtype=F16), dict(norm=2), dict(norm=-1),
    dict(x_stride=7), dict(r_stride=7), dict(g_stride=7), dict(g_stride=-8), dict(g_stride=BIG), dict(x=0), dict(r=0), dict(s=0),
    dict(y=0), dict(w=0), dict(x=X + 1), dict(r=R + 1), dict(gate=G + 2), dict(stats=ST + 2), dict(s=X), dict(s=R + 8),
    dict(y=S), dict(y=W), dict(stats=PW), dict(s=G), dict(eps=-1.0), dict(eps=NAN), dict(scale=NAN), dict(scale=INF))]
CASES += [("gemm_relu_add_norm_backward", NORM_BWD, o) for o in (
    dict(rows=-1), dict(cols=0), dict(dtype=8), dict(wdtype=BF16), dict(norm=2), dict(scale=-INF), dict(dy=0), dict(x=0),
    dict(r=0), dict(stats=0), dict(w=0), dict(gate=0), dict(pw=0), dict(dy_stride=7), dict(ds_stride=7), dict(g_stride=4),
    dict(dx=DY), dict(dr=Z), dict(dx=X), dict(dr=R), dict(dgate=G), dict(dpw=PW), dict(dw=W), dict(db=DW), dict(dr=DX),
    dict(ws=0), dict(ws=WS + 128), dict(ws_bytes=8), dict(ws=X), dict(dw=DW + 1))]


@pytest.mark.parametrize("name,args,over", CASES)
def test_invalid_arguments_fail_before_the_device(name, args, over):
    assert call(name, args, **over) == gr.EINVAL


@pytest.mark.parametrize("name,args,over", [
    ("gemm_relu_act", ACT, dict(rows=0, x=0, y=0, r=0, z=0)), ("gemm_relu_act", ACT, dict(n=0, r_stride=0)),
    ("gemm_relu_act_backward", ACT_BWD, dict(rows=0, n=0)), ("gemm_relu_act_backward", ACT_BWD, dict(n=0, k=0)),
    ("gemm_relu_act_backward", ACT_BWD, dict(k=0, db=0)),
    ("gemm_relu_add_norm", NORM, dict(rows=0, x=0, r=0, s=0, y=0, stats=0)), ("gemm_relu_add_norm", NORM, dict(rows=0, cols=0)),
    ("gemm_relu_add_norm_backward", NORM_BWD, dict(rows=0, cols=0)),
])
def test_calls_without_outputs_are_a_no_op(name, args, over):
    assert call(name, args, **over) == gr.OK


@pytest.mark.parametrize("name,args,over", [
    ("gemm_relu_act", ACT, dict(k=BIG - 1, x_stride=BIG - 1, w_stride=BIG - 1)),
    ("gemm_relu_act", ACT, dict(rows=BIG - 1, x=1 << 40, w=1 << 50, y=1 << 62, z=0, b=0, r=0, n=BIG - 1)),
    ("gemm_relu_act_backward", ACT_BWD, dict(rows=2 ** 30 + 1)), ("gemm_relu_act_backward", ACT_BWD, dict(n=2 ** 30 + 1)),
])
def test_sizes_past_the_limits_are_refused(name, args, over):
    assert call(name, args, **over) == gr.EUNSUPPORTED


def test_workspaces_and_plans():
    lib = gr.library()
    # dz in both layouts and the sums of its 64-row tiles
    assert lib.gemm_relu_act_backward_workspace(100, 20, 30) >= 2 * 2 * 100 * 20 + 2 * 20 * 4
    assert lib.gemm_relu_act_backward_workspace(10, -20, 30) == gr.EINVAL
    assert lib.gemm_relu_act_backward_workspace(2 ** 30 + 1, 1, 1) == gr.EUNSUPPORTED
    assert lib.gemm_relu_act_backward_workspace(2 ** 20, 2 ** 20, 8) >= 2 ** 42          # grows without wrapping
    assert lib.gemm_relu_act_plan(4, 6, 8, F32) is None
    assert lib.gemm_relu_act_plan(0, 6, 8, F16) == b"none"
    assert lib.gemm_relu_act_plan(4, 6, BIG - 1, F16) == b"unsupported"
    assert lib.gemm_relu_act_plan(4, 6, 8, F16)
    assert lib.gemm_relu_act_backward_plan(4, 6, 8, F32) is None
    assert lib.gemm_relu_act_backward_plan(4, 6, 0, F16) == b"none"
    assert lib.gemm_relu_act_backward_plan(2 ** 30 + 1, 6, 8, F16) == b"unsupported"
    assert lib.gemm_relu_act_backward_plan(4, 6, 8, F16).count(b",") == 1
    assert lib.gemm_relu_add_norm_backward_workspace(0, 100) == 0
    assert lib.gemm_relu_add_norm_backward_workspace(1, 100) >= 3 * 100 * 4
    assert lib.gemm_relu_add_norm_backward_workspace(-1, 100) == gr.EINVAL
    assert lib.gemm_relu_add_norm_backward_workspace(BIG - 1, BIG - 1) >= 256 * 3 * 4 * (BIG - 1)
    assert lib.gemm_relu_orthogonalize_workspace(0, 5, 5) == 0
    assert lib.gemm_relu_orthogonalize_workspace(1, 64, 64) == 0                      # one launch, all in LDS
    assert lib.gemm_relu_orthogonalize_workspace(1, 256, 256) >= 256 * 256 * 10
    assert lib.gemm_relu_orthogonalize_workspace(1, -1, 64) == gr.EINVAL
    assert lib.gemm_relu_orthogonalize_workspace(65535, 2 ** 14, 2 ** 20) >= 65535 * 2 ** 36            # grows without wrapping
    for sizes in ((1, 2 ** 16 + 1, 2 ** 17), (1, 4, 2 ** 22 + 1), (1, 2 ** 15, 2 ** 20), (65536, 4, 4)):
        assert lib.gemm_relu_orthogonalize_workspace(*sizes) == gr.EUNSUPPORTED


def test_orthogonalize_plans():
    plan = gr.library().gemm_relu_orthogonalize_plan
    assert plan(1, -1, 4) is None and plan(0, 4, 4) == b"none" and plan(1, 2 ** 16 + 1, 2 ** 17) == b"unsupported"
    assert plan(1, 128, 256) == plan(1, 512, 64) == b"small"
    names = {plan(b, m, n): None for b in (1, 4, 8) for m in range(200, 9000, 200) for n in (m, m + 1000)}
    assert all(len(name.split(b",")) == 3 for name in names) and any(b"/" in name for name in names)


class Coefficients(ctypes.Array):
    _type_, _length_ = ctypes.c_float, 3


STEP, BAD = Coefficients(3.0, -4.0, 2.0), Coefficients(3.0, float("inf"), 2.0)
ORTHO = dict(g=X, stride=200, batch_stride=40000, out=Y, batch=2, rows=200, cols=200, dtype=BF16, c=ctypes.addressof(STEP), steps=1,
             eps=1e-7, ws=WS, ws_bytes=1 << 24)


@pytest.mark.parametrize("over", [
    dict(batch=-1), dict(rows=-1), dict(cols=BIG), dict(dtype=3), dict(stride=199), dict(stride=BIG), dict(batch_stride=-64), dict(batch_stride=2 ** 40 + 1),
    dict(g=0), dict(g=X + 1), dict(out=0), dict(out=Y + 1), dict(out=X), dict(out=X + 159998), dict(out=WS + 256), dict(c=0),
    dict(c=ctypes.addressof(BAD)), dict(steps=-1), dict(steps=65), dict(eps=-1.0), dict(eps=NAN), dict(ws=0), dict(ws=WS + 8),
    dict(ws_bytes=1000), dict(ws=X)])
def test_orthogonalize_refuses(over):
    assert call("gemm_relu_orthogonalize", ORTHO, **over) == gr.EINVAL


@pytest.mark.parametrize("over", [dict(batch=0), dict(rows=0, g=0), dict(cols=0, g=0, out=0)])
def test_orthogonalize_of_nothing(over):
    assert call("gemm_relu_orthogonalize", ORTHO, **over) == gr.OK


@pytest.mark.parametrize("over", [dict(rows=2 ** 16 + 1, cols=2 ** 17, stride=2 ** 17), dict(cols=2 ** 22 + 1, stride=2 ** 23),
                                  dict(batch=65536)])
def test_orthogonalize_past_the_limits(over):
    assert call("gemm_relu_orthogonalize", ORTHO, **over) == gr.EUNSUPPORTED


# ---- the tensor front ends (CPU tensors: every refusal comes before the device is looked at, the last one is it)
def t(*shape, dtype=torch.float16):
    return torch.zeros(shape, dtype=dtype)


F = torch.float32
H = torch.bfloat16


@pytest.mark.parametrize("error,fn", [
    (ValueError, lambda: gr.matmul_act(t(4, 8), t(6, 8), act="swish")),
    (TypeError, lambda: gr.matmul_act([1.0], t(6, 8))),
    (TypeError, lambda: gr.matmul_act(t(4, 8, dtype=F), t(6, 8, dtype=F))),
    (TypeError, lambda: gr.matmul_act(t(4, 8), t(6, 8, dtype=H))),
    (ValueError, lambda: gr.matmul_act(t(4, 8), t(6, 9))),
    (ValueError, lambda: gr.matmul_act(t(4, 8), t(8, 6).t())),
    (ValueError, lambda: gr.matmul_act(t(4, 8), t(2, 3, 8))),
    (ValueError, lambda: gr.matmul_act(t(4, 8), t(6, 8), t(8))),
    (TypeError, lambda: gr.matmul_act(t(4, 8), t(6, 8), t(6, dtype=H))),
    (TypeError, lambda: gr.matmul_act(t(4, 8), t(6, 8), residual=t(4, 6, dtype=F))),
    (ValueError, lambda: gr.matmul_act(t(4, 8), t(6, 8), residual=t(4, 8))),
    (ValueError, lambda: gr.matmul_act(t(4, 8), t(6, 8), residual=t(6, 4).t())),
    (ValueError, lambda: gr.matmul_act(t(4, 8), t(6, 8), t(6), "gelu", t(4, 6))),          # not on a GPU
    (TypeError, lambda: gr.matmul_act_backward(t(4, 6, dtype=H), t(4, 6, dtype=F), t(4, 8), t(6, 8), "silu")),
    (ValueError, lambda: gr.matmul_act_backward(t(4, 5), t(4, 6, dtype=F), t(4, 8), t(6, 8), "silu")),
    (TypeError, lambda: gr.matmul_act_backward(t(4, 6), None, t(4, 8), t(6, 8), "silu")),
    (TypeError, lambda: gr.matmul_act_backward(t(4, 6), t(4, 6), t(4, 8), t(6, 8), "silu")),
    (ValueError, lambda: gr.matmul_act_backward(t(4, 6), t(4, 5, dtype=F), t(4, 8), t(6, 8), "silu")),
    (ValueError, lambda: gr.matmul_act_backward(t(4, 6), None, t(4, 8), t(6, 8), "none", t(5))),
    (ValueError, lambda: gr.matmul_act_backward(t(4, 6), None, t(4, 8), t(6, 8), "none", t(6))),
    (ValueError, lambda: gr.add_norm(t(4, 8), t(4, 8), t(8), norm="batch")),
    (TypeError, lambda: gr.orthogonalize(t(4, 8, dtype=torch.int8))),
    (ValueError, lambda: gr.orthogonalize(t(8))),
    (ValueError, lambda: gr.orthogonalize(t(2, 3, 4, 8))),
    (ValueError, lambda: gr.orthogonalize(t(8, 4).t())),
    (ValueError, lambda: gr.orthogonalize(t(4, 1).expand(4, 8))),
    (ValueError, lambda: gr.orthogonalize(t(4, 8), 65)),
    (ValueError, lambda: gr.orthogonalize(t(4, 8), -1)),
    (ValueError, lambda: gr.orthogonalize(t(4, 8), 2, (1.0, 2.0))),
    (ValueError, lambda: gr.orthogonalize(t(4, 8), 2, [(1.0, 2.0, 3.0)])),
    (ValueError, lambda: gr.orthogonalize(t(4, 8), 2, [(1.0, 2.0, 3.0), (1.0, 2.0)])),
    (TypeError, lambda: gr.orthogonalize(t(4, 8), 1, [("a", "b", "c")])),
    (ValueError, lambda: gr.orthogonalize(t(4, 8))),                                           # not on a GPU
    (TypeError, lambda: gr.add_norm(t(4, 8, dtype=torch.int8), t(4, 8), t(8))),
    (TypeError, lambda: gr.add_norm(t(4, 8), t(4, 8, dtype=F), t(8))),
    (ValueError, lambda: gr.add_norm(t(4, 8), t(4, 7), t(8))),
    (ValueError, lambda: gr.add_norm(t(4, 8), t(4, 8), t(7))),
    (TypeError, lambda: gr.add_norm(t(4, 8), t(4, 8), t(8, dtype=H))),
    (TypeError, lambda: gr.add_norm(t(4, 8), t(4, 8), t(8), t(8, dtype=F))),                   # one type for all of them
    (TypeError, lambda: gr.add_norm(t(4, 8), t(4, 8), t(8), gate=t(8, dtype=F))),
    (TypeError, lambda: gr.add_norm(t(4, 8), t(4, 8), t(8), post_weight=t(8, dtype=F))),
    (TypeError, lambda: gr.add_norm(t(4, 8), t(4, 8), t(8, dtype=F), gate=t(4, 8, dtype=F))),
    (ValueError, lambda: gr.add_norm(t(4, 8), t(4, 8), t(8), gate=t(4, 1))),
    (ValueError, lambda: gr.add_norm(t(4, 8), t(4, 8), bias=t(8))),
    (TypeError, lambda: gr.add_norm(t(4, 8), t(4, 8), t(8), scale="1")),
    (ValueError, lambda: gr.add_norm(t(4, 8), t(4, 8), t(8))),                                 # not on a GPU
    (ValueError, lambda: gr.add_norm_backward(None, t(4, 8), t(4, 8), t(4, 8), t(4, 4, dtype=F), t(8))),
    (ValueError, lambda: gr.add_norm_backward(t(4, 8), t(4, 8), t(4, 8), t(4, 8), t(4, 4, dtype=F))),
    (ValueError, lambda: gr.add_norm_backward(None, None, t(4, 8), t(4, 8), t(4, 4, dtype=F))),
    (TypeError, lambda: gr.add_norm_backward(t(4, 8), t(4, 8, dtype=F), t(4, 8), t(4, 8), t(4, 4, dtype=F), t(8))),
    (TypeError, lambda: gr.add_norm_backward(t(4, 8), t(4, 8), t(4, 8), t(4, 8), t(4, 4), t(8))),
    (ValueError, lambda: gr.add_norm_backward(t(4, 8), t(4, 8), t(4, 8), t(4, 8), t(4, 2, dtype=F), t(8))),
    (ValueError, lambda: gr.add_norm_backward(t(4, 8), t(4, 8), t(4, 8), t(4, 8), t(4, 4, dtype=F), t(8))),
])
def test_front_ends_refuse(error, fn):
    with pytest.raises(error):
        fn()
