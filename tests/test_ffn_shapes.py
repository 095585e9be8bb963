"""Sizes at which the feed-forward kernels change their way of working: K cut into
parts, rows longer than a wave, rings that wrap, tiles that end inside a block.
Bounds as in test_ffn.py.
"""
import os
import sys

import pytest
import torch

import dense_tiled_gemm_relu_amd as gr
from test_ffn import (BF16, F16, F32, F64, gated_check, gated_grad_check, gated_inputs, i8_check, i8_inputs, norm_grad_ref,
                      norm_inputs, norm_ref, close, rnd, shifted, strided)

pytestmark = pytest.mark.gpu


@pytest.fixture(autouse=True)
def _gpu():
    assert torch.cuda.is_available(), "GPU tests need the MI355X"
    yield


# K of dx (2 hidden) or of dweight (rows) cut into parts; ragged ends of K, rows and columns
SPLIT_SIZES = [(2, 3001, 104), (34, 2816, 119), (105, 1664, 64), (7, 2500, 257), (130, 2047, 200), (2048, 64, 64),
               (4097, 33, 65), (3001, 70, 130)]


@pytest.mark.parametrize("dtype", [F16, BF16])
@pytest.mark.parametrize("rows,hidden,cols", SPLIT_SIZES)
def test_gated_backward_with_k_in_parts(rows, hidden, cols, dtype):
    x, w = gated_inputs(rows, hidden, cols, dtype, 7)
    h, gu = gr.matmul_gated(x, w, "silu", save=True)
    gated_check(x, w, "silu", h, gu)
    dh = rnd(8, rows, hidden).to(dtype)
    dx, dw = gr.matmul_gated_backward(dh, gu, x, w, "silu")
    gated_grad_check(dh, gu, x, w, "silu", dx, dw)
    for _ in range(3):                     # the parts are added in one order, whichever ends last
        again = gr.matmul_gated_backward(dh, gu, x, w, "silu")
        assert torch.equal(again[0], dx) and torch.equal(again[1], dw)
    got = gr.matmul_gated_backward(strided(dh, 3), gu, strided(x, 5), strided(w, 1), "silu")
    assert torch.equal(got[0], dx) and torch.equal(got[1], dw)


def test_gated_backward_in_parts_keeps_rows_apart():
    rows, hidden, cols = 34, 2816, 120
    x, w = gated_inputs(rows, hidden, cols, BF16, 9)
    _, gu = gr.matmul_gated(x, w, save=True)
    dh = rnd(10, rows, hidden).to(BF16)
    clean, _ = gr.matmul_gated_backward(dh, gu, x, w)
    bad = dh.clone()
    bad[3, hidden - 1] = float("nan")
    dx, dw = gr.matmul_gated_backward(bad, gu, x, w)
    others = [i for i in range(rows) if i != 3]
    assert torch.isnan(dx[3]).all() and torch.equal(dx[others], clean[others])
    left = [j for j in range(2 * hidden) if j not in (hidden - 1, 2 * hidden - 1)]
    assert torch.isnan(dw[[hidden - 1, 2 * hidden - 1]]).all() and torch.isfinite(dw[left]).all()


def test_gated_backward_in_parts_in_a_graph():
    rows, hidden, cols = 20, 2048, 128
    x, w = gated_inputs(rows, hidden, cols, F16, 11)
    _, gu = gr.matmul_gated(x, w, save=True)
    dh = rnd(12, rows, hidden).to(F16)
    want = gr.matmul_gated_backward(dh, gu, x, w)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        gr.matmul_gated_backward(dh, gu, x, w)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=s):
        out = gr.matmul_gated_backward(dh, gu, x, w)
    for _ in range(4):
        for o in out:
            o.zero_()
        gr.matmul_gated_backward(dh, gu, x, w)
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(p, q) for p, q in zip(out, want))


# rows a workgroup takes in turn: more than the copies it holds ahead; every number of waves a row
@pytest.mark.parametrize("dtype,wdtype", [(F16, F32), (BF16, BF16), (F32, F32)])
@pytest.mark.parametrize("rows,cols", [(3000, 600), (2500, 1030), (9000, 200), (1300, 1537), (600, 2050), (550, 3590),
                                       (530, 5121), (520, 7001), (515, 9000)])
def test_layer_norm_many_rows(rows, cols, dtype, wdtype):
    x, w, b = norm_inputs(rows, cols, dtype, wdtype, rows + cols)
    dy = rnd(13, rows, cols).to(dtype)
    y, mean, rstd = gr.layer_norm(x, w, b, 1e-3, stats=True)
    ref, _, _, slack, _, _ = norm_ref(x, w, b, 1e-3)
    close(y, ref, slack)
    refs, slacks = norm_grad_ref(dy, x, w, mean, rstd)
    got = gr.layer_norm_backward(dy, x, w, mean, rstd)
    for g, r, s in zip(got, refs, slacks):
        close(g, r, s)
    again = gr.layer_norm_backward(shifted(dy), strided(x, 3), w, mean, rstd)
    assert all(torch.equal(p, q) for p, q in zip(got, again))


@pytest.mark.parametrize("cols", [200, 1030, 4096])
def test_layer_norm_backward_keeps_rows_apart(cols):
    rows = 700
    x, w, b = norm_inputs(rows, cols, F16, F32, 15)
    dy = rnd(16, rows, cols).to(F16)
    _, mean, rstd = gr.layer_norm(x, w, b, stats=True)
    clean = gr.layer_norm_backward(dy, x, w, mean, rstd)
    bad = dy.clone()
    bad[rows - 1, cols - 1] = float("inf")
    dx, dw, db = gr.layer_norm_backward(bad, x, w, mean, rstd)
    assert torch.equal(dx[:-1], clean[0][:-1]) and not torch.isfinite(dx[-1]).any()
    assert torch.equal(dw[:-1], clean[1][:-1]) and torch.equal(db[:-1], clean[2][:-1])
    assert not torch.isfinite(dw[-1]) and torch.isinf(db[-1])


# every tile's edge, and K that ends inside a 16-byte piece, a step and a chunk
@pytest.mark.parametrize("rows,hidden,cols", [(1, 9, 8), (17, 8, 9), (33, 17, 71), (3, 1000, 1025), (129, 2051, 72),
                                              (1025, 1030, 68), (257, 4097, 65), (1027, 2003, 150)])
def test_gated_edges(rows, hidden, cols):
    x, w = gated_inputs(rows, hidden, cols, F16, 17)
    h, gu = gr.matmul_gated(x, w, "gelu", save=True)
    gated_check(x, w, "gelu", h, gu)
    assert torch.equal(gr.matmul_gated(shifted(x), strided(w, 3), "gelu"), h)


@pytest.mark.parametrize("rows,n,k", [(1, 17, 16), (18, 33, 17), (5, 1000, 1031), (130, 2051, 129), (1025, 2050, 140),
                                      (2049, 129, 255), (3000, 3001, 65)])
def test_i8_edges(rows, n, k):
    x, sx, w, sw = i8_inputs(rows, n, k, 19)
    y = gr.matmul_i8(x, sx, w, sw, BF16)
    i8_check(x, sx, w, sw, y)
    assert torch.equal(gr.matmul_i8(shifted(x), sx, strided(w, 3), sw, BF16), y)


# a last tile row of a few rows goes to a second launch
@pytest.mark.parametrize("rows,n,k", [(1027, 4006, 1501), (2051, 2000, 2000), (4100, 2002, 1000)])
def test_rows_in_two_launches(rows, n, k):
    assert b"+" in gr.library().gemm_relu_gated_plan(rows, n // 2, k, gr.F16)
    x, w = gated_inputs(rows, n // 2, k, F16, 31)
    h, gu = gr.matmul_gated(x, w, "silu", save=True)
    gated_check(x, w, "silu", h, gu)
    xs, ws = strided(x, 5), strided(w, 3)
    h2, gu2 = gr.matmul_gated(xs, ws, "silu", save=True)
    assert torch.equal(h2, h) and torch.equal(gu2, gu) and torch.equal(gr.matmul_gated(x, w, "silu"), h)
    x, sx, w, sw = i8_inputs(rows, n, k, 33)
    y = gr.matmul_i8(x, sx, w, sw, F32)
    i8_check(x, sx, w, sw, y)
    assert torch.equal(gr.matmul_i8(strided(x, 5), sx, strided(w, 3), sw, F32), y)


def test_inputs_dropped_after_a_call_on_another_stream():
    # the caching allocator may give an input's memory away as soon as it is dropped;
    # the kernel on the other stream must still read what was there
    s = torch.cuda.Stream()
    w = rnd(21, 8192).to(F32)
    b = rnd(22, 8192).to(F32)
    x = rnd(23, 4096, 8192).to(F32)
    want = gr.layer_norm(x, w, b)
    for _ in range(4):
        y = x.clone()
        s.wait_stream(torch.cuda.current_stream())
        out = gr.layer_norm(y, w, b, stream=s)
        del y
        torch.full((4096, 8192), float("nan"), device="cuda")
        s.synchronize()
        assert torch.equal(out, want)


def test_example_trains_and_serves():
    sys.path.insert(0, os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples"))
    import feed_forward
    layer = feed_forward.HalfLayer(cols=264, hidden=520)
    x = rnd(25, 96, 264).to(BF16)
    target = x.roll(1, dims=1)
    # the gradient of x against a central difference of the binary64 layer
    y, saved = layer.forward(x)
    dy = rnd(26, 96, 264).to(BF16)
    dx, _ = layer.backward(dy, saved)

    def loss(xd):
        m = xd.mean(1, keepdim=True)
        n = (xd - m) * (((xd - m) ** 2).mean(1, keepdim=True) + feed_forward.EPS) ** -0.5
        gu = n @ layer.gate_up.to(F64).t()
        g, u = gu[:, :520], gu[:, 520:]
        return ((xd + (g * torch.sigmoid(g) * u) @ layer.down.to(F64).t()) * dy.to(F64)).sum()

    v = rnd(27, 96, 264).to(F64)
    step = 1e-4
    diff = (loss(x.to(F64) + step * v) - loss(x.to(F64) - step * v)) / (2 * step)
    want = (dx.to(F64) * v).sum()
    # bf16 activations and gradients: a few roundings of 2^-8 of each element, of random sign
    assert abs(diff - want) <= 8 * 2.0 ** -8 * (dx.to(F64) * v).norm() * 4
    # a rate at which the same steps in binary64 converge (at 30 they diverge)
    first = layer.step(x, target, 3.0)
    for _ in range(5):
        last = layer.step(x, target, 3.0)
    assert last < first
    exact = layer.forward(x)[0].to(F64)
    served = feed_forward.QuantisedHalfLayer(layer)(x).to(F64)
    # three products of 8-bit operands: each rounds its inputs by up to 1/254 of the row's largest value
    assert (served - exact).norm() <= 0.05 * exact.norm()
