"""Every kernel configuration of the feed-forward products, by name: ragged sizes,
rows further apart than they are long, odd addresses, the exactness of whole
numbers.  Bounds as in test_ffn.py.
"""
import pytest
import torch

import dense_tiled_gemm_relu_amd as gr
from test_ffn import (BF16, F16, F32, F64, gated_check, gated_grad_check, gated_inputs, i8_check, i8_inputs, ints, rnd, shifted,
                      strided)

pytestmark = pytest.mark.gpu


@pytest.fixture(autouse=True)
def _gpu():
    assert torch.cuda.is_available(), "GPU tests need the MI355X"
    yield
    torch.cuda.empty_cache()


T256, T128, T128X2, T64 = "d256x256x32_s4_i16w8", "d128x128x64_s4_i16w8", "d128x128x64_s2w8", "d64x64x64_s4"
G64 = "g64x64x64"
# K of dx is 2 hidden, of dweight rows; both end inside a step, and columns inside a tile
GRADIENTS = [(T256, 1501, 700, 3001), (T256, 2003, 1003, 2003), (T128X2, 2003, 515, 3001), (T128X2, 1003, 1500, 3001),
             (T128, 517, 333, 777), (T128, 1003, 701, 1500), (T64, 300, 333, 257), (G64, 130, 70, 63)]


def gradient_plan(rows, hidden, cols):
    a, b = gr.library().gemm_relu_gated_backward_plan(rows, hidden, cols, gr.F16).decode().split(",")
    assert a == b
    return a


@pytest.mark.parametrize("dtype", [F16, BF16])
@pytest.mark.parametrize("tile,rows,hidden,cols", GRADIENTS)
def test_gradients_on_every_tile(tile, rows, hidden, cols, dtype):
    assert gradient_plan(rows, hidden, cols) == tile
    x, w = gated_inputs(rows, hidden, cols, dtype, 7)
    h, gu = gr.matmul_gated(x, w, "silu", save=True)
    gated_check(x, w, "silu", h, gu)
    dh = rnd(8, rows, hidden).to(dtype)
    dx, dw = gr.matmul_gated_backward(dh, gu, x, w, "silu")
    gated_grad_check(dh, gu, x, w, "silu", dx, dw)
    for xs, ws, ds in [(strided(x, 5), strided(w, 1), strided(dh, 3)), (shifted(x), shifted(w), shifted(dh))]:
        got = gr.matmul_gated_backward(ds, gu, xs, ws, "silu")
        assert torch.equal(got[0], dx) and torch.equal(got[1], dw)


@pytest.mark.parametrize("tile,rows,hidden,cols", GRADIENTS)
def test_gradients_of_whole_numbers_on_every_tile(tile, rows, hidden, cols):
    # g and u small whole numbers, dh -1, 0 or 1: every product and sum is exact
    g, u = ints(1, -3, 3, rows, hidden), ints(2, -3, 3, rows, hidden)
    x, w = ints(3, -1, 1, rows, cols), ints(4, -1, 1, 2 * hidden, cols)
    dh = ints(5, -1, 1, rows, hidden)
    gu = torch.cat([g, u], 1).float()
    d = torch.cat([dh * u * (g > 0), dh * g.clamp(min=0)], 1).to(F64)
    dx, dw = gr.matmul_gated_backward(dh.to(BF16), gu, x.to(BF16), w.to(BF16), "relu")
    assert torch.equal(dx.to(F64), (d @ w.to(F64)).to(BF16).to(F64))
    assert torch.equal(dw.to(F64), (d.t() @ x.to(F64)).to(BF16).to(F64))


@pytest.mark.parametrize("tile,rows,hidden,cols", GRADIENTS)
def test_a_bad_row_stays_apart_on_every_tile(tile, rows, hidden, cols):
    x, w = gated_inputs(rows, hidden, cols, F16, 9)
    _, gu = gr.matmul_gated(x, w, save=True)
    dh = rnd(10, rows, hidden).to(F16)
    clean, _ = gr.matmul_gated_backward(dh, gu, x, w)
    dh[rows - 1, hidden - 1] = float("nan")
    dx, dw = gr.matmul_gated_backward(dh, gu, x, w)
    assert torch.isnan(dx[-1]).all() and torch.equal(dx[:-1], clean[:-1])
    left = [j for j in range(2 * hidden) if j not in (hidden - 1, 2 * hidden - 1)]
    assert torch.isnan(dw[[hidden - 1, 2 * hidden - 1]]).all() and torch.isfinite(dw[left]).all()


# the last tile row's and column's edges, K inside a 16-byte piece
FORWARD = [("k16x16x64_s4", 17, 50, 65), ("k32x32x64_s4", 130, 257, 129), ("k32x48x64_s3", 77, 1500, 515),
           ("k48x32x64_s3", 33, 3500, 129), ("k48x32x64_s3", 40, 3501, 67), (T64, 130, 1500, 65), (T64, 200, 1001, 129),
           (T128, 1027, 1001, 65), (T128X2, 520, 3500, 65), (T128X2, 1027, 2501, 129), (T256, 2050, 2501, 65),
           (T256, 2050, 3500, 131), (T128 + "+k16x16x64_s4", 2050, 1001, 515),
           (T128X2 + "+k16x16x64_s4", 2050, 2000, 515)]


@pytest.mark.parametrize("dtype", [F16, BF16])
@pytest.mark.parametrize("tile,rows,hidden,cols", FORWARD)
def test_gated_on_every_tile(tile, rows, hidden, cols, dtype):
    assert gr.library().gemm_relu_gated_plan(rows, hidden, cols, gr.F16).decode() == tile
    x, w = gated_inputs(rows, hidden, cols, dtype, 17)
    h, gu = gr.matmul_gated(x, w, "gelu_tanh", save=True)
    gated_check(x, w, "gelu_tanh", h, gu)
    assert torch.equal(gr.matmul_gated(shifted(x), strided(w, 3), "gelu_tanh"), h)


@pytest.mark.parametrize("out", [F16, F32])
@pytest.mark.parametrize("tile,rows,hidden,cols", FORWARD)
def test_i8_on_every_tile(tile, rows, hidden, cols, out):
    # twice the K elements a step: twice the K, odd, for the same choice
    n, k = 2 * hidden, 2 * cols - 1
    assert gr.library().gemm_relu_i8_plan(rows, n, k, gr.F16).decode() == tile
    x, sx, w, sw = i8_inputs(rows, n, k, 19)
    y = gr.matmul_i8(x, sx, w, sw, out)
    i8_check(x, sx, w, sw, y)
    assert torch.equal(gr.matmul_i8(shifted(x), sx, strided(w, 3), sw, out), y)


# ---- rows too far apart for the copies' 32-bit offsets, and K of less than 16 bytes
def far_apart(t, stride):
    wide = torch.empty((t.shape[0] - 1) * stride + t.shape[1], dtype=t.dtype, device=t.device)
    out = wide.as_strided(t.shape, (stride, 1))
    out.copy_(t)
    return out


FAR = 2 ** 22 + 1


@pytest.mark.parametrize("rows,hidden", [(1, 1), (70, 40), (130, 65)])
def test_short_far_rows_take_the_register_staged_tile(rows, hidden):
    for dtype in (F16, BF16):
        for cols in (1, 7):
            x, w = gated_inputs(rows, hidden, cols, dtype, 21)
            h, gu = gr.matmul_gated(x, w, "silu", save=True)
            h2, gu2 = gr.matmul_gated(far_apart(x, FAR), far_apart(w, FAR), "silu", save=True)
            gated_check(x, w, "silu", h2, gu2)
            assert torch.equal(h2, h) and torch.equal(gu2, gu)
    for k in (1, 15):
        x, sx, w, sw = i8_inputs(rows, 2 * hidden, k, 23)
        for out in (F16, BF16, F32):
            y = gr.matmul_i8(far_apart(x, FAR), sx, far_apart(w, FAR), sw, out)
            i8_check(x, sx, w, sw, y)
            assert torch.equal(y, gr.matmul_i8(x, sx, w, sw, out))


@pytest.mark.parametrize("tile,rows,hidden,cols", [(T64, 400, 520, 203), (T128, 1030, 520, 515), (T128X2, 4100, 520, 300),
                                                   (T256, 8200, 520, 264)])
def test_up_rows_past_32_bits_from_their_gate_rows(tile, rows, hidden, cols):
    # 520 rows 2^22 elements apart: the up rows start 4.4 GB behind the gate rows
    assert gr.library().gemm_relu_gated_plan(rows, hidden, cols, gr.F16).decode() == tile
    x, w = gated_inputs(rows, hidden, cols, F16, 25)
    h, gu = gr.matmul_gated(x, w, "silu", save=True)
    gated_check(x, w, "silu", h, gu)
    far = far_apart(w, 2 ** 22)
    h2, gu2 = gr.matmul_gated(x, far, "silu", save=True)
    assert torch.equal(h2, h) and torch.equal(gu2, gu)
    dh = rnd(26, rows, hidden).to(F16)
    assert all(torch.equal(p, q) for p, q in zip(gr.matmul_gated_backward(dh, gu, x, far), gr.matmul_gated_backward(dh, gu, x, w)))


def test_i8_rows_past_32_bits_of_the_first():
    rows, n, k = 300, 1100, 200
    x, sx, w, sw = i8_inputs(rows, n, k, 27)
    far = far_apart(w, 2 ** 22)                       # 4.6 GB
    assert torch.equal(gr.matmul_i8(x, sx, far, sw), gr.matmul_i8(x, sx, w, sw))


@pytest.mark.parametrize("rows,hidden,cols", [(1024, 512, 32), (1000, 500, 121), (900, 450, 515)])
def test_far_rows_of_many_tiles(rows, hidden, cols):
    # short rows take the register-staged tile, the last the 32 x 32 one: whole numbers, so
    # both have the dense rows' bits
    x, w = ints(31, -2, 2, rows, cols), ints(32, -2, 2, 2 * hidden, cols)
    for dtype in (F16, BF16):
        h, gu = gr.matmul_gated(x.to(dtype), w.to(dtype), "silu", save=True)
        h2, gu2 = gr.matmul_gated(far_apart(x.to(dtype), FAR), far_apart(w.to(dtype), FAR), "silu", save=True)
        assert torch.equal(gu2.to(F64), x.to(F64) @ w.to(F64).t()) and torch.equal(gu, gu2) and torch.equal(h, h2)
    sx, sw = torch.rand(rows, device="cuda"), torch.rand(2 * hidden, device="cuda")
    xi, wi = x.to(torch.int8), w.to(torch.int8)
    assert torch.equal(gr.matmul_i8(far_apart(xi, FAR), sx, far_apart(wi, FAR), sw), gr.matmul_i8(xi, sx, wi, sw))
