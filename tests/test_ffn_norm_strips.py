"""The norm's backward pass where a wave holds a row (1024 bytes: 512 columns of 16
bits, 256 of fp32) and just past it, over more rows than the device takes at once."""
import pytest
import torch

import dense_tiled_gemm_relu_amd as gr
from test_ffn import BF16, F16, F32, close, norm_grad_ref, norm_inputs, rnd, strided


@pytest.mark.parametrize("cols,strips", [(256, 512), (257, 512), (300, 512), (512, 512), (513, 256)])
def test_workspace_holds_two_strips_a_cu_for_every_type_that_takes_them(cols, strips):
    # 16384 rows fill every turn: no fewer strips than the device has room for
    assert gr.library().gemm_relu_layer_norm_backward_workspace(16384, cols) == strips * 2 * cols * 4


@pytest.mark.gpu
@pytest.mark.parametrize("dtype,wdtype", [(F16, F32), (BF16, BF16), (F32, F32)])
@pytest.mark.parametrize("rows,cols", [(513, 257), (2049, 512), (12000, 300), (9001, 511), (4097, 256), (5000, 513), (20001, 400)])
def test_backward_where_a_wave_holds_a_row(rows, cols, dtype, wdtype):
    x, w, b = norm_inputs(rows, cols, dtype, wdtype, rows + cols)
    dy = rnd(13, rows, cols).to(dtype)
    _, mean, rstd = gr.layer_norm(x, w, b, 1e-3, stats=True)
    refs, slacks = norm_grad_ref(dy, x, w, mean, rstd)
    got = gr.layer_norm_backward(dy, x, w, mean, rstd)
    for g, r, s in zip(got, refs, slacks):
        close(g, r, s)
    again = gr.layer_norm_backward(strided(dy, 3), strided(x, 5), w, mean, rstd)
    assert all(torch.equal(p, q) for p, q in zip(got, again))
