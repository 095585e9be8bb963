"""The gated backward pass's workspace, on the host: the size that the workspace
function gives for dense rows is what every call takes, to the byte."""
import itertools

import pytest
import torch

import dense_tiled_gemm_relu_amd as gr

DH, GU, X, W, DX, DW, WS = (i << 56 for i in range(1, 8))      # fake addresses: inspected, never read

# with a GPU at hand the accepted calls would run on them
pytestmark = pytest.mark.skipif(torch.cuda.is_available(), reason="fake addresses")

SIZES = [(1, 1, 1), (34, 2816, 119), (2, 3001, 104), (105, 1664, 64), (2048, 64, 64), (4097, 33, 65), (1027, 2003, 1501),
         (320, 704, 4096), (4096, 7168, 4096), (300, 200, 2 ** 24 + 5), (40, 900, 2 ** 24 - 3)]
CUT = [(34, 2816, 119), (2, 3001, 104), (105, 1664, 64), (2048, 64, 64)]        # K in parts


def backward(rows, hidden, cols, pad_dh, pad_x, pad_w, ws_bytes):
    return gr.library().gemm_relu_gated_backward(
        DH, hidden + pad_dh, GU, X, cols + pad_x, W, cols + pad_w, DX, DW, rows, hidden, cols, gr.BF16, 0, WS, ws_bytes, 0)


@pytest.mark.parametrize("rows,hidden,cols", SIZES)
def test_the_dense_size_serves_every_stride(rows, hidden, cols):
    need = gr.library().gemm_relu_gated_backward_workspace(rows, hidden, cols)
    for pads in itertools.product((0, 3), (0, 5, 2 ** 22, 2 ** 24, 2 ** 30), (0, 7, 2 ** 22, 2 ** 24, 2 ** 30)):
        assert backward(rows, hidden, cols, *pads, need) != gr.EINVAL, pads


@pytest.mark.parametrize("rows,hidden,cols", SIZES)
def test_a_byte_less_is_refused(rows, hidden, cols):
    need = gr.library().gemm_relu_gated_backward_workspace(rows, hidden, cols)
    assert backward(rows, hidden, cols, 0, 0, 0, need - 1) == gr.EINVAL


@pytest.mark.parametrize("rows,hidden,cols", CUT)
def test_parts_of_k_have_their_sums_and_counters(rows, hidden, cols):
    # beside dg and du in both layouts (rows of 16 bytes, 256-byte pieces): at least two
    # parts of a 64 x 64 tile of fp32 sums, and a counter
    def pieces(n):
        return -(-n // 256) * 256
    both = (pieces(2 * rows * (-(-2 * hidden // 8) * 8)) + pieces(2 * 2 * hidden * (-(-rows // 8) * 8)))
    need = gr.library().gemm_relu_gated_backward_workspace(rows, hidden, cols)
    assert need >= both + pieces(4) + 2 * 64 * 64 * 4
    assert b"d64x64x64_s4,d64x64x64_s4" == gr.library().gemm_relu_gated_backward_plan(rows, hidden, cols, gr.BF16)
