"""What is no tensor is refused alike, whether or not the front end has been loaded."""
import numpy
import pytest
import torch

import dense_tiled_gemm_relu_amd as gr


def t(*shape, dtype=torch.float16):
    return torch.zeros(shape, dtype=dtype)


F, I8 = torch.float32, torch.int8


@pytest.mark.parametrize("x", [None, 1.0, [[1.0]], numpy.zeros((4, 8), numpy.float16)])
@pytest.mark.parametrize("name,fn", [
    ("layer_norm", lambda x: gr.layer_norm(x, t(8))),
    ("layer_norm_backward", lambda x: gr.layer_norm_backward(t(4, 8), x, t(8), t(4, dtype=F), t(4, dtype=F))),
    ("matmul_gated", lambda x: gr.matmul_gated(x, t(6, 8))),
    ("matmul_gated_backward", lambda x: gr.matmul_gated_backward(t(4, 3), t(4, 6, dtype=F), x, t(6, 8))),
    ("quantize_rows", gr.quantize_rows),
    ("matmul_i8", lambda x: gr.matmul_i8(x, t(4, dtype=F), t(6, 8, dtype=I8), t(6, dtype=F))),
])
def test_x_must_be_a_tensor(name, fn, x):
    for _ in range(2):                     # the second call finds the front end loaded
        with pytest.raises(TypeError, match="x must be a tensor"):
            fn(x)
