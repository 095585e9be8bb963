"""The operators around the half layer return results without an autograd graph, and say
so where a gradient would have been recorded."""
import warnings

import pytest
import torch

import dense_tiled_gemm_relu_amd as gr

F = torch.float32


def t(*shape, dtype=torch.float16, grad=False):
    return torch.zeros(shape, dtype=dtype, requires_grad=grad)


# one input of each operator requires a gradient (CPU tensors are refused afterwards)
CASES = [
    ("matmul_act:", lambda: gr.matmul_act(t(4, 8, grad=True), t(6, 8))),
    ("matmul_act:", lambda: gr.matmul_act(t(4, 8), t(6, 8), t(6, grad=True))),
    ("matmul_act:", lambda: gr.matmul_act(t(4, 8), t(6, 8), residual=t(4, 6, grad=True))),
    ("matmul_act_backward:", lambda: gr.matmul_act_backward(t(4, 6), None, t(4, 8), t(6, 8, grad=True))),
    ("add_norm:", lambda: gr.add_norm(t(4, 8), t(4, 8, grad=True), t(8))),
    ("add_norm:", lambda: gr.add_norm(t(4, 8), t(4, 8), t(8), gate=t(8, grad=True))),
    ("add_norm:", lambda: gr.add_norm(t(4, 8), t(4, 8), t(8), post_weight=t(8, grad=True))),
    ("add_norm_backward:", lambda: gr.add_norm_backward(t(4, 8), None, t(4, 8), t(4, 8), t(4, 4, dtype=F), t(8, grad=True))),
    ("orthogonalize:", lambda: gr.orthogonalize(t(4, 8, grad=True))),
]


@pytest.mark.parametrize("name,fn", CASES)
def test_a_lost_gradient_is_named(name, fn):
    with pytest.warns(UserWarning, match="^" + name), pytest.raises(ValueError, match="same GPU"):
        fn()


@pytest.mark.parametrize("name,fn", CASES)
def test_nothing_is_lost_where_gradients_are_off(name, fn):
    with torch.no_grad(), warnings.catch_warnings():
        warnings.simplefilter("error")
        with pytest.raises(ValueError, match="same GPU"):
            fn()
