"""The feed-forward operators return results without an autograd graph, and say so
where a gradient would have been recorded."""
import warnings

import pytest
import torch

import dense_tiled_gemm_relu_amd as gr

F = torch.float32


def t(*shape, dtype=torch.float16, grad=False):
    return torch.zeros(shape, dtype=dtype, requires_grad=grad)


def i(*shape):
    return torch.zeros(shape, dtype=torch.int8)


# one input of each operator requires a gradient (CPU tensors are refused afterwards)
CASES = [
    ("layer_norm:", lambda: gr.layer_norm(t(4, 8, grad=True), t(8))),
    ("layer_norm:", lambda: gr.layer_norm(t(4, 8), t(8, grad=True))),
    ("layer_norm:", lambda: gr.layer_norm(t(4, 8), t(8), t(8, grad=True))),
    ("layer_norm_backward:", lambda: gr.layer_norm_backward(t(4, 8), t(4, 8), t(8, grad=True), t(4, dtype=F), t(4, dtype=F))),
    ("matmul_gated:", lambda: gr.matmul_gated(t(4, 8), t(6, 8, grad=True))),
    ("matmul_gated_backward:", lambda: gr.matmul_gated_backward(t(4, 3), t(4, 6, dtype=F), t(4, 8, grad=True), t(6, 8))),
    ("quantize_rows:", lambda: gr.quantize_rows(t(4, 8, grad=True))),
    ("matmul_i8:", lambda: gr.matmul_i8(i(4, 8), t(4, dtype=F), i(6, 8), t(6, dtype=F, grad=True))),
]


@pytest.mark.parametrize("name,fn", CASES)
def test_a_lost_gradient_is_named(name, fn):
    with pytest.warns(UserWarning, match="^" + name), pytest.raises(ValueError, match="same GPU"):
        fn()


@pytest.mark.parametrize("name,fn", CASES)
def test_nothing_is_lost_where_gradients_are_off(name, fn):
    for off in (torch.no_grad, torch.inference_mode):
        with off(), warnings.catch_warnings():
            warnings.simplefilter("error")
            with pytest.raises(ValueError, match="same GPU"):
                fn()


def test_plain_inputs_give_no_warning():
    with warnings.catch_warnings():
        warnings.simplefilter("error")
        with pytest.raises(ValueError, match="same GPU"):
            gr.layer_norm(t(4, 8), t(8), t(8))


def test_a_warning_made_an_error_is_one():
    with warnings.catch_warnings():
        warnings.simplefilter("error")
        with pytest.raises(UserWarning, match="no autograd graph"):
            gr.layer_norm(t(4, 8, grad=True), t(8))


def test_a_lost_tangent_is_named():
    with torch.autograd.forward_ad.dual_level():
        x = torch.autograd.forward_ad.make_dual(t(4, 8), t(4, 8))
        with pytest.warns(UserWarning, match="^layer_norm:"), pytest.raises(ValueError, match="same GPU"):
            gr.layer_norm(x, t(8))


@pytest.mark.gpu
def test_results_are_the_same_with_the_warning():
    gen = torch.Generator(device="cuda")
    gen.manual_seed(1)
    x = torch.randn(40, 264, generator=gen, device="cuda").half()
    w = torch.randn(264, generator=gen, device="cuda").half()
    want = gr.layer_norm(x, w)
    with pytest.warns(UserWarning, match="^layer_norm:"):
        got = gr.layer_norm(x, w.clone().requires_grad_())
    assert torch.equal(got, want) and not got.requires_grad

    class Norm(torch.autograd.Function):
        """The use that the functions are made for."""
        @staticmethod
        def forward(ctx, x, w):
            y, mean, rstd = gr.layer_norm(x, w, stats=True)
            ctx.save_for_backward(x, w, mean, rstd)
            return y

        @staticmethod
        def backward(ctx, dy):
            return gr.layer_norm_backward(dy.contiguous(), *ctx.saved_tensors)[:2]
    wg = w.clone().requires_grad_()
    with warnings.catch_warnings():
        warnings.simplefilter("error")
        y = Norm.apply(x, wg)
        y.float().sum().backward()
    assert torch.equal(y, want) and wg.grad is not None and wg.grad.any()
