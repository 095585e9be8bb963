"""A transformer's feed-forward half layer on the package's operators.

    y = x + Wd (act(norm(x) Wg^T) * (norm(x) Wu^T))

A training step runs the norm and the gated projections forward and backward; the
down projection, a plain matrix product, is torch's, and so is the optimiser's
update.  The serving path holds all three weights in 8 bits, one scale per output
channel, and quantises the activations row by row on the way in.

    python examples/feed_forward.py        # trains a few steps, then serves one batch
"""
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import dense_tiled_gemm_relu_amd as gr  # noqa: E402

EPS = 1e-5


class HalfLayer:
    """Weights of one half layer: `cols` wide, `hidden` gated units."""

    def __init__(self, cols, hidden, dtype=torch.bfloat16, act="silu", seed=0):
        gen = torch.Generator(device="cuda")
        gen.manual_seed(seed)

        def randn(*shape):
            return torch.randn(*shape, generator=gen, device="cuda")
        self.act = act
        self.norm_w = torch.ones(cols, device="cuda")                # fp32 beside 16-bit activations
        self.norm_b = torch.zeros(cols, device="cuda")
        self.gate_up = (randn(2 * hidden, cols) * cols ** -0.5).to(dtype)   # gate rows, then up rows
        self.down = (randn(cols, hidden) * hidden ** -0.5).to(dtype)

    def forward(self, x):
        """The output, and what `backward` needs."""
        n, mean, rstd = gr.layer_norm(x, self.norm_w, self.norm_b, EPS, stats=True)
        h, gu = gr.matmul_gated(n, self.gate_up, self.act, save=True)
        return x + h @ self.down.t(), (x, n, mean, rstd, h, gu)

    def backward(self, dy, saved):
        """Gradients of x and of (norm_w, norm_b, gate_up, down)."""
        x, n, mean, rstd, h, gu = saved
        ddown = dy.t() @ h
        dn, dgate_up = gr.matmul_gated_backward(dy @ self.down, gu, n, self.gate_up, self.act)
        dx, dw, db = gr.layer_norm_backward(dn, x, self.norm_w, mean, rstd)
        return dx + dy, (dw, db, dgate_up, ddown)

    def step(self, x, target, rate):
        """One step of gradient descent on the squared error; returns the loss."""
        y, saved = self.forward(x)
        error = (y - target).float()
        _, grads = self.backward((2 * error / error.numel()).to(y.dtype), saved)
        for w, g in zip((self.norm_w, self.norm_b, self.gate_up, self.down), grads):
            w -= rate * g
        return (error * error).mean()


class QuantisedHalfLayer:
    """The same layer for serving, its weights in 8 bits."""

    def __init__(self, layer):
        self.layer = layer
        hidden = layer.gate_up.shape[0] // 2
        self.gate, self.up = (gr.quantize_rows(w) for w in (layer.gate_up[:hidden], layer.gate_up[hidden:]))
        self.down = gr.quantize_rows(layer.down)

    def __call__(self, x):
        n = gr.layer_norm(x, self.layer.norm_w, self.layer.norm_b, EPS)
        q, s = gr.quantize_rows(n)
        g, u = (gr.matmul_i8(q, s, w, ws, x.dtype) for w, ws in (self.gate, self.up))
        h = torch.nn.functional.silu(g) * u
        return x + gr.matmul_i8(*gr.quantize_rows(h), *self.down, x.dtype)


def main():
    torch.manual_seed(1)
    layer = HalfLayer(cols=1024, hidden=2816)
    x = torch.randn(512, 1024, device="cuda").bfloat16()
    target = x.roll(1, dims=1)
    for k in range(5):
        print("step %d: loss %.4f" % (k, layer.step(x, target, rate=20.0)))
    exact = layer.forward(x)[0]
    served = QuantisedHalfLayer(layer)(x)
    print("8-bit weights: relative difference %.4f" % ((served - exact).float().norm() / exact.float().norm()))


if __name__ == "__main__":
    main()
