"""A stack of residual feed-forward blocks on the package's operators.

A block takes the last one's output and the residual stream.  It adds the first to the
second (normed, scaled per channel), norms the sum for its own use and leaves

    s = stream + gate * norm(out),  h = act(norm(s) W1^T + b1),  out' = h W2^T + b2.

Both directions run on add_norm and matmul_act; the weights' updates are orthogonalised
momenta, the vectors' plain steps.

    python examples/residual_block.py        # trains a few steps
"""
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import dense_tiled_gemm_relu_amd as gr  # noqa: E402


class Block:
    """Weights of one block, `cols` wide with `hidden` units."""
    NAMES = ("norm", "post", "gate", "w1", "b1", "w2", "b2")

    def __init__(self, cols, hidden, dtype=torch.bfloat16, act="gelu", norm="rms", seed=0):
        gen = torch.Generator(device="cuda")
        gen.manual_seed(seed)

        def randn(*shape):
            return torch.randn(*shape, generator=gen, device="cuda")
        self.act, self.kind = act, norm
        # fp32 vectors beside 16-bit matrices
        self.norm, self.post = (torch.ones(cols, device="cuda") for _ in range(2))
        self.gate = torch.full((cols,), 0.5, device="cuda")
        self.w1, self.b1 = (randn(hidden, cols) * cols ** -0.5).to(dtype), torch.zeros(hidden, device="cuda")
        self.w2, self.b2 = (randn(cols, hidden) * hidden ** -0.5).to(dtype), torch.zeros(cols, device="cuda")

    def options(self):
        return {"gate": self.gate, "post_weight": self.post, "norm": self.kind}

    def forward(self, out, stream):
        """The block's output and the residual stream, and what `backward` needs."""
        s, n, stats = gr.add_norm(out, stream, self.norm, stats=True, **self.options())
        h, z = gr.matmul_act(n, self.w1, self.b1, self.act, save=True)
        return gr.matmul_act(h, self.w2, self.b2), s, (out, stream, stats, n, z, h)

    def backward(self, dout, ds, saved):
        """Gradients of both inputs, and of the weights by name."""
        out, stream, stats, n, z, h = saved
        dh, dw2, db2 = gr.matmul_act_backward(dout, None, h, self.w2, "none", self.b2)
        dn, dw1, db1 = gr.matmul_act_backward(dh, z, n, self.w1, self.act, self.b1)
        dx, dstream, dnorm, _, dgate, dpost = gr.add_norm_backward(dn, ds, out, stream, stats, self.norm, **self.options())
        return dx, dstream, dict(zip(self.NAMES, (dnorm, dpost, dgate, dw1, db1, dw2, db2)))


class Stack:
    """Blocks one after the other, then the sum of the last output and the stream."""

    def __init__(self, blocks):
        self.blocks = blocks
        self.momenta = [{} for _ in blocks]

    def forward(self, x):
        out, stream, saved = x, x, []
        for block in self.blocks:
            out, stream, keep = block.forward(out, stream)
            saved.append(keep)
        y, _ = gr.add_norm(out, stream)
        return y, saved

    def backward(self, dy, saved):
        dout = ds = dy
        grads = []
        for block, keep in zip(reversed(self.blocks), reversed(saved)):
            dout, ds, g = block.backward(dout, ds, keep)
            grads.append(g)
        return dout + ds, grads[::-1]

    def update(self, grads, rate, beta=0.9):
        """Matrices move along the orthogonalised momentum, by `rate` of their usual size."""
        for block, momenta, g in zip(self.blocks, self.momenta, grads):
            for name, d in g.items():
                w = getattr(block, name)
                if w.dim() == 2:
                    m = momenta[name] = beta * momenta[name] + d if name in momenta else d.float()
                    w -= (rate * max(1.0, w.shape[0] / w.shape[1]) ** 0.5) * gr.orthogonalize(m).to(w.dtype)
                else:
                    w -= rate * d.to(w.dtype)

    def step(self, x, target, rate):
        y, saved = self.forward(x)
        error = (y - target).float()
        _, grads = self.backward((2 * error / error.numel()).to(y.dtype), saved)
        self.update(grads, rate)
        return (error * error).mean()


def main():
    torch.manual_seed(1)
    stack = Stack([Block(512, 2048, seed=k) for k in range(3)])
    x = torch.randn(1024, 512, device="cuda").bfloat16()
    target = x.roll(1, dims=1)
    for k in range(8):
        print("step %d: loss %.4f" % (k, stack.step(x, target, rate=0.02)))


if __name__ == "__main__":
    main()
