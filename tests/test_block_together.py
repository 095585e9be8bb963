"""The operators around the half layer used together: on streams, in graphs, as a stack of
blocks with its gradients."""
import importlib.util
import os

import pytest
import torch

import dense_tiled_gemm_relu_amd as gr
from tests.block_helpers import BF16, F16, F32, F64, act_ref, half_step, rnd

pytestmark = pytest.mark.gpu


def block(x, r, w, gate, w1, b1, w2, dy, ds, stream=None):
    """A training step through every operator."""
    options = {"gate": gate, "scale": 0.5, "post_weight": w, "norm": "layer"}
    s, n, stats = gr.add_norm(x, r, w, w, stats=True, stream=stream, **options)
    h, z = gr.matmul_act(n, w1, b1, "gelu", save=True, stream=stream)
    y = gr.matmul_act(h, w2, None, "none", s, stream=stream)
    dh, dw2, _ = gr.matmul_act_backward(dy, None, h, w2, stream=stream)
    dn, dw1, db1 = gr.matmul_act_backward(dh, z, n, w1, "gelu", b1, stream=stream)
    grads = gr.add_norm_backward(dn, ds, x, r, stats, w, w, stream=stream, **options)
    return (s, n, h, z, y, dw2, dw1, db1, *grads, gr.orthogonalize(dw1, stream=stream), gr.orthogonalize(dw2, 3, stream=stream))


def inputs(rows, cols, hidden, seed, dtype=BF16):
    return (rnd(seed, rows, cols).to(dtype), rnd(seed + 1, rows, cols).to(dtype), 1 + 0.1 * rnd(seed + 2, cols),
            0.5 + 0.1 * rnd(seed + 3, cols), (rnd(seed + 4, hidden, cols) * cols ** -0.5).to(dtype), 0.1 * rnd(seed + 5, hidden),
            (rnd(seed + 6, cols, hidden) * hidden ** -0.5).to(dtype), rnd(seed + 7, rows, cols).to(dtype),
            rnd(seed + 8, rows, cols).to(dtype))


SIZES = [(1, 264, 72), (40, 520, 264), (300, 520, 1040), (129, 33, 65)]


@pytest.mark.parametrize("rows,cols,hidden", SIZES)
def test_on_another_stream(rows, cols, hidden):
    args = inputs(rows, cols, hidden, 81)
    want = block(*args)
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    for given in (s, s.cuda_stream, 0):
        got = block(*args, stream=given)
        torch.cuda.synchronize()
        assert all(torch.equal(p, q) for p, q in zip(got, want))
    with torch.cuda.stream(s):
        got = block(*args)
    s.synchronize()
    assert all(torch.equal(p, q) for p, q in zip(got, want))


def test_two_streams_at_once():
    a, b = inputs(300, 520, 1040, 11), inputs(300, 520, 1040, 12)
    want = block(*a), block(*b)
    streams = torch.cuda.Stream(), torch.cuda.Stream()
    torch.cuda.synchronize()
    for _ in range(3):
        got = [block(*args, stream=s) for args, s in zip((a, b), streams)]
        torch.cuda.synchronize()
        for g, w in zip(got, want):
            assert all(torch.equal(p, q) for p, q in zip(g, w))


@pytest.mark.parametrize("rows,cols,hidden", SIZES)
def test_captured_into_a_graph(rows, cols, hidden):
    args, other = inputs(rows, cols, hidden, 91), inputs(rows, cols, hidden, 191)
    want, want2 = block(*args), block(*other)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        block(*args)
    torch.cuda.synchronize()
    graphs, outs = [], []
    for _ in range(2):                     # two graphs of the same step, each with workspaces of its own
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=s):
            outs.append(block(*args))
        graphs.append(graph)
    kept = [a.clone() for a in args]
    for k in range(4):                     # the program's own work in between, and other inputs every second time
        for a, n in zip(args, other if k % 2 else kept):
            a.copy_(n)
        for out in outs:
            for o in out:
                if o.data_ptr() not in (args[8].data_ptr(),):
                    o.zero_()
        block(*other)
        graphs[0].replay()
        graphs[1].replay()
        torch.cuda.synchronize()
        for out in outs:
            assert all(torch.equal(p, q) for p, q in zip(out, want2 if k % 2 else want)), k


def test_batched_and_small_orthogonalisations_in_a_graph():
    shapes = [(50, 100), (3, 128, 200), (300, 700), (2, 1030, 600)]
    gs = [rnd(k, *shape).to(BF16) for k, shape in enumerate(shapes)]
    want = [gr.orthogonalize(g) for g in gs]
    s = torch.cuda.Stream()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=s):
        out = [gr.orthogonalize(g) for g in gs]
    for k in range(3):
        for o in out:
            o.zero_()
        [gr.orthogonalize(g.flip(0)) for g in gs]
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(p, q) for p, q in zip(out, want)), k


def load_example():
    path = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples", "residual_block.py")
    spec = importlib.util.spec_from_file_location("residual_block", path)
    module = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(module)
    return module


@pytest.mark.parametrize("kind,act", [("rms", "gelu"), ("layer", "silu")])
def test_example_gradients(kind, act):
    # against binary64 automatic differentiation of the formulas.  A result passes at most 20
    # roundings to float16 on its way through two blocks, each half a step of the norm of what
    # it rounds, and the blocks pass such a change on with gains near 1: 32 half steps.
    ex = load_example()
    stack = ex.Stack([ex.Block(136, 264, F16, act, kind, seed=k) for k in range(2)])
    for k, b in enumerate(stack.blocks):
        b.norm += 0.2 * rnd(30 + k, 136)
        b.post += 0.2 * rnd(40 + k, 136)
        b.b1 += 0.2 * rnd(50 + k, 264)
        b.b2 += 0.2 * rnd(60 + k, 136)
    x, dy = rnd(1, 75, 136).to(F16), rnd(2, 75, 136).to(F16)
    y, saved = stack.forward(x)
    dx, grads = stack.backward(dy, saved)

    def normed(v):
        if kind == "layer":
            v = v - v.mean(1, keepdim=True)
        return v * ((v * v).mean(1, keepdim=True) + 1e-5) ** -0.5
    xd = x.to(F64).requires_grad_()
    out, stream, leaves = xd, xd, []
    for b in stack.blocks:
        p = {n: getattr(b, n).to(F64).requires_grad_() for n in b.NAMES}
        stream = stream + p["gate"] * (normed(out) * p["post"])
        out = act_ref(normed(stream) * p["norm"] @ p["w1"].t() + p["b1"], act)[0] @ p["w2"].t() + p["b2"]
        leaves.append(p)
    want = out + stream
    want.backward(dy.to(F64))

    def near(got, ref):
        assert (got.to(F64) - ref).norm() <= 32 * half_step(F16) * ref.norm()
    near(y, want.detach())
    near(dx, xd.grad)
    for g, p in zip(grads, leaves):
        for n in p:
            near(g[n], p[n].grad)


def test_example_trains():
    ex = load_example()
    stack = ex.Stack([ex.Block(72, 200, BF16, seed=k) for k in range(2)])
    x = rnd(3, 50, 72).to(BF16)
    before = [b.w1.clone() for b in stack.blocks]
    losses = [stack.step(x, x.roll(1, dims=1), 0.02) for _ in range(3)]
    assert all(torch.isfinite(v) for v in losses)
    assert all(not torch.equal(b.w1, w) for b, w in zip(stack.blocks, before))
    assert stack.momenta[0]["w1"].dtype == F32
