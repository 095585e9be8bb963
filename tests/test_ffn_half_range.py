"""Gated gradients whose dg or du float16 cannot hold: |dh u act'(g)| or |dh act(g)|
of 65520 and more, where dx and dweight are finite.  Bounds as in test_ffn.py.
"""
import pytest
import torch

import dense_tiled_gemm_relu_amd as gr
from test_ffn import ACTS, BF16, F16, F64, act_ref, gated_grad_check, ints, rnd, shifted, strided
from test_ffn_tiles import GRADIENTS

pytestmark = pytest.mark.gpu
LIMIT = 65520.0


@pytest.fixture(autouse=True)
def _gpu():
    assert torch.cuda.is_available(), "GPU tests need the MI355X"
    yield


def inputs(rows, hidden, cols, seed, dtype=F16):
    """x and w so small that gradients of some 10^5 keep dx and dweight in range."""
    return ((rnd(seed, rows, cols) * 2.0 ** -9).to(dtype), (rnd(seed + 1, 2 * hidden, cols) * 2.0 ** -9).to(dtype),
            rnd(seed + 2, rows, hidden).to(dtype), rnd(seed + 3, rows, 2 * hidden))


def over(dh, gu, act, hidden):
    """Which elements of dg and du pass float16."""
    g, u = gu.to(F64)[:, :hidden], gu.to(F64)[:, hidden:]
    value, slope = act_ref(g, act)
    return (dh.to(F64) * u * slope).abs() >= LIMIT, (dh.to(F64) * value).abs() >= LIMIT


def plant(dh, gu, hidden, at, kind):
    """Element `at` of dg (a large u) or of du (a large g) past the range."""
    r, j = at
    dh[r, j] = 2000.0 if (r + j) % 2 else -2000.0
    gu[r, j] = 1.0 if kind == "gate" else 40.0
    gu[r, hidden + j] = 40.0 if kind == "gate" else 1.0


@pytest.mark.parametrize("tile,rows,hidden,cols", GRADIENTS + [("k in parts", 34, 2816, 119), ("k in parts", 2048, 64, 64),
                                                               ("few", 1, 1, 1), ("few", 3, 5, 200)])
@pytest.mark.parametrize("kind", ["gate", "up"])
def test_single_elements(tile, rows, hidden, cols, kind):
    x, w, dh, gu = inputs(rows, hidden, cols, 1)
    spots = {(0, 0), (rows - 1, hidden - 1), (rows // 2, hidden // 3), (rows // 2, hidden // 2), (rows // 3, hidden - 1)}
    for at in spots:
        plant(dh, gu, hidden, at, kind)
    og, ou = over(dh, gu, "silu", hidden)
    assert int((og | ou).sum()) == len(spots) and bool((og if kind == "gate" else ou).any())
    dx, dw = gr.matmul_gated_backward(dh, gu, x, w, "silu")
    gated_grad_check(dh, gu, x, w, "silu", dx, dw)
    for xs, ws, ds in [(strided(x, 5), strided(w, 1), strided(dh, 3)), (shifted(x), shifted(w), shifted(dh))]:
        got = gr.matmul_gated_backward(ds, gu, xs, ws, "silu")
        assert torch.equal(got[0], dx) and torch.equal(got[1], dw)
    # rows of dx and of dweight that hold none of them are what they are without them
    rest = dh.clone()
    for at in spots:
        rest[at] = 0.0
    dx0, dw0 = gr.matmul_gated_backward(rest, gu, x, w, "silu")
    rows_left = ~(og | ou).any(1)
    units_left = torch.cat([~(og | ou).any(0)] * 2)
    assert torch.equal(dx[rows_left], dx0[rows_left]) and torch.equal(dw[units_left], dw0[units_left])


@pytest.mark.parametrize("act", ACTS)
@pytest.mark.parametrize("rows,hidden,cols", [(5, 7, 70), (130, 70, 63), (300, 333, 257), (517, 333, 777)])
def test_whole_gradients(rows, hidden, cols, act):
    x, w, dh, gu = inputs(rows, hidden, cols, 11)
    dh = (dh.float() * 15000).clamp(-60000, 60000).to(F16)
    gu = gu * 4
    og, ou = over(dh, gu, act, hidden)
    assert og.any() and ou.any() and not (og & ou).all()
    dx, dw = gr.matmul_gated_backward(dh, gu, x, w, act)
    assert torch.isfinite(dx).all() and torch.isfinite(dw).all()
    gated_grad_check(dh, gu, x, w, act, dx, dw)
    again = gr.matmul_gated_backward(dh, gu, x, w, act)
    assert torch.equal(again[0], dx) and torch.equal(again[1], dw)


@pytest.mark.parametrize("rows,hidden,cols", [(70, 130, 65), (300, 333, 257)])
def test_whole_numbers_on_both_sides_of_the_limit(rows, hidden, cols):
    # du = dh g: 65504 is the largest float16, 65519 rounds to it, 65520 would round to
    # infinity; x picks single rows and columns, so that each result is one product
    g = torch.tensor([8188.0, 8189.875, 8190.0, 8191.0, 16000.0], device="cuda")
    gu = torch.ones(rows, 2 * hidden, device="cuda")
    gu[:, :hidden] = g[ints(1, 0, 4, rows, hidden)]
    dh = (8 * ints(2, -1, 1, rows, hidden)).to(F16)
    x = torch.zeros(rows, cols, dtype=F16, device="cuda")
    pick = ints(3, 0, rows - 1, cols)
    x[pick, torch.arange(cols, device="cuda")] = 2.0 ** -3
    w = torch.zeros(2 * hidden, cols, dtype=F16, device="cuda")
    unit = ints(4, 0, hidden - 1, cols)
    w[hidden + unit, torch.arange(cols, device="cuda")] = 2.0 ** -3
    dx, dw = gr.matmul_gated_backward(dh, gu, x, w, "relu")
    du = dh.to(F64) * gu[:, :hidden].to(F64)
    passed = du.abs() >= LIMIT
    rounded = du.clamp(-65504, 65504)            # an element that stays in range is rounded to 16 bits
    for got, row_passed, pair in ((dx, passed.any(1), lambda d: d[:, unit] / 8), (dw[hidden:], passed.any(0), lambda d: d.t()[:, pick] / 8)):
        want = torch.where(row_passed[:, None], pair(du), pair(rounded))
        assert torch.equal(got, want.to(F16))


def test_infinities_and_nan_stay_what_they_are():
    rows, hidden, cols = 300, 200, 257
    x, w, dh, gu = inputs(rows, hidden, cols, 21)
    plant(dh, gu, hidden, (5, 70), "gate")
    want = gr.matmul_gated_backward(dh, gu, x, w, "silu")
    bad = dh.clone()
    bad[6, 71] = float("inf")
    bad[200, 3] = float("nan")
    bad[5, 72] = float("inf")                    # in a row that passes the range too
    dx, dw = gr.matmul_gated_backward(bad, gu, x, w, "silu")
    assert not torch.isfinite(dx[[5, 6, 200]]).any()
    left = [i for i in range(rows) if i not in (5, 6, 200)]
    assert torch.equal(dx[left], want[0][left])
    for k in (3, 71, 72):
        assert not torch.isfinite(dw[[k, hidden + k]]).any()
    left = [j for j in range(2 * hidden) if j % hidden not in (3, 71, 72)]
    assert torch.equal(dw[left], want[1][left])


def test_bfloat16_holds_them_itself():
    rows, hidden, cols = 130, 70, 200
    x, w, dh, gu = inputs(rows, hidden, cols, 31, BF16)
    dh = dh * 30000
    gated_grad_check(dh, gu, x, w, "gelu", *gr.matmul_gated_backward(dh, gu, x, w, "gelu"))


def test_in_a_graph():
    rows, hidden, cols = 200, 130, 257
    x, w, small, gu = inputs(rows, hidden, cols, 41)
    large = small.clone()
    large[7, 9] = large[150, 129] = 60000.0
    gu[7, hidden + 9] = gu[150, hidden + 129] = 30.0
    gu[7, 9] = gu[150, 129] = 1.0
    wants = [gr.matmul_gated_backward(d, gu, x, w) for d in (small, large)]
    assert all(torch.isfinite(t).all() for pair in wants for t in pair)
    dh = small.clone()
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        gr.matmul_gated_backward(dh, gu, x, w)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=s):
        out = gr.matmul_gated_backward(dh, gu, x, w)
    for k in range(5):
        dh.copy_((small, large)[k % 2])
        for o in out:
            o.zero_()
        gr.matmul_gated_backward(small, gu, x, w)
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(p, q) for p, q in zip(out, wants[k % 2])), k
