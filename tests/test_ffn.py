"""The feed-forward operators on the GPU, against their definitions in binary64.

Tolerances are bounds on the kernels' arithmetic: one rounding of the result
(half a step of its type), fp32 sums of n terms (n 2^-24 of the sum of
magnitudes, whatever the order), a few fp32 steps for the activations, and for
the gated gradients the rounding of dg and du to 16 bits.
"""
import math

import pytest
import torch

import dense_tiled_gemm_relu_amd as gr

pytestmark = pytest.mark.gpu

F16, BF16, F32, F64 = torch.float16, torch.bfloat16, torch.float32, torch.float64
U = 2.0 ** -24                                             # half a step of fp32
# smallest step of a result, for values below the normal range
TINY = {F16: 2.0 ** -24, BF16: 2.0 ** -133, F32: 2.0 ** -149}


@pytest.fixture(autouse=True)
def _gpu():
    assert torch.cuda.is_available(), "GPU tests need the MI355X"
    yield


def half_step(t):
    return torch.finfo(t).eps / 2


def rnd(seed, *shape):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(seed)
    return torch.randn(*shape, generator=gen, device="cuda")


def close(got, ref, slack):
    """|got - ref| <= one rounding of ref to got's type + slack, everywhere."""
    assert got.shape == ref.shape
    err = (got.to(F64) - ref).abs()
    bound = half_step(got.dtype) * (ref.abs() + slack) + slack + TINY[got.dtype]
    bad = ~(err <= bound)
    if bad.any():
        at = bad.nonzero()[:4]
        raise AssertionError("%d of %d off, first at %s: %s, not %s (bound %s)" % (
            int(bad.sum()), bad.numel(), at.tolist(), got[bad][:4].tolist(), ref[bad][:4].tolist(),
            bound[bad][:4].tolist()))


def strided(t, pad):
    """t with rows `pad` elements further apart than they are long."""
    wide = torch.full((t.shape[0], t.shape[1] + pad), 77 if t.dtype == torch.int8 else float("nan"), dtype=t.dtype,
                      device=t.device)
    wide[:, :t.shape[1]] = t
    return wide[:, :t.shape[1]]


def shifted(t):
    """t one element past an aligned address."""
    flat = torch.empty(t.numel() + 1, dtype=t.dtype, device=t.device)
    flat[1:] = t.reshape(-1)
    return flat[1:].view(t.shape)


# ------------------------------------------------------------- layer norm
def norm_ref(x, w, b, eps):
    x, w = x.to(F64), w.to(F64)
    b = torch.zeros_like(w) if b is None else b.to(F64)
    mean = x.mean(-1, keepdim=True)
    var = ((x - mean) ** 2).mean(-1, keepdim=True)
    rstd = (var + eps) ** -0.5
    steps = (x.shape[-1] / 64 + 16) * U
    off = steps * x.abs().mean(-1, keepdim=True)              # of the mean
    lost = 2 * steps + off ** 2 / (2 * (var + eps))           # of rstd, relative
    slack = off * rstd * w.abs() + lost * ((x - mean) * rstd * w).abs() + 4 * U * b.abs()
    return (x - mean) * rstd * w + b, mean[..., 0], rstd[..., 0], slack, off[..., 0], (lost * rstd)[..., 0]


NORM_SIZES = [(1, 1), (3, 2), (2, 7), (5, 64), (4, 100), (67, 257), (130, 512), (9, 1000), (33, 2048), (6, 3001),
              (129, 4096), (3, 5003), (2, 8191), (4, 8192), (3, 16384), (2, 20001), (2, 40000)]


def norm_inputs(rows, cols, dtype, wdtype, seed, offset=0.5):
    x = (rnd(seed, rows, cols) * (1 + 7 * (rnd(seed + 1, cols).abs() > 2)) + offset).to(dtype)
    return x, (1 + 0.3 * rnd(seed + 2, cols)).to(wdtype), (0.2 * rnd(seed + 3, cols)).to(wdtype)


@pytest.mark.parametrize("dtype,wdtype", [(F16, F16), (F16, F32), (BF16, BF16), (BF16, F32), (F32, F32)])
@pytest.mark.parametrize("rows,cols", NORM_SIZES)
def test_layer_norm(rows, cols, dtype, wdtype):
    x, w, b = norm_inputs(rows, cols, dtype, wdtype, rows * 31 + cols)
    ref, mean, rstd, slack, off_mean, off_rstd = norm_ref(x, w, b, 1e-5)
    y, m, r = gr.layer_norm(x, w, b, 1e-5, stats=True)
    assert y.dtype == dtype and m.dtype == r.dtype == F32
    close(y, ref, slack)
    close(m, mean, off_mean + 4 * U * mean.abs())
    close(r, rstd, off_rstd + 4 * U * rstd)
    assert torch.equal(gr.layer_norm(x, w, b, 1e-5), y)
    close(gr.layer_norm(x, w, eps=1e-5), norm_ref(x, w, None, 1e-5)[0], slack)


@pytest.mark.parametrize("cols", [256, 1000, 4096, 20001])
def test_layer_norm_large_offset_and_constant_rows(cols):
    # mean 300 times the spread; a row without spread is bias (eps keeps rstd finite)
    x, w, b = norm_inputs(6, cols, F32, F32, 5, offset=300.0)
    x[2] = 3.25
    ref, _, _, slack, _, _ = norm_ref(x, w, b, 1e-5)
    y = gr.layer_norm(x, w, b, 1e-5)
    close(y, ref, slack)
    if cols <= 4096:                                        # sums of 3.25 that fp32 holds exactly
        assert torch.equal(y[2], b)


@pytest.mark.parametrize("dtype", [F16, BF16, F32])
@pytest.mark.parametrize("cols", [64, 1000, 8192, 20001])
def test_layer_norm_non_finite_rows_stay_apart(cols, dtype):
    x, w, b = norm_inputs(9, cols, dtype, dtype, 6)
    clean, m0, r0 = gr.layer_norm(x, w, b, stats=True)
    x[1, cols // 2] = float("nan")
    x[4, 0] = float("inf")
    x[7, cols - 1] = float("-inf")
    y = gr.layer_norm(x, w, b)
    bad = [1, 4, 7]
    good = [i for i in range(9) if i not in bad]
    assert torch.isnan(y[bad]).all()
    assert torch.equal(y[good], clean[good])


def test_layer_norm_shapes_strides_and_alignment():
    x, w, b = norm_inputs(24, 1001, F16, F32, 7)
    y = gr.layer_norm(x, w, b)
    assert torch.equal(gr.layer_norm(x.view(2, 3, 4, 1001), w, b).view(24, 1001), y)
    assert torch.equal(gr.layer_norm(x[0], w, b), y[0])
    assert torch.equal(gr.layer_norm(strided(x, 5), w, b), y)
    assert torch.equal(gr.layer_norm(shifted(x), shifted(w), shifted(b)), y)
    assert gr.layer_norm(x[:0], w, b).shape == (0, 1001)


def norm_grad_ref(dy, x, w, mean, rstd):
    dy, x, w = dy.to(F64), x.to(F64), w.to(F64)
    rows, cols = x.shape
    xhat = (x - mean.to(F64)[:, None]) * rstd.to(F64)[:, None]
    # x - mean rounds once to fp32
    c = dy * w
    s0, s1 = c.mean(1, keepdim=True), (c * xhat).mean(1, keepdim=True)
    dx = rstd.to(F64)[:, None] * (c - s0 - xhat * s1)
    steps = (cols / 64 + 16) * U
    slack = steps * rstd.to(F64)[:, None] * (c.abs() + c.abs().mean(1, keepdim=True) +
                                             2 * xhat.abs() * (c * xhat).abs().mean(1, keepdim=True))
    return (dx, (dy * xhat).sum(0), dy.sum(0)), (slack, (rows + 16) * U * (dy * xhat).abs().sum(0),
                                                 (rows + 16) * U * dy.abs().sum(0))


@pytest.mark.parametrize("dtype,wdtype", [(F16, F16), (F16, F32), (BF16, BF16), (BF16, F32), (F32, F32)])
@pytest.mark.parametrize("rows,cols", NORM_SIZES + [(1000, 64), (700, 1001), (5000, 130)])
def test_layer_norm_backward(rows, cols, dtype, wdtype):
    x, w, b = norm_inputs(rows, cols, dtype, wdtype, rows * 37 + cols)
    dy = rnd(9, rows, cols).to(dtype)
    _, mean, rstd = gr.layer_norm(x, w, b, 1e-3, stats=True)
    refs, slacks = norm_grad_ref(dy, x, w, mean, rstd)
    got = gr.layer_norm_backward(dy, x, w, mean, rstd)
    assert [g.dtype for g in got] == [dtype, wdtype, wdtype]
    for g, ref, slack in zip(got, refs, slacks):
        close(g, ref, slack)
    again = gr.layer_norm_backward(dy, x, w, mean, rstd)
    assert all(torch.equal(g, a) for g, a in zip(got, again))


def test_layer_norm_backward_shapes_and_strides():
    x, w, b = norm_inputs(70, 1001, BF16, F32, 8)
    dy = rnd(9, 70, 1001).to(BF16)
    _, mean, rstd = gr.layer_norm(x, w, b, stats=True)
    got = gr.layer_norm_backward(dy, x, w, mean, rstd)
    for a, bb in [(strided(dy, 3), strided(x, 9)), (shifted(dy), shifted(x))]:
        assert all(torch.equal(p, q) for p, q in zip(gr.layer_norm_backward(a, bb, w, mean, rstd), got))
    nd = gr.layer_norm_backward(dy.view(2, 35, 1001), x.view(2, 35, 1001), w, mean.view(2, 35), rstd.view(2, 35))
    assert nd[0].shape == (2, 35, 1001)
    assert all(torch.equal(p.view(q.shape), q) for p, q in zip(nd, got))
    # no rows: the gradients of weight and bias are empty sums
    dx, dw, db = gr.layer_norm_backward(dy[:0], x[:0], w, mean[:0], rstd[:0])
    assert dx.shape == (0, 1001) and not dw.any() and not db.any()


def test_layer_norm_backward_against_differences():
    # directional derivatives of the binary64 forward pass, step h: the central
    # difference is off by O(h^2) of the third derivative (1e-8 of the value at
    # h = 1e-4 and unit directions) and by rounding (2^-53 / h)
    rows, cols, h = 7, 65, 1e-4
    x, w, b = norm_inputs(rows, cols, F32, F32, 11)
    dy = rnd(12, rows, cols)
    _, mean, rstd = gr.layer_norm(x, w, b, stats=True)
    dx, dw, db = gr.layer_norm_backward(dy, x, w, mean, rstd)

    def loss(x, w, b):
        m = x.mean(1, keepdim=True)
        return (dy.to(F64) * ((x - m) * (((x - m) ** 2).mean(1, keepdim=True) + 1e-5) ** -0.5 * w + b)).sum()

    args = [a.to(F64) for a in (x, w, b)]
    for k, grad in enumerate((dx, dw, db)):
        for seed in range(3):
            v = rnd(20 + seed, *args[k].shape).to(F64)
            up, down = list(args), list(args)
            up[k], down[k] = args[k] + h * v, args[k] - h * v
            diff = (loss(*up) - loss(*down)) / (2 * h)
            want = (grad.to(F64) * v).sum()
            size = (grad.to(F64) * v).abs().sum()
            # fp32 gradients, each off by at most a few hundred fp32 steps of the largest term
            assert abs(diff - want) <= 1e-4 * size + 1e-6


# ------------------------------------------------------ gated projections
ACTS = ["silu", "gelu", "gelu_tanh", "relu"]
GATED_SIZES = [(1, 1, 1), (1, 64, 64), (2, 33, 100), (5, 7, 513), (16, 100, 250), (17, 130, 96), (33, 48, 257),
               (64, 128, 192), (65, 64, 33), (100, 260, 130), (130, 67, 1000), (257, 129, 64), (300, 200, 333)]


def act_ref(g, act):
    if act == "relu":
        return g.clamp(min=0), (g > 0).to(F64)
    if act == "silu":
        s = torch.sigmoid(g)
        return g * s, s * (1 + g * torch.sigmoid(-g))
    if act == "gelu":
        p = 0.5 * torch.erfc(-g / math.sqrt(2))
        return g * p, p + g * torch.exp(-g * g / 2) / math.sqrt(2 * math.pi)
    c = 2 * math.sqrt(2 / math.pi)
    z = c * (g + 0.044715 * g ** 3)
    s = torch.sigmoid(z)
    return g * s, s + g * s * torch.sigmoid(-z) * c * (1 + 0.134145 * g * g)


def gated_inputs(rows, hidden, cols, dtype, seed):
    return rnd(seed, rows, cols).to(dtype), (rnd(seed + 1, 2 * hidden, cols) * 2 * cols ** -0.5).to(dtype)


def gated_check(x, w, act, h, gu=None):
    hidden, cols = w.shape[0] // 2, w.shape[1]
    xd, wd = x.to(F64), w.to(F64)
    sums = xd @ wd.t()
    off = (cols + 1) * U * (xd.abs() @ wd.abs().t())
    g, u, og, ou = sums[:, :hidden], sums[:, hidden:], off[:, :hidden], off[:, hidden:]
    value, _ = act_ref(g, act)
    # slopes are below 1.2; a relative step of the argument moves the tails by up to its square
    slack = 1.2 * og * (u.abs() + ou) + value.abs() * ou + (16 + 4 * g * g) * U * (value * u).abs()
    close(h, value * u, slack)
    if gu is not None:
        assert gu.dtype == F32
        close(gu, sums, off)


@pytest.mark.parametrize("act", ACTS)
@pytest.mark.parametrize("dtype", [F16, BF16])
@pytest.mark.parametrize("rows,hidden,cols", GATED_SIZES)
def test_matmul_gated(rows, hidden, cols, dtype, act):
    x, w = gated_inputs(rows, hidden, cols, dtype, rows + hidden + cols)
    h, gu = gr.matmul_gated(x, w, act, save=True)
    gated_check(x, w, act, h, gu)
    assert torch.equal(gr.matmul_gated(x, w, act), h)


# sizes that take each kernel configuration
BIG_GATED = [(1, 5000, 1024), (64, 2050, 2048), (48, 515, 3000), (200, 1030, 640), (1000, 1100, 520),
             (2050, 4000, 264)]


@pytest.mark.parametrize("dtype", [F16, BF16])
@pytest.mark.parametrize("rows,hidden,cols", BIG_GATED)
def test_matmul_gated_large(rows, hidden, cols, dtype):
    x, w = gated_inputs(rows, hidden, cols, dtype, 3)
    h, gu = gr.matmul_gated(x, w, "silu", save=True)
    gated_check(x, w, "silu", h, gu)


def ints(seed, lo, hi, *shape):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(seed)
    return torch.randint(lo, hi + 1, shape, generator=gen, device="cuda")


@pytest.mark.parametrize("dtype", [F16, BF16])
@pytest.mark.parametrize("rows,hidden,cols", [(1, 300, 200), (30, 300, 200), (64, 1000, 72), (150, 300, 120),
                                              (600, 900, 64), (1500, 2100, 72)])
def test_gated_integers_are_exact(rows, hidden, cols, dtype):
    # few non-zero weights, so that every sum and product is an integer of at
    # most 8 bits: each result has exactly one right value
    x = ints(1, -1, 1, rows, cols)
    w = ints(2, -1, 1, 2 * hidden, cols) * (ints(3, 0, 31, 2 * hidden, cols) == 0)
    sums = x.to(F64) @ w.to(F64).t()
    g, u = sums[:, :hidden], sums[:, hidden:]
    keep = (g * u).abs().amax(0) <= 256                    # columns of h that fit in 8 bits
    h, gu = gr.matmul_gated(x.to(dtype), w.to(dtype), "relu", save=True)
    assert keep.any()
    assert torch.equal(gu.to(F64), sums)
    assert torch.equal(h.to(F64)[:, keep], (g.clamp(min=0) * u)[:, keep])
    dh = ints(4, -1, 1, rows, hidden)
    dg, du = dh * u * (g > 0), dh * g.clamp(min=0)
    d = torch.cat([dg, du], 1)
    dx, dw = gr.matmul_gated_backward(dh.to(dtype), gu, x.to(dtype), w.to(dtype), "relu")
    rx, rw = d @ w.to(F64), d.t() @ x.to(F64)
    assert torch.equal(dx.to(F64), rx.to(dtype).to(F64))
    assert torch.equal(dw.to(F64), rw.to(dtype).to(F64))


def gated_grad_check(dh, gu, x, w, act, dx, dw):
    hidden = w.shape[0] // 2
    rows = x.shape[0]
    gud, dhd, xd, wd = gu.to(F64), dh.to(F64), x.to(F64), w.to(F64)
    g, u = gud[:, :hidden], gud[:, hidden:]
    value, slope = act_ref(g, act)
    d = torch.cat([dhd * u * slope, dhd * value], 1)
    # fp32 evaluation of slope and value, then the rounding to 16 bits
    fn = torch.cat([(dhd * u).abs(), (dhd * g).abs()], 1) * (16 + 4 * torch.cat([g, g], 1) ** 2).clamp(max=256) * U
    off = half_step(x.dtype) * (d.abs() + fn) + fn + TINY[x.dtype]
    mag = d.abs() + off
    close(dx, d @ wd, off @ wd.abs() + (2 * hidden + 1) * U * (mag @ wd.abs()))
    close(dw, d.t() @ xd, off.t() @ xd.abs() + (rows + 1) * U * (mag.t() @ xd.abs()))


@pytest.mark.parametrize("act", ACTS)
@pytest.mark.parametrize("dtype", [F16, BF16])
@pytest.mark.parametrize("rows,hidden,cols", GATED_SIZES)
def test_matmul_gated_backward(rows, hidden, cols, dtype, act):
    x, w = gated_inputs(rows, hidden, cols, dtype, rows + hidden + cols)
    _, gu = gr.matmul_gated(x, w, act, save=True)
    dh = rnd(5, rows, hidden).to(dtype)
    dx, dw = gr.matmul_gated_backward(dh, gu, x, w, act)
    gated_grad_check(dh, gu, x, w, act, dx, dw)
    again = gr.matmul_gated_backward(dh, gu, x, w, act)
    assert torch.equal(again[0], dx) and torch.equal(again[1], dw)


@pytest.mark.parametrize("dtype", [F16, BF16])
@pytest.mark.parametrize("rows,hidden,cols", BIG_GATED)
def test_matmul_gated_backward_large(rows, hidden, cols, dtype):
    x, w = gated_inputs(rows, hidden, cols, dtype, 3)
    _, gu = gr.matmul_gated(x, w, "gelu_tanh", save=True)
    dh = rnd(5, rows, hidden).to(dtype)
    gated_grad_check(dh, gu, x, w, "gelu_tanh", *gr.matmul_gated_backward(dh, gu, x, w, "gelu_tanh"))


@pytest.mark.parametrize("act", ACTS)
def test_gated_backward_against_differences(act):
    # as for layer norm; the gradients' own error is the 16-bit rounding of dg,
    # du and the results: 2 half steps of fp16 of the sum of magnitudes
    rows, hidden, cols, h = 5, 24, 40, 1e-4
    x, w = gated_inputs(rows, hidden, cols, F16, 21)
    dh = rnd(22, rows, hidden).to(F16)
    _, gu = gr.matmul_gated(x, w, act, save=True)
    dx, dw = gr.matmul_gated_backward(dh, gu, x, w, act)
    xd, wd, dhd = x.to(F64), w.to(F64), dh.to(F64)
    if act == "relu":                                   # its kink stays outside the steps
        assert (xd @ wd[:hidden].t()).abs().min() > 20 * h

    def loss(x, w):
        s = x @ w.t()
        return (dhd * act_ref(s[:, :hidden], act)[0] * s[:, hidden:]).sum()

    d = dhd.abs() * (gu.to(F64).abs().amax() + 1) * 1.2
    for k, grad in enumerate((dx, dw)):
        size = d.sum() * (wd.abs().amax() if k == 0 else xd.abs().amax())
        for seed in range(3):
            v = rnd(30 + seed, *grad.shape).to(F64).sign() / grad.numel() ** 0.5
            args = [(xd + h * v, wd), (xd - h * v, wd)] if k == 0 else [(xd, wd + h * v), (xd, wd - h * v)]
            diff = (loss(*args[0]) - loss(*args[1])) / (2 * h)
            want = (grad.to(F64) * v).sum()
            assert abs(diff - want) <= 2 * half_step(F16) * (grad.to(F64).abs() * v.abs()).sum() + 1e-3 * size * v.abs().max() + 1e-6


@pytest.mark.parametrize("rows", [3, 40, 150])
def test_gated_shapes_strides_and_alignment(rows):
    x, w = gated_inputs(rows, 77, 131, BF16, 31)
    h, gu = gr.matmul_gated(x, w, "gelu", save=True)
    dh = rnd(32, rows, 77).to(BF16)
    grads = gr.matmul_gated_backward(dh, gu, x, w, "gelu")
    for xs, ws, ds in [(strided(x, 3), strided(w, 5), strided(dh, 1)), (shifted(x), shifted(w), shifted(dh))]:
        h2, gu2 = gr.matmul_gated(xs, ws, "gelu", save=True)
        assert torch.equal(h2, h) and torch.equal(gu2, gu)
        assert all(torch.equal(p, q) for p, q in zip(gr.matmul_gated_backward(ds, gu, xs, ws, "gelu"), grads))
    one = gr.matmul_gated(x[:1].view(1, 1, 131), w, "gelu")
    assert one.shape == (1, 1, 77)


def test_gated_empty_sizes():
    x, w = gated_inputs(4, 6, 8, F16, 1)
    assert gr.matmul_gated(x[:0], w).shape == (0, 6)
    assert gr.matmul_gated(x, w[:0]).shape == (4, 0)
    h, gu = gr.matmul_gated(x[:, :0], w[:, :0], save=True)          # empty sums
    assert h.shape == (4, 6) and not h.any() and not gu.any()
    dh = rnd(2, 4, 6).to(F16)
    dx, dw = gr.matmul_gated_backward(dh[:0], gu[:0], x[:0], w)
    assert dx.shape == (0, 8) and dw.shape == w.shape and not dw.any()
    dx, dw = gr.matmul_gated_backward(dh[:, :0], gu[:, :0], x, w[:0])
    assert dx.shape == x.shape and not dx.any() and dw.shape == (0, 8)


@pytest.mark.parametrize("rows,hidden,cols", [(2, 40, 70), (40, 40, 70), (70, 40, 70), (400, 900, 70)])
def test_gated_non_finite_values_stay_in_their_rows(rows, hidden, cols):
    x, w = gated_inputs(rows, hidden, cols, F16, 41)
    clean, gu0 = gr.matmul_gated(x, w, save=True)
    bad = x.clone()
    bad[1, cols - 1] = float("nan")
    h, gu = gr.matmul_gated(bad, w, save=True)
    others = [i for i in range(rows) if i != 1]
    assert torch.isnan(h[1]).all() and torch.isnan(gu[1]).all()
    assert torch.equal(h[others], clean[others]) and torch.equal(gu[others], gu0[others])
    wbad = w.clone()
    wbad[hidden + 3, 0] = float("inf")                    # an up row: column 3 of h alone
    h = gr.matmul_gated(x, wbad)
    cols_left = [j for j in range(hidden) if j != 3]
    assert not torch.isfinite(h[:, 3]).any() and torch.equal(h[:, cols_left], clean[:, cols_left])


def test_gated_activations_over_their_range():
    # sums from -40 to 40 and the far ends, against an up sum of 1
    for dtype in (F16, BF16):
        g = torch.cat([torch.linspace(-40, 40, 1601), torch.tensor([-60000.0, -1000.0, 1000.0, 60000.0])]).to(dtype).cuda()
        x = torch.stack([g, torch.ones_like(g)], 1)
        w = torch.tensor([[1.0, 0.0], [0.0, 1.0]], device="cuda", dtype=dtype)
        for act in ACTS:
            h, gu = gr.matmul_gated(x, w, act, save=True)
            value, slope = act_ref(g.to(F64), act)
            close(h[:, 0], value, (16 + 4 * g.to(F64) ** 2).clamp(max=2000) * U * value.abs())
            dx, _ = gr.matmul_gated_backward(torch.ones_like(h), gu, x, w, act)
            assert torch.isfinite(dx).all()
            close(dx[:, 0], slope, half_step(dtype) * slope.abs() + 2.0 ** -16 + TINY[dtype])


# -------------------------------------------------------- 8-bit integers
@pytest.mark.parametrize("dtype", [F16, BF16, F32])
@pytest.mark.parametrize("rows,cols", [(1, 1), (3, 5), (4, 64), (77, 100), (5, 513), (130, 1024), (6, 5003), (3, 8192),
                                       (2, 20001)])
def test_quantize_rows(rows, cols, dtype):
    x = (rnd(rows + cols, rows, cols) * torch.exp(3 * rnd(1, rows, 1))).to(dtype)
    q, s = gr.quantize_rows(x)
    assert q.dtype == torch.int8 and s.dtype == F32 and q.shape == x.shape and s.shape == (rows,)
    top = x.to(F64).abs().amax(1)
    ref = torch.round(127 * x.to(F64) / top[:, None])
    if dtype == F32:                                     # one fp32 step may cross a border
        assert ((q.to(F64) - ref).abs() <= 1).all() and (q.to(F64) != ref).to(F64).mean() < 1e-3
    else:
        assert torch.equal(q.to(F64), ref)
    close(s, top / 127, U * top / 127)


@pytest.mark.parametrize("dtype", [F16, BF16])
def test_quantize_rows_ties_and_extremes(dtype):
    # a largest value of 127 (or its powers of two): quotients are the values themselves
    rows = []
    for scale in (1.0, 2.0 ** -10, 2.0 ** 8 if dtype == F16 else 2.0 ** 100):
        halves = torch.arange(-253, 254, 2, dtype=F64) / 2          # every tie, exact in bf16
        rows.append(torch.cat([torch.tensor([127.0, -127.0, 0.0, -0.0]), halves]) * scale)
    x = torch.stack(rows).to(dtype)
    assert torch.equal(x.to(F64), torch.stack(rows))
    q, s = gr.quantize_rows(x.cuda())
    ref = torch.round(127 * x.to(F64) / x.to(F64).abs().amax(1, keepdim=True))
    assert torch.equal(q.cpu().to(F64), ref)
    # the type's largest and smallest values; a zero row; rows that are not finite
    info = torch.finfo(dtype)
    y = torch.zeros(6, 40, dtype=dtype)
    y[0, 3], y[0, 5] = info.max, -info.max / 2
    y[1, 39] = -info.tiny
    y[2, 1], y[2, 2] = info.tiny / 4, info.tiny / 8               # below the normal range
    y[4, 0], y[4, 1] = float("inf"), 1.0
    y[5, 7], y[5, 8] = float("nan"), 1.0
    q, s = gr.quantize_rows(y.cuda())
    q, s = q.cpu(), s.cpu()
    assert q[0, 3] == 127 and q[0, 5] == -64 and q[1, 39] == -127 and q[2, 1] == 127 and q[2, 2] == 64
    assert not q[3:].any() and s[3] == 0 and torch.isnan(s[4:]).all() and torch.isfinite(s[:4]).all()


I8_SIZES = [(1, 1, 1), (1, 100, 300), (3, 65, 64), (16, 33, 1000), (17, 200, 128), (40, 130, 65), (64, 512, 777),
            (65, 64, 130), (77, 301, 503), (130, 260, 512), (300, 190, 257)]


def i8_inputs(rows, n, k, seed):
    return (ints(seed, -128, 127, rows, k).to(torch.int8), torch.exp(rnd(seed + 1, rows)) * 1e-3,
            ints(seed + 2, -128, 127, n, k).to(torch.int8), torch.exp(rnd(seed + 3, n)) * 1e-3)


def i8_check(x, sx, w, sw, y):
    # the sum rounds to fp32 once, the two products once each
    ref = (x.to(F64) @ w.to(F64).t()) * sx.to(F64)[:, None] * sw.to(F64)
    close(y, ref, 4 * U * ref.abs())


@pytest.mark.parametrize("out", [F16, BF16, F32])
@pytest.mark.parametrize("rows,n,k", I8_SIZES + [(1, 5000, 4096), (64, 3000, 2048), (200, 1500, 1300),
                                                 (900, 2000, 520), (2000, 2100, 264)])
def test_matmul_i8(rows, n, k, out):
    x, sx, w, sw = i8_inputs(rows, n, k, rows + n + k)
    y = gr.matmul_i8(x, sx, w, sw, out)
    assert y.dtype == out
    i8_check(x, sx, w, sw, y)


@pytest.mark.parametrize("rows,n", [(1, 3), (20, 40), (70, 40), (300, 300)])
def test_matmul_i8_largest_sums_do_not_wrap(rows, n):
    k = 131071
    x = torch.full((rows, k), -128, dtype=torch.int8, device="cuda")
    w = torch.full((n, k), -128, dtype=torch.int8, device="cuda")
    one = torch.ones(max(rows, n), device="cuda")
    y = gr.matmul_i8(x, one[:rows], w, one[:n], F32)
    assert (y == float(torch.tensor(128.0 * 128 * k, dtype=F32))).all()
    assert (gr.matmul_i8(x, one[:rows], -1 - w, one[:n], F32) == float(torch.tensor(-128.0 * 127 * k, dtype=F32))).all()


@pytest.mark.parametrize("rows", [2, 30, 130])
def test_matmul_i8_shapes_strides_and_alignment(rows):
    x, sx, w, sw = i8_inputs(rows, 90, 111, 51)
    y = gr.matmul_i8(x, sx, w, sw, F16)
    assert torch.equal(gr.matmul_i8(strided(x, 3), sx, strided(w, 7), sw, F16), y)
    assert torch.equal(gr.matmul_i8(shifted(x), shifted(sx), shifted(w), shifted(sw), F16), y)
    assert torch.equal(gr.matmul_i8(x.view(2, rows // 2, 111), sx.view(2, rows // 2), w, sw, F16).view(rows, 90), y)
    assert gr.matmul_i8(x[:0], sx[:0], w, sw).shape == (0, 90)
    zero = gr.matmul_i8(x[:, :0], sx, w[:, :0], sw, F32)
    assert zero.shape == (rows, 90) and not zero.any()
    assert gr.matmul_i8(x, sx, w, sw).dtype == BF16


def test_quantised_product_of_a_bad_row_is_nan():
    x = rnd(1, 6, 200).to(F16)
    x[2, 5] = float("inf")
    _, _, w, sw = i8_inputs(6, 50, 200, 61)
    q, s = gr.quantize_rows(x)
    y = gr.matmul_i8(q, s, w, sw, F16)
    assert torch.isnan(y[2]).all() and torch.isfinite(y[[0, 1, 3, 4, 5]]).all()


# ------------------------------------------- far rows, streams and graphs
def test_rows_past_32_bit_offsets():
    # rows 2^30 elements apart: the third starts past 2^31 elements, 2^32 bytes
    far = 2 ** 30
    buf = torch.zeros(2 * far + 4096, dtype=F16, device="cuda")
    x = buf.as_strided((3, 200), (far, 1))
    x.copy_(rnd(71, 3, 200))
    near = x.contiguous()
    w, b = rnd(72, 200).to(F16), rnd(73, 200).to(F16)
    y, mean, rstd = gr.layer_norm(near, w, b, stats=True)
    assert torch.equal(gr.layer_norm(x, w, b), y)
    assert all(torch.equal(p, q) for p, q in zip(gr.layer_norm_backward(x, x, w, mean, rstd),
                                                 gr.layer_norm_backward(near, near, w, mean, rstd)))
    wg = rnd(74, 80, 200).to(F16)
    h, gu = gr.matmul_gated(near, wg, save=True)
    assert torch.equal(gr.matmul_gated(x, wg), h)
    got = gr.matmul_gated_backward(near[:, :40].contiguous(), gu, x, wg)
    want = gr.matmul_gated_backward(near[:, :40].contiguous(), gu, near, wg)
    assert all(torch.equal(p, q) for p, q in zip(got, want))
    q, s = gr.quantize_rows(near)
    assert all(torch.equal(p, r) for p, r in zip(gr.quantize_rows(x), (q, s)))
    # a weight whose up rows lie past 2^32 bytes from its gate rows
    ww = buf.as_strided((2, 200), (far, 1))
    assert torch.equal(gr.matmul_gated(near, ww), gr.matmul_gated(near, ww.contiguous()))
    xi = buf.view(torch.int8).as_strided((3, 200), (2 ** 31 - 1, 1))
    xi.copy_(ints(75, -128, 127, 3, 200).to(torch.int8))
    _, _, wi, sw = i8_inputs(3, 30, 200, 76)
    assert torch.equal(gr.matmul_i8(xi, s, wi, sw), gr.matmul_i8(xi.contiguous(), s, wi, sw))


def half_layer(x, w, b, wg, dh, wi, sw, stream=None):
    """Everything once, as a training step and a serving step use it."""
    y, mean, rstd = gr.layer_norm(x, w, b, stats=True, stream=stream)
    h, gu = gr.matmul_gated(y, wg, "silu", save=True, stream=stream)
    q, s = gr.quantize_rows(h, stream=stream)
    out = gr.matmul_i8(q, s, wi, sw, x.dtype, stream=stream)
    dy, dwg = gr.matmul_gated_backward(dh, gu, y, wg, "silu", stream=stream)
    dx, dw, db = gr.layer_norm_backward(dy, x, w, mean, rstd, stream=stream)
    return y, h, q, s, out, dwg, dx, dw, db


def half_layer_inputs(rows, cols, hidden, seed):
    x, w, b = norm_inputs(rows, cols, BF16, F32, seed)
    _, wg = gated_inputs(rows, hidden, cols, BF16, seed + 4)
    _, _, wi, sw = i8_inputs(rows, cols, hidden, seed + 6)
    return x, w, b, wg, rnd(seed + 9, rows, hidden).to(BF16), wi, sw


@pytest.mark.parametrize("rows", [1, 40, 300])
def test_on_another_stream(rows):
    args = half_layer_inputs(rows, 520, 264, 81)
    want = half_layer(*args)
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    for given in (s, s.cuda_stream):
        got = half_layer(*args, stream=given)
        s.synchronize()
        assert all(torch.equal(p, q) for p, q in zip(got, want))
    with torch.cuda.stream(s):
        got = half_layer(*args)
    s.synchronize()
    assert all(torch.equal(p, q) for p, q in zip(got, want))


@pytest.mark.parametrize("rows", [1, 40, 300])
def test_captured_into_a_graph(rows):
    args = half_layer_inputs(rows, 520, 264, 91)
    other = half_layer_inputs(rows, 520, 264, 191)
    want, want2 = half_layer(*args), half_layer(*other)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        half_layer(*args)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=s):
        out = half_layer(*args)
    kept = [a.clone() for a in args]
    for k in range(4):                     # the program's own work in between, and other inputs every second time
        for a, n in zip(args, other if k % 2 else kept):
            a.copy_(n)
        for o in out:
            o.zero_()
        half_layer(*other)
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(p, q) for p, q in zip(out, want2 if k % 2 else want)), k
