"""The product with bias, activation and residual, and its gradients, on the GPU against
their definitions in binary64.

Tolerances are bounds on the kernels' arithmetic: one rounding of the result (half a
step of its type), fp32 sums of n terms (n 2^-24 of the sum of magnitudes, whatever the
order), a few fp32 steps for the activations, and for the gradients the rounding of dz
to 16 bits.
"""
import pytest
import torch

import dense_tiled_gemm_relu_amd as gr
from tests.block_helpers import (ACTS, BF16, F16, F32, F64, TINY, U, act_ref, close, half_step, ints, rnd, shifted, strided)

pytestmark = pytest.mark.gpu

SIZES = [(1, 1, 1), (1, 64, 64), (2, 33, 100), (5, 7, 513), (3, 3, 40), (16, 100, 250), (17, 130, 96), (33, 48, 257),
         (64, 128, 192), (65, 64, 33), (100, 260, 130), (130, 67, 1000), (257, 129, 64), (300, 200, 333)]
# sizes that take each kernel configuration
BIG = [(1, 5000, 1024), (64, 2050, 2048), (48, 515, 3000), (200, 2060, 640), (1000, 2200, 520), (2050, 4100, 264),
       (2048, 8192, 264), (2003, 2006, 2003), (77, 3001, 2500), (100, 3000, 3000),
       (50, 8100, 333), (128, 4096, 520)]


def inputs(rows, n, k, dtype, seed, bias_dtype=None):
    x, w = rnd(seed, rows, k).to(dtype), (rnd(seed + 1, n, k) * 2 * max(k, 1) ** -0.5).to(dtype)
    return x, w, (0.5 * rnd(seed + 2, n)).to(bias_dtype or dtype), rnd(seed + 3, rows, n).to(dtype)


def check(y, x, w, bias, act, residual, z=None):
    xd, wd = x.to(F64), w.to(F64)
    b = torch.zeros(w.shape[0], device=x.device, dtype=F64) if bias is None else bias.to(F64)
    r = torch.zeros_like(y, dtype=F64) if residual is None else residual.to(F64)
    sums = xd @ wd.t() + b
    off = (x.shape[1] + 2) * U * (xd.abs() @ wd.abs().t() + b.abs())
    value, _ = act_ref(sums, act)
    # slopes are below 1.2; a relative step of the argument moves the tails by up to its
    # square; one fp32 step of the sum with the residual
    own = 0.0 if act == "none" else (16 + 4 * sums * sums).clamp(max=1e4) * U * value.abs()
    slack = 1.2 * off + own + U * (value.abs() + r.abs())
    close(y, value + r, slack)
    if z is not None:
        assert z.dtype == F32
        close(z, sums, off)


@pytest.mark.parametrize("act", ACTS)
@pytest.mark.parametrize("dtype,bias_dtype", [(F16, F16), (F16, F32), (BF16, BF16), (BF16, F32)])
@pytest.mark.parametrize("rows,n,k", SIZES)
def test_matmul_act(rows, n, k, dtype, bias_dtype, act):
    x, w, b, r = inputs(rows, n, k, dtype, rows + n + k, bias_dtype)
    y, z = gr.matmul_act(x, w, b, act, r, save=True)
    assert y.dtype == dtype and (z is None) == (act == "none")
    check(y, x, w, b, act, r, z)
    assert torch.equal(gr.matmul_act(x, w, b, act, r), y)
    check(gr.matmul_act(x, w, None, act, r), x, w, None, act, r)
    check(gr.matmul_act(x, w, b, act), x, w, b, act, None)
    check(gr.matmul_act(x, w, act=act), x, w, None, act, None)


@pytest.mark.parametrize("dtype", [F16, BF16])
@pytest.mark.parametrize("rows,n,k", BIG)
def test_matmul_act_large(rows, n, k, dtype):
    x, w, b, r = inputs(rows, n, k, dtype, 3)
    y, z = gr.matmul_act(x, w, b, "silu", r, save=True)
    check(y, x, w, b, "silu", r, z)
    check(gr.matmul_act(x, w, b, "none", r), x, w, b, "none", r)


def test_every_configuration_is_taken():
    lib, names, grads = gr.library(), set(), set()
    for rows, n, k in SIZES + BIG + EXACT:
        names.update(lib.gemm_relu_act_plan(rows, n, k, gr.BF16).decode().split("+"))
        grads.update(lib.gemm_relu_act_backward_plan(rows, n, k, gr.BF16).decode().split(","))
    tiles = {"d256x256x32_s4_i16w8", "d128x128x64_s4_i16w8", "d64x64x64_s4"}
    assert names >= tiles | {"d128x128x64_s2w8", "k16x16x64_s4", "k32x32x64_s4", "k32x48x64_s3",
                     "k64x32x64_s3"}, names
    assert grads >= tiles | {"g64x64x64"}, grads


def test_rows_far_apart():
    # past what the tiles' 32-bit offsets reach: the register-staged tile for a short K,
    # the small ones for a longer
    for k in (5, 40):
        x, w, b, r = inputs(5, 70, k, BF16, 61)
        far = torch.zeros(5, (1 << 22) + 8, dtype=BF16, device="cuda")
        far[:, :k] = x
        y, z = gr.matmul_act(far[:, :k], w, b, "silu", r, save=True)
        check(y, x, w, b, "silu", r, z)
        dy = rnd(62, 5, 70).to(BF16)
        got = gr.matmul_act_backward(dy, z, far[:, :k], w, "silu", b)
        grad_check(dy, z, x, w, "silu", b, *got)
        far[:, :70] = dy
        for act in ("none", "silu"):
            want = gr.matmul_act_backward(dy, z, x, w, act, b)
            got = gr.matmul_act_backward(far[:, :70], z, x, w, act, b)
            assert all(torch.equal(p, q) for p, q in zip(got, want))


EXACT = [(1, 300, 200), (30, 300, 200), (64, 1000, 72), (150, 600, 120), (600, 1800, 64), (1500, 4200, 72)]


@pytest.mark.parametrize("dtype", [F16, BF16])
@pytest.mark.parametrize("rows,n,k", EXACT)
def test_integers_are_exact(rows, n, k, dtype):
    # every sum is an integer of at most 8 bits: each result has exactly one right value
    x, w = ints(1, -1, 1, rows, k), ints(2, -1, 1, n, k) * (ints(3, 0, 15, n, k) == 0)
    b, r = ints(4, -8, 8, n), ints(5, -64, 64, rows, n)
    z = x.to(F64) @ w.to(F64).t() + b
    assert z.abs().max() <= 128
    y, saved = gr.matmul_act(x.to(dtype), w.to(dtype), b.to(dtype), "relu", r.to(dtype), save=True)
    assert torch.equal(saved.to(F64), z) and torch.equal(y.to(F64), z.clamp(min=0) + r)
    assert torch.equal(gr.matmul_act(x.to(dtype), w.to(dtype), b.float(), "none", r.to(dtype)).to(F64), z + r)
    dy = ints(6, -1, 1, rows, n)
    for act, d in (("relu", dy.to(F64) * (z > 0)), ("none", dy.to(F64))):
        dx, dw, db = gr.matmul_act_backward(dy.to(dtype), saved, x.to(dtype), w.to(dtype), act, b.float())
        assert torch.equal(dx.to(F64), (d @ w.to(F64)).to(dtype).to(F64))
        assert torch.equal(dw.to(F64), (d.t() @ x.to(F64)).to(dtype).to(F64))
        assert torch.equal(db.to(F64), d.sum(0))


def grad_check(dy, z, x, w, act, bias, dx, dw, db):
    n, rows = w.shape[0], x.shape[0]
    zd, dyd, xd, wd = z.to(F64), dy.to(F64), x.to(F64), w.to(F64)
    _, slope = act_ref(zd, act)
    d = dyd * slope
    # fp32 evaluation of the slope, then the rounding to 16 bits (of half of dz in float16)
    fn = 0.0 * d if act == "none" else dyd.abs() * (16 + 4 * zd ** 2).clamp(max=256) * U
    off = (half_step(x.dtype) * (d.abs() + fn) + 2 * TINY[x.dtype] + fn) if act != "none" else fn
    mag = d.abs() + off
    close(dx, d @ wd, off @ wd.abs() + (n + 1) * U * (mag @ wd.abs()))
    close(dw, d.t() @ xd, off.t() @ xd.abs() + (rows + 1) * U * (mag.t() @ xd.abs()))
    if bias is None:
        assert db is None
    else:
        assert db.dtype == bias.dtype
        close(db, d.sum(0), fn.sum(0) + (rows + 1) * U * mag.sum(0))


@pytest.mark.parametrize("act", ACTS)
@pytest.mark.parametrize("dtype,bias_dtype", [(F16, F16), (F16, F32), (BF16, BF16), (BF16, F32)])
@pytest.mark.parametrize("rows,n,k", SIZES)
def test_matmul_act_backward(rows, n, k, dtype, bias_dtype, act):
    x, w, b, _ = inputs(rows, n, k, dtype, rows + n + k, bias_dtype)
    z = x.float() @ w.float().t() + b.float()
    dy = rnd(5, rows, n).to(dtype)
    saved = None if act == "none" else z
    dx, dw, db = gr.matmul_act_backward(dy, saved, x, w, act, b)
    grad_check(dy, z, x, w, act, b, dx, dw, db)
    again = gr.matmul_act_backward(dy, saved, x, w, act, b)
    assert all(torch.equal(p, q) for p, q in zip(again, (dx, dw, db)))
    without = gr.matmul_act_backward(dy, saved, x, w, act)
    assert torch.equal(without[0], dx) and torch.equal(without[1], dw) and without[2] is None


@pytest.mark.parametrize("act", ["none", "gelu"])
@pytest.mark.parametrize("dtype", [F16, BF16])
@pytest.mark.parametrize("rows,n,k", BIG)
def test_matmul_act_backward_large(rows, n, k, dtype, act):
    x, w, b, _ = inputs(rows, n, k, dtype, 3, F32)
    _, z = gr.matmul_act(x, w, b, "gelu", save=True)
    dy = rnd(5, rows, n).to(dtype)
    grad_check(dy, z, x, w, act, b, *gr.matmul_act_backward(dy, z, x, w, act, b))


@pytest.mark.parametrize("act", ACTS)
def test_backward_against_differences(act):
    # a central difference of the forward formula in binary64: its own error is below
    # h^2 times third derivatives, 1e-6 of the sizes here; the gradients' is the 16-bit
    # rounding of dz and of the results, two half steps of fp16 of the magnitudes
    rows, n, k, h = 5, 24, 40, 1e-4
    x, w, b, r = inputs(rows, n, k, F16, 21)
    dy = rnd(22, rows, n).to(F16)
    _, z = gr.matmul_act(x, w, b, act, r, save=True)
    grads = gr.matmul_act_backward(dy, z, x, w, act, b)
    args, dyd = [t.to(F64) for t in (x, w, b)], dy.to(F64)
    if act == "relu":                                   # its kink stays outside the steps
        assert z.abs().min() > 20 * h

    def loss(x, w, b):
        return (dyd * act_ref(x @ w.t() + b, act)[0]).sum()

    mag = 1.2 * dyd.abs()
    sizes = (mag @ args[1].abs(), mag.t() @ args[0].abs(), mag.sum(0))
    for j, grad in enumerate(grads):
        for seed in range(3):
            v = rnd(30 + seed, *grad.shape).to(F64).sign()
            up, down = list(args), list(args)
            step = h / max(1.0, float(grad.numel()) ** 0.5)
            up[j], down[j] = args[j] + step * v, args[j] - step * v
            diff = (loss(*up) - loss(*down)) / (2 * step)
            want = (grad.to(F64) * v).sum()
            assert abs(diff - want) <= 2.1 * half_step(F16) * sizes[j].sum() + 1e-5


@pytest.mark.parametrize("rows", [3, 40, 150])
@pytest.mark.parametrize("n", [77, 128])
def test_strides_and_alignment(rows, n):
    x, w, b, r = inputs(rows, n, 131, BF16, 31)
    y, z = gr.matmul_act(x, w, b, "gelu", r, save=True)
    dy = rnd(32, rows, n).to(BF16)
    for act in ("gelu", "none"):
        grads = gr.matmul_act_backward(dy, z, x, w, act, b)
        for xs, ws, ds in [(strided(x, 3), strided(w, 5), strided(dy, 1)), (shifted(x), shifted(w), shifted(dy)),
                           (x, w, strided(dy, 64))]:
            assert all(torch.equal(p, q) for p, q in zip(gr.matmul_act_backward(ds, z, xs, ws, act, b), grads))
    for xs, ws, rs, bs in [(strided(x, 3), strided(w, 5), strided(r, 1), shifted(b)),
                           (shifted(x), shifted(w), shifted(r), b)]:
        y2, z2 = gr.matmul_act(xs, ws, bs, "gelu", rs, save=True)
        assert torch.equal(y2, y) and torch.equal(z2, z)
    one = gr.matmul_act(x[:1].view(1, 1, 131), w, b, "gelu", r[:1].view(1, 1, n))
    assert one.shape == (1, 1, n) and torch.equal(one.view(1, n), gr.matmul_act(x[:1], w, b, "gelu", r[:1]))


def test_empty_sizes():
    x, w, b, r = inputs(4, 6, 8, F16, 1)
    assert gr.matmul_act(x[:0], w, b, "silu", r[:0]).shape == (0, 6)
    assert gr.matmul_act(x, w[:0]).shape == (4, 0)
    y, z = gr.matmul_act(x[:, :0], w[:, :0], b, "relu", r, save=True)          # empty sums
    assert torch.equal(z, b.float().expand(4, 6))
    assert torch.equal(y, (b.float().clamp(min=0) + r.float()).to(F16))
    dy = rnd(2, 4, 6).to(F16)
    dx, dw, db = gr.matmul_act_backward(dy[:0], z[:0], x[:0], w, "relu", b)
    assert dx.shape == (0, 8) and dw.shape == w.shape and not dw.any() and not db.any()
    dx, dw, db = gr.matmul_act_backward(dy[:, :0], z[:, :0].contiguous(), x, w[:0], "relu", b[:0])
    assert dx.shape == x.shape and not dx.any() and dw.shape == (0, 8) and db.shape == (0,)
    dx, dw, db = gr.matmul_act_backward(dy, None, x[:, :0], w[:, :0], "none", b)
    assert dx.shape == (4, 0) and dw.shape == (6, 0)
    close(db, dy.to(F64).sum(0), 5 * U * dy.to(F64).abs().sum(0))


@pytest.mark.parametrize("rows,n,k", [(2, 40, 70), (40, 40, 70), (70, 40, 70), (400, 900, 70), (1500, 4200, 72)])
def test_non_finite_values_stay_in_their_rows(rows, n, k):
    x, w, b, r = inputs(rows, n, k, F16, 41)
    clean, z0 = gr.matmul_act(x, w, b, "silu", r, save=True)
    bad = x.clone()
    bad[1, k - 1] = float("nan")
    y, z = gr.matmul_act(bad, w, b, "silu", r, save=True)
    others = [i for i in range(rows) if i != 1]
    assert torch.isnan(y[1]).all() and torch.isnan(z[1]).all()
    assert torch.equal(y[others], clean[others]) and torch.equal(z[others], z0[others])
    rb, bb = r.clone(), b.clone()
    rb[1, 3], bb[5] = float("inf"), float("nan")
    y = gr.matmul_act(x, w, bb, "none", rb)
    good = gr.matmul_act(x, w, b, "none", r)
    assert y[1, 3] == float("inf") and torch.isnan(y[:, 5]).all()
    good[1, 3] = y[1, 3]
    keep = [j for j in range(n) if j != 5]
    assert torch.equal(y[:, keep], good[:, keep])


@pytest.mark.parametrize("act", ["none", "silu"])
@pytest.mark.parametrize("rows,n,k", [(3, 64, 70), (70, 72, 40), (40, 41, 33), (300, 192, 900), (1500, 1600, 72), (2048, 2048, 512)])
def test_non_finite_gradients_stay_in_their_rows(rows, n, k, act):
    # a row of dx takes its row of dy, a row of dweight its column; nothing of the next row, and
    # nothing between rows that are further apart than they are long
    x, w, b, _ = inputs(rows, n, k, F16, 61)
    z = None if act == "none" else x.float() @ w.float().t()
    dy = rnd(62, rows, n).to(F16)
    clean = gr.matmul_act_backward(dy, z, x, w, act, b)
    for pad in (8, 3):
        for got, want in zip(gr.matmul_act_backward(strided(dy, pad), z, x, w, act, b), clean):
            assert torch.equal(got, want)
    bad = dy.clone()
    bad[1, 0], bad[1, n - 1] = float("inf"), float("nan")
    dx, dw, db = gr.matmul_act_backward(bad, z, x, w, act, b)
    assert torch.isnan(dx[1]).all() and torch.isnan(dw[n - 1]).all() and torch.isnan(db[n - 1]) and not torch.isfinite(dw[0]).any()
    others, inner = [i for i in range(rows) if i != 1], slice(1, n - 1)
    assert torch.equal(dx[others], clean[0][others])
    assert torch.equal(dw[inner], clean[1][inner]) and torch.equal(db[inner], clean[2][inner])


@pytest.mark.parametrize("act", ["silu", "gelu", "gelu_tanh"])
def test_largest_float16_gradients_stay_finite(act):
    # slopes pass 1 (at most 1.13), so dz can pass float16's largest value; dx and dw here do not
    rows, n, k = 70, 40, 33
    x, w, b, _ = inputs(rows, n, k, F16, 51)
    z = torch.full((rows, n), 1.8 if act != "silu" else 2.4, device="cuda")
    dy = (65000 * rnd(52, rows, n).sign()).to(F16)
    w, x = w * 2.0 ** -8, x * 2.0 ** -8
    assert (dy.to(F64) * act_ref(z.to(F64), act)[1]).abs().max() > 65520
    grad_check(dy, z, x, w, act, None, *gr.matmul_act_backward(dy, z, x, w, act))


@pytest.mark.parametrize("act", ACTS)
@pytest.mark.parametrize("dtype", [F16, BF16])
def test_activations_over_their_range(dtype, act):
    # sums from -40 to 40 and the far ends, and their slopes (dy = 1)
    g = torch.cat([torch.linspace(-40, 40, 1601), torch.tensor([-60000.0, -1000.0, 1000.0, 60000.0])]).to(dtype).cuda()[:, None]
    w = torch.ones(1, 1, device="cuda", dtype=dtype)
    y, z = gr.matmul_act(g, w, None, act, save=True)
    check(y, g, w, None, act, None, z)
    z = g.float()
    grad_check(torch.ones_like(g), z, g, w, act, None, *gr.matmul_act_backward(torch.ones_like(g), z, g, w, act))
