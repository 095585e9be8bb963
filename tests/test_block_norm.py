"""The residual sum with norms before and after, and its gradients, on the GPU against
their definitions in binary64.

Tolerances follow the kernels' fp32 arithmetic: a sum of n terms, added a thread's share
at a time and then across threads, is off by at most (n / 64 + 16) steps of 2^-24 of the
sum of magnitudes; the results carry one rounding to their type.
"""
import itertools

import pytest
import torch

import dense_tiled_gemm_relu_amd as gr
from tests.block_helpers import BF16, F16, F32, F64, U, close, half_step, rnd, shifted, strided

pytestmark = pytest.mark.gpu

TYPES = [(F16, F16), (F16, F32), (BF16, BF16), (BF16, F32), (F32, F32)]
SIZES = [(1, 1), (3, 2), (2, 7), (5, 64), (4, 100), (67, 257), (130, 512), (9, 1000), (33, 2048), (6, 3001), (129, 4096),
         (3, 5003), (2, 8191), (4, 8192), (3, 16384), (2, 20001), (2, 40000)]
# (norm, bias, post, gate, scale)
FORMS = [("rms", False, False, None, 1.0), ("rms", False, True, "row", 1.0), ("layer", True, True, "matrix", 0.5),
         ("layer", True, False, "row", -1.5), ("rms", True, True, None, 0.7), ("layer", False, False, "matrix", 1.0)]


class Case:
    """Inputs of one call, and the definition of what it returns in binary64 with bounds."""

    def __init__(self, rows, cols, dtype, wdtype, form, seed=0, weighted=True, eps=1e-5):
        self.norm, bias, post, gate, self.scale = form
        self.eps = eps
        spread = 1 + 7 * (rnd(seed + 1, cols).abs() > 2)
        self.x = (rnd(seed, rows, cols) * spread + 0.5).to(dtype)
        self.r = (rnd(seed + 2, rows, cols) * spread - 0.25).to(dtype)
        self.w = (1 + 0.3 * rnd(seed + 3, cols)).to(wdtype) if weighted else None
        self.b = (0.2 * rnd(seed + 4, cols)).to(wdtype) if bias and weighted else None
        self.pw = (0.6 + 0.3 * rnd(seed + 5, cols)).to(wdtype) if post else None
        self.gate = None if gate is None else (0.3 * rnd(seed + 6, cols)).to(wdtype) if gate == "row" else \
            torch.sigmoid(rnd(seed + 6, rows, cols)).to(dtype)
        self.dy = rnd(seed + 7, rows, cols).to(dtype) if weighted else None
        self.ds = rnd(seed + 8, rows, cols).to(dtype)

    def options(self):
        return {"gate": self.gate, "scale": self.scale, "post_weight": self.pw, "norm": self.norm}

    def forward(self, stats=True):
        return gr.add_norm(self.x, self.r, self.w, self.b, eps=self.eps, stats=stats, **self.options())

    def backward(self, stats, dy=True, ds=True):
        return gr.add_norm_backward(self.dy if dy else None, self.ds if ds else None, self.x, self.r, stats, self.w, self.b,
                                    **self.options())

    # A value with a bound of its error: pairs (v, e) of binary64 tensors
    def normed(self, v, e):
        """norm(v), its 1 / deviation and its mean, all with bounds."""
        n = v.shape[1]
        steps = (n / 64 + 16) * U
        mean = v.mean(1, keepdim=True) if self.norm == "layer" else torch.zeros_like(v[:, :1])
        e_mean = (e.mean(1, keepdim=True) + steps * v.abs().mean(1, keepdim=True)) if self.norm == "layer" else 0.0
        d = v - mean
        e_d = e + e_mean + U * (v.abs() + mean.abs())
        var = (d * d).mean(1, keepdim=True) + self.eps
        rstd = var ** -0.5
        e_var = (2 * d.abs() * e_d + e_d ** 2).mean(1, keepdim=True) + 2 * steps * var
        e_rstd = rstd * (e_var / var + 4 * U)          # first order doubled: e_var is far below var
        vhat = d * rstd
        return (vhat, (e_d * rstd + d.abs() * e_rstd) * (1 + 1e-3) + 4 * U * vhat.abs()), (rstd, e_rstd), (mean, e_mean)

    def run(self):
        f = F64
        x, r = self.x.to(f), self.r.to(f)
        one = torch.ones((), dtype=f, device=x.device)
        self.g = one if self.gate is None else self.gate.to(f)
        zero = torch.zeros_like(x)
        if self.pw is None:
            self.xhat, self.xr = (x, zero), (one, 0 * one)
            t = (x, zero)
        else:
            self.xhat, self.xr, _ = self.normed(x, zero)
            pw = self.pw.to(f)
            t = (self.xhat[0] * pw, (self.xhat[1] + U * self.xhat[0].abs()) * pw.abs())
        self.t = t
        k = abs(self.scale) * self.g.abs()
        gated = self.scale * self.g * t[0]
        self.s = (r + gated, k * t[1] + 3 * U * gated.abs() + U * (r + gated).abs())
        if self.w is None:
            return
        self.shat, self.sr, _ = self.normed(*self.s)
        w = self.w.to(f)
        b = 0 * w if self.b is None else self.b.to(f)
        self.y = (self.shat[0] * w + b, self.shat[1] * w.abs() + 4 * U * ((self.shat[0] * w).abs() + b.abs()))

    def through(self, c, vhat, rstd):
        """The norm's gradient of c, all pairs."""
        n = c[0].shape[1]
        steps = (n / 64 + 16) * U

        def mean(v, e):
            return v.mean(1, keepdim=True), e.mean(1, keepdim=True) + steps * v.abs().mean(1, keepdim=True)
        q = mean(c[0] * vhat[0], c[1] * vhat[0].abs() + (c[0].abs() + c[1]) * vhat[1] + U * (c[0] * vhat[0]).abs())
        p = mean(*c) if self.norm == "layer" else (0.0 * q[0], 0.0 * q[0])
        inner = c[0] - p[0] - vhat[0] * q[0]
        e = c[1] + p[1] + vhat[0].abs() * q[1] + vhat[1] * (q[0].abs() + q[1]) + 3 * U * (
            c[0].abs() + p[0].abs() + (vhat[0] * q[0]).abs())
        return rstd[0] * inner, rstd[0] * e + rstd[1] * (inner.abs() + e) + 2 * U * (rstd[0] * inner).abs()

    def grads(self, dy=True, ds=True):
        f = F64
        n = self.x.shape[0]
        d = self.ds.to(f) if ds else torch.zeros_like(self.s[0])
        out = [None] * 6
        total = (d, torch.zeros_like(d))

        def summed(v, e):
            return v.sum(0), e.sum(0) + (n + 2) * U * (v.abs() + e).sum(0)
        if self.w is not None:
            dyd, w = self.dy.to(f), self.w.to(f)
            c = (dyd * w, U * (dyd * w).abs())
            v, e = self.through(c, self.shat, self.sr)
            # the norm's terms are added to ds one at a time: each rounding is of a partial
            # sum below |ds| and those terms, whose share `through` counts
            total = (d + v, e + 3 * U * d.abs() + U * (d + v).abs())
            out[2] = summed(dyd * self.shat[0], dyd.abs() * self.shat[1])
            if self.b is not None:
                out[3] = summed(dyd, 0 * dyd)
        out[1] = total
        k = abs(self.scale)
        if self.gate is not None:
            v = self.scale * total[0] * self.t[0]
            e = k * (total[1] * self.t[0].abs() + (total[0].abs() + total[1]) * self.t[1]) + 3 * U * v.abs()
            out[4] = (v, e) if self.gate.dim() == 2 else summed(v, e)
        dt = (self.scale * self.g * total[0], k * self.g.abs() * (total[1] + 3 * U * total[0].abs()))
        if self.pw is None:
            out[0] = dt
        else:
            out[5] = summed(dt[0] * self.xhat[0], dt[1] * self.xhat[0].abs() + (dt[0].abs() + dt[1]) * self.xhat[1])
            pw = self.pw.to(f)
            out[0] = self.through((dt[0] * pw, (dt[1] + U * dt[0].abs()) * pw.abs()), self.xhat, self.xr)
        return out


def check_forward(case, got):
    case.run()
    s, y = got[:2]
    close(s, *case.s)
    if case.w is None:
        assert y is None
    else:
        close(y, *case.y)


def check_backward(case, got, **which):
    want = case.grads(**which)
    for name, g, ref in zip(("dx", "dresidual", "dweight", "dbias", "dgate", "dpost_weight"), got, want):
        assert (g is None) == (ref is None), name
        if g is not None:
            try:
                close(g, *ref)
            except AssertionError as e:
                raise AssertionError("%s: %s" % (name, e))


@pytest.mark.parametrize("form", FORMS)
@pytest.mark.parametrize("dtype,wdtype", TYPES)
@pytest.mark.parametrize("rows,cols", SIZES)
def test_forward_and_backward(rows, cols, dtype, wdtype, form):
    case = Case(rows, cols, dtype, wdtype, form, seed=rows * 31 + cols)
    got = case.forward()
    assert got[0].dtype == got[1].dtype == dtype and got[2].shape == (rows, 4)
    check_forward(case, got)
    again = case.forward(stats=False)
    assert len(again) == 2 and torch.equal(again[0], got[0]) and torch.equal(again[1], got[1])
    grads = case.backward(got[2])
    check_backward(case, grads)
    assert all(p is q or torch.equal(p, q) for p, q in zip(case.backward(got[2]), grads))


@pytest.mark.parametrize("gate", [None, "row", "matrix"])
@pytest.mark.parametrize("norm,bias,post", list(itertools.product(["rms", "layer"], [False, True], [False, True])))
def test_every_form(norm, bias, post, gate):
    for rows, cols, scale in ((300, 520, 1.0), (40, 1003, 0.3)):
        for weighted in (True, False):
            case = Case(rows, cols, BF16, F32, (norm, bias, post, gate, scale), seed=cols, weighted=weighted)
            got = case.forward()
            check_forward(case, got)
            grads = case.backward(got[2])
            check_backward(case, grads)
            assert (grads[0] is grads[1]) == (gate is None and not post and scale == 1.0)
            assert (grads[1] is case.ds) == (not weighted)
            if weighted:
                check_backward(case, case.backward(got[2], ds=False), ds=False)


def test_many_rows():
    # more rows than workgroups take at once, and a last turn of a few
    for rows, cols, dtype in ((5000, 264, F16), (1029, 4096, BF16), (2061, 1000, F32)):
        case = Case(rows, cols, dtype, F32, ("layer", True, True, "row", 0.5), seed=3)
        got = case.forward()
        check_forward(case, got)
        check_backward(case, case.backward(got[2]))


@pytest.mark.parametrize("cols", [256, 1000, 4096, 20001])
def test_large_offset_and_constant_rows(cols):
    # mean 300 times the spread; a row without spread gives the bias (eps keeps it finite)
    case = Case(6, cols, F32, F32, ("layer", True, False, None, 1.0), seed=5)
    case.r += 300
    case.x[2], case.r[2] = 1.25, 2.0
    got = case.forward()
    check_forward(case, got)
    if cols <= 4096:                                        # sums of 3.25 that fp32 holds exactly
        assert torch.equal(got[1][2], case.b)


@pytest.mark.parametrize("dtype", [F16, BF16, F32])
@pytest.mark.parametrize("cols", [64, 1000, 8192, 20001])
def test_non_finite_rows_stay_apart(cols, dtype):
    case = Case(9, cols, dtype, dtype, ("layer", True, True, "matrix", 0.5), seed=6)
    clean = case.forward()
    grads = case.backward(clean[2])
    case.x[1, cols // 2] = float("nan")
    case.r[4, 0] = float("inf")
    case.gate[7, cols - 1] = float("-inf")
    got = case.forward()
    bad, good = [1, 4, 7], [0, 2, 3, 5, 6, 8]
    assert torch.isnan(got[1][bad]).all()
    assert all(torch.equal(p[good], q[good]) for p, q in zip(got, clean))
    after = case.backward(got[2])
    for k in (0, 1, 4):
        assert torch.equal(after[k][good], grads[k][good])
    for k in (2, 5):
        assert not torch.isfinite(after[k]).all()


def test_shapes_strides_and_alignment():
    case = Case(24, 1001, F16, F32, ("layer", True, True, "matrix", 0.5), seed=7)
    got = case.forward()
    grads = case.backward(got[2])
    plain = {k: getattr(case, k) for k in ("x", "r", "gate", "dy", "ds")}
    vectors = {k: getattr(case, k) for k in ("w", "b", "pw")}
    for move in (lambda t: strided(t, 5), shifted, lambda t: t.view(2, 3, 4, 1001)):
        for k, v in plain.items():
            setattr(case, k, move(v))
        for k, v in vectors.items():
            setattr(case, k, shifted(v))
        other = case.forward()
        assert all(torch.equal(p.reshape(q.shape), q) for p, q in zip(other, got))
        assert all(torch.equal(p.reshape(q.shape), q) for p, q in zip(case.backward(other[2]), grads))
    for k, v in plain.items():
        setattr(case, k, v[0])
    for k, v in vectors.items():
        setattr(case, k, v)
    one = gr.add_norm(case.x, case.r, case.w, case.b, scale=0.5, post_weight=case.pw, norm="layer")
    assert one[0].shape == (1001,) and one[1].shape == (1001,)


def test_no_rows():
    case = Case(0, 100, F16, F32, ("layer", True, True, "row", 0.5))
    s, y, stats = case.forward()
    assert s.shape == y.shape == (0, 100) and stats.shape == (0, 4)
    dx, dr, dw, db, dg, dp = case.backward(stats)
    assert dx.shape == dr.shape == (0, 100)
    assert all(v.shape == (100,) and not v.any() for v in (dw, db, dg, dp))


@pytest.mark.parametrize("form", [("rms", True, True, "row", 0.7), ("layer", True, True, "matrix", 0.7),
                                  ("layer", True, False, None, 1.0)])
def test_backward_against_differences(form):
    # central differences of the formula in binary64 (their own error is 1e-7 of the sizes
    # here); fp32 gradients, each off by at most a few hundred fp32 steps of the largest term
    rows, cols, h = 7, 65, 1e-4
    case = Case(rows, cols, F32, F32, form, seed=11)
    grads = case.backward(case.forward()[2])
    names = ["x", "r", "w", "b", "gate", "pw"]
    args = {k: None if getattr(case, k) is None else getattr(case, k).to(F64) for k in names}

    def normed(v):
        if case.norm == "layer":
            v = v - v.mean(1, keepdim=True)
        return v * ((v * v).mean(1, keepdim=True) + 1e-5) ** -0.5

    def loss(x, r, w, b, gate, pw):
        t = x if pw is None else normed(x) * pw
        s = r + case.scale * (t if gate is None else gate * t)
        return (case.ds.to(F64) * s).sum() + (case.dy.to(F64) * (normed(s) * w + b)).sum()

    for name, grad in zip(names, grads):
        if grad is None:
            assert args[name] is None
            continue
        for seed in range(3):
            v = rnd(20 + seed, *grad.shape).to(F64)
            diff = (loss(**{**args, name: args[name] + h * v}) - loss(**{**args, name: args[name] - h * v})) / (2 * h)
            assert abs(diff - (grad.to(F64) * v).sum()) <= 1e-4 * (grad.to(F64) * v).abs().sum() + 1e-6
