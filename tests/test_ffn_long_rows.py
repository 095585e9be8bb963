"""Rows longer than a workgroup's registers hold, up to the longest a call takes.

The largest sizes hold rows of 2^31 - 1 elements: column numbers and their
successors pass 31 bits, and a thread adds millions of terms.
"""
import pytest
import torch

import dense_tiled_gemm_relu_amd as gr

pytestmark = pytest.mark.gpu

F16, F32, F64 = torch.float16, torch.float32, torch.float64
U = 2.0 ** -24                             # half a step of fp32
LONGEST = 2 ** 31 - 1
PIECE = 2 ** 27
# a thread's batch of at most 16 terms is added in fp32: its terms and its partial sums
# round once each (32 roundings at most); all else is binary64
BATCH = 32 * U


@pytest.fixture(autouse=True)
def _gpu():
    assert torch.cuda.is_available(), "GPU tests need the MI355X"
    yield
    torch.cuda.empty_cache()


def pieces(n):
    return [slice(k, min(n, k + PIECE)) for k in range(0, n, PIECE)]


def total(f, n):
    """Sum of f(piece) in binary64."""
    return sum(float(f(p).sum()) for p in pieces(n))


def row(n, seed, dtype=F16):
    """An offset of 1.3 with noise: sums that fp32 cannot hold term by term."""
    gen = torch.Generator(device="cuda")
    gen.manual_seed(seed)
    x = torch.empty(1, n, dtype=dtype, device="cuda")
    for p in pieces(n):
        x[0, p] = (1.3 + 0.5 * torch.randn(p.stop - p.start, generator=gen, device="cuda")).to(dtype)
    return x


def near(got, ref, bound):
    bad = ~((got.to(F64) - ref).abs() <= bound)
    assert not bad.any(), (int(bad.sum()), got[bad][:3], ref[bad][:3], bound[bad][:3])


@pytest.mark.parametrize("n", [5, 40000, 10 ** 7 + 3, LONGEST])
def test_layer_norm_of_one_long_row(n):
    eps = 1e-5
    x = row(n, 1)
    w = torch.ones(n, dtype=F16, device="cuda")
    w[n - 1] = 2.0
    w[0] = -1.0
    y, mean, rstd = gr.layer_norm(x, w, None, eps, stats=True)
    m = total(lambda p: x[0, p].to(F64), n) / n
    var = total(lambda p: (x[0, p].to(F64) - m) ** 2, n) / n
    r = (var + eps) ** -0.5
    off = (BATCH + U) * total(lambda p: x[0, p].to(F64).abs(), n) / n          # of the mean
    assert abs(float(mean) - m) <= off
    # x - mean and its square round; a mean off by d adds d^2 to the variance; the quotient and the root
    lost = BATCH + 4 * U + off ** 2 / (2 * (var + eps)) + 3 * U
    assert abs(float(rstd) - r) <= lost * r
    for p in pieces(n):
        ref = (x[0, p].to(F64) - m) * r * w[p].to(F64)
        near(y[0, p], ref, 2.0 ** -11 * ref.abs() + 2 * (lost + 4 * U) * ref.abs() + 2 * off * r * w[p].to(F64).abs() + 2.0 ** -24)


@pytest.mark.parametrize("n", [5, 40000, 10 ** 7 + 3, LONGEST])
def test_layer_norm_backward_of_one_long_row(n):
    x, dy = row(n, 2), row(n, 3)
    w = torch.ones(n, dtype=F16, device="cuda")
    w[n - 1] = 2.0
    mean, rstd = torch.full((1,), 1.25, device="cuda"), torch.full((1,), 1.75, device="cuda")
    dx, dw, db = gr.layer_norm_backward(dy, x, w, mean, rstd)

    def xhat(p):
        return (x[0, p].to(F64) - 1.25) * 1.75

    def c(p):
        return dy[0, p].to(F64) * w[p].to(F64)
    s0, s1 = total(c, n) / n, total(lambda p: c(p) * xhat(p), n) / n
    a0, a1 = total(lambda p: c(p).abs(), n) / n, total(lambda p: (c(p) * xhat(p)).abs(), n) / n
    for p in pieces(n):
        xh = xhat(p)
        ref = 1.75 * (c(p) - s0 - xh * s1)
        # the sums, then a dozen roundings of terms of at most the magnitudes' size
        slack = 1.75 * ((BATCH + 12 * U) * (a0 + xh.abs() * a1) + 12 * U * c(p).abs())
        near(dx[0, p], ref, 2.0 ** -11 * (ref.abs() + slack) + slack + 2.0 ** -24)
        # one row: no sums
        ref = dy[0, p].to(F64) * xh
        near(dw[p], ref, (2.0 ** -11 + 4 * U) * ref.abs() + 2.0 ** -24)
        assert torch.equal(db[p], dy[0, p])


@pytest.mark.parametrize("n", [5, 40000, LONGEST])
def test_quantize_one_long_row(n):
    x = row(n, 4)
    x[0, n - 1] = -60.0                    # the largest is the last
    q, s = gr.quantize_rows(x)
    assert abs(float(s) - 60 / 127) <= U
    for p in pieces(n):
        assert torch.equal(q[0, p].to(F64), torch.round(127 * x[0, p].to(F64) / 60))


@pytest.mark.parametrize("dtype", [F16, torch.bfloat16, F32])
def test_long_rows_of_several(dtype):
    # the rows' sums use two buffers in turn
    x = torch.cat([row(40001, k, dtype) for k in range(7)])
    w = torch.ones(40001, dtype=dtype, device="cuda")
    y, mean, rstd = gr.layer_norm(x, w, stats=True)
    dx = gr.layer_norm_backward(y, x, w, mean, rstd)[0]
    q, s = gr.quantize_rows(x)
    for k in range(7):
        one, m, r = gr.layer_norm(x[k:k + 1], w, stats=True)
        assert torch.equal(one, y[k:k + 1]) and torch.equal(m, mean[k:k + 1]) and torch.equal(r, rstd[k:k + 1])
        assert torch.equal(gr.layer_norm_backward(one, x[k:k + 1], w, m, r)[0], dx[k:k + 1])
        qk, sk = gr.quantize_rows(x[k:k + 1])
        assert torch.equal(qk, q[k:k + 1]) and torch.equal(sk, s[k:k + 1])
