"""Orthogonalisation by Newton-Schulz steps on the GPU, against the steps in binary64.

Where every operand is exact in float16 the results have one right value.  Elsewhere the
bound is carried along the steps: with u = 2^-11 (float16's half step) and norms |.| of
Frobenius, ||.|| the largest singular value,
  E_A <= 2 u ||X|| |X| + u |A|,  E_B <= (|b| + 2 |c| ||A||) E_A + 2 |c| u ||A|| |A| + u |B|,
  E_X' <= L E_X + ||X|| E_B + u ||B|| |X|,  L the largest slope |a| + 3 |b| s^2 + 5 |c| s^4
at s = ||X||, to which a tenth is added for the products of errors and the fp32 sums.
"""
import ctypes

import pytest
import torch

import dense_tiled_gemm_relu_amd as gr
from tests.block_helpers import BF16, F16, F32, F64, ints, rnd

pytestmark = pytest.mark.gpu

QUINTIC = (3.4445, -4.7750, 2.0315)
SIZES = [(1, 1), (1, 64), (64, 1), (2, 3), (64, 64), (17, 300), (400, 33), (64, 512), (512, 64), (64, 513), (65, 65), (65, 200),
         (200, 65), (128, 128), (128, 256), (256, 128), (128, 257), (129, 129), (128, 130), (256, 256), (300, 1001), (1001, 300),
         (520, 520), (129, 2050), (1030, 1024), (2100, 2100), (4100, 700), (1, 700), (33, 5000), (16384, 64), (64, 16385), (128, 2048), (128, 4096),
         (4095, 90), (65, 1111)]


def largest(a):
    """At least a symmetric matrix's largest singular value, and at most p^(1/64) of it:
    the 32nd root of the norm of its 32nd power."""
    scale = a.norm()
    if scale == 0:
        return scale
    a = a / scale
    log = 0.0
    for k in range(5):
        a = a @ a
        size = a.norm()
        a, log = a / size, 2 * log + size.log()
    return scale * (log / 32).exp()


def steps_of(g, steps, coefficients, eps=1e-7):
    """The steps in binary64 and the bound of the Frobenius error."""
    x = g.to(F64)
    tall = x.shape[0] > x.shape[1]
    x = (x.t() if tall else x) / (x.norm() + eps)
    u, err = 2.0 ** -11, 0.0
    err = 2.0 ** -23 * x.norm()
    for a, b, c in ([coefficients] * steps if len(coefficients) == 3 and not hasattr(coefficients[0], "__len__") else coefficients):
        gram = x @ x.t()
        poly = b * gram + c * gram @ gram
        s = largest(gram) ** 0.5
        fx, fa, fb, s2b = x.norm(), gram.norm(), poly.norm(), largest(poly)
        ea = 2 * u * s * fx + u * fa
        eb = (abs(b) + 2 * abs(c) * s ** 2) * ea + 2 * abs(c) * u * s ** 2 * fa + u * fb
        slope = abs(a) + 3 * abs(b) * s ** 2 + 5 * abs(c) * s ** 4
        # below s the slope is largest at 0 or at s; |a| is the one that lifts what is small
        at_s = (a + 3 * b * s ** 2 + 5 * c * s ** 4).abs()
        err = (slope if s > 0.6 else torch.clamp(at_s, min=abs(a))) * err + 1.1 * (s * eb + u * s2b * fx)
        x = a * x + poly @ x
    return (x.t() if tall else x), err


def spectra(m, n, seed):
    p = min(m, n)
    yield "noise", rnd(seed, m, n)
    yield "few directions", rnd(seed + 1, m, max(1, p // 16)) @ rnd(seed + 2, max(1, p // 16), n) + rnd(seed + 3, m, n)
    if p >= 64:
        # columns nearly orthogonal, of lengths over four decades
        yield "decades", (rnd(seed + 4, m, p) * torch.logspace(0, -4, p, device="cuda")) @ rnd(seed + 5, p, n)


@pytest.mark.parametrize("dtype", [F16, BF16, F32])
@pytest.mark.parametrize("m,n", SIZES)
def test_orthogonalize(m, n, dtype):
    for name, g in spectra(m, n, m + 7 * n):
        g = (1e-2 * g).to(dtype)
        want, err = steps_of(g, 5, QUINTIC)
        got = gr.orthogonalize(g)
        assert got.dtype == BF16 and got.shape == g.shape
        off, size = (got.to(F64) - want).norm(), want.norm()
        assert off <= err + 2.0 ** -8 * size, name
        # what is documented: 1e-3, and the rounding
        assert off <= (1e-3 + 2.0 ** -8) * size, (name, float(off / size))
        assert torch.equal(gr.orthogonalize(g), got)


def scattered(m, n, k, seed):
    """4^k entries of +-1, the others 0, so that the norm is 2^k."""
    gen = torch.Generator(device="cuda")
    gen.manual_seed(seed)
    g = torch.zeros(m * n, device="cuda")
    at = torch.randperm(m * n, generator=gen, device="cuda")[:4 ** k]
    g[at] = (2 * ints(seed, 0, 1, 4 ** k) - 1).float()
    return g.view(m, n)


@pytest.mark.parametrize("dtype", [F16, BF16, F32])
@pytest.mark.parametrize("m,n,k", [(1, 1, 0), (1, 64, 2), (64, 1, 2), (5, 7, 2), (64, 64, 4), (60, 500, 4), (500, 60, 4),
                                   (30, 300, 3), (300, 30, 3), (33, 100, 3), (128, 128, 4), (100, 250, 4), (250, 100, 4), (65, 200, 4), (200, 65, 4),
                                   (130, 131, 4), (256, 256, 5), (300, 1001, 5), (1001, 300, 5), (520, 520, 5), (129, 2050, 5),
                                   (1030, 1024, 5), (2100, 2100, 6), (4100, 700, 6), (700, 9000, 6), (50, 4001, 4), (16384, 64, 4),
                                   (128, 2048, 4), (128, 4096, 4), (3000, 100, 4), (70, 300, 4)])
def test_exact_step(m, n, k, dtype):
    # few entries a row: A and A^2 are whole numbers of at most 9 bits times a power of two,
    # and so is B where it is a multiple of one of them
    g = scattered(m, n, k, m + n)
    x = g.to(F64) / 2 ** k
    x = x.t() if m > n else x
    gram = x @ x.t()
    scaled = gram * 4 ** k
    assert (scaled @ scaled).abs().max() < 2 ** 9
    for a, b, c in ((1.5, -0.5, 0.0), (1.0, 0.0, 4.0 ** k), (2.0, -1.5, 0.5)):
        poly = b * gram + c * gram @ gram
        want = a * x + poly @ x
        got = gr.orthogonalize(g.to(dtype), 1, (a, b, c), 0.0).to(F64)
        got = got.t() if m > n else got
        if b == 0 or c == 0:
            assert torch.equal(got, want.to(BF16).to(F64))
        else:
            # b A has up to 9 + 2 k bits more than c A^2, so B off its diagonal takes one
            # rounding to float16 (half a step 2^-11; below 2^-22 a multiple of 2^-32);
            # everything else is exact, or an fp32 sum of at most 2^9 such terms
            off = poly - torch.diag(poly.diag())
            lost = (2.0 ** -11 * off.abs() + 2.0 ** -33 * (off != 0)) @ x.abs()
            bound = lost * (1 + 2.0 ** -8) + (2.0 ** -8 + 2.0 ** -20) * want.abs()
            assert ((got - want).abs() <= bound).all()


def test_no_steps_give_the_scaled_matrix():
    g = scattered(70, 90, 3, 1).to(F16)
    assert torch.equal(gr.orthogonalize(g, 0, eps=0.0), (g.float() / 8).to(BF16))


def test_coefficients_of_each_step():
    g = rnd(3, 200, 333).to(BF16)
    schedule = [(3.4445, -4.7750, 2.0315)] * 3 + [(1.875, -1.25, 0.375)] * 5
    want, err = steps_of(g, len(schedule), schedule)
    got = gr.orthogonalize(g, len(schedule), schedule)
    assert (got.to(F64) - want).norm() <= err + 2.0 ** -8 * want.norm()
    # the last five converge: the rows are orthonormal to the rounding of the result
    gram = got.to(F64) @ got.to(F64).t()
    assert (gram - torch.eye(200, device="cuda", dtype=F64)).abs().max() <= 4 * 2.0 ** -9
    assert torch.equal(gr.orthogonalize(g, 3, schedule[:3]), gr.orthogonalize(g, 3))


@pytest.mark.parametrize("m,n", [(50, 31), (50, 1000), (1500, 100), (100, 70), (70, 100), (200, 300), (300, 200), (256, 512), (1100, 1200)])
def test_batches_and_strides(m, n):
    g = rnd(5, 5, m, n).to(BF16)
    g[1] *= 1e-20
    g[2] *= 1e20
    g[3] = 0
    one = torch.stack([gr.orthogonalize(v) for v in g])
    assert torch.equal(gr.orthogonalize(g), one) and not one[3].any() and torch.isfinite(one).all()
    wide = torch.full((5, m + 3, n + 5), float("nan"), dtype=BF16, device="cuda")
    wide[:, 1:m + 1, 2:n + 2] = g
    assert torch.equal(gr.orthogonalize(wide[:, 1:m + 1, 2:n + 2]), one)
    assert torch.equal(gr.orthogonalize(wide[0, 1:m + 1, 2:n + 2]), one[0])
    assert torch.equal(gr.orthogonalize(g.transpose(0, 1).contiguous().transpose(0, 1)), one)      # rows of the batch in turn
    assert torch.equal(gr.orthogonalize(g[:1].expand(3, m, n)), one[:1].expand(3, m, n))


def test_scale_does_not_matter():
    g = rnd(6, 90, 200)
    want = gr.orthogonalize(g)
    for k in (-100, -20, 20, 100):
        assert torch.equal(gr.orthogonalize(g * 2.0 ** k, eps=0.0), gr.orthogonalize(g, eps=0.0)), k
    assert torch.isfinite(want).all()


def test_non_finite_matrices_stay_apart():
    for m, n in ((100, 130), (300, 130), (100, 600), (3000, 40)):
        g = rnd(7, 4, m, n)
        clean = gr.orthogonalize(g)
        g[1, m - 1, n - 1], g[2, 0, 0] = float("nan"), float("inf")
        got = gr.orthogonalize(g)
        assert torch.isnan(got[1]).all() and torch.isnan(got[2]).all()
        assert torch.equal(got[[0, 3]], clean[[0, 3]])


def test_plans_by_size():
    plan = lambda *size: gr.library().gemm_relu_orthogonalize_plan(*size).decode()
    assert plan(1, 64, 512) == plan(1000, 256, 128) == "small"
    assert plan(1, 64, 513) == plan(85, 600, 20) == plan(1, 128, 2048) == plan(4, 16384, 64) == "long"
    assert all("," in plan(*size) for size in ((1, 129, 300), (1, 128, 2049), (5, 16384, 64), (1, 64, 16385)))


def test_long_workspace_with_nothing_behind_it():
    # sizes at the ends of the rule: what lies behind each of its parts stays as it is
    g = rnd(9, 3, 100, 700)
    want = gr.orthogonalize(g)
    lib = gr.library()
    need = lib.gemm_relu_orthogonalize_workspace(3, 100, 700)
    ws = torch.full((need + 4096,), 77, dtype=torch.uint8, device="cuda")
    out = torch.full((3 * 100 * 700 + 512,), 5.0, dtype=BF16, device="cuda")
    c = (ctypes.c_float * 15)(*(QUINTIC * 5))
    status = lib.gemm_relu_orthogonalize(g.data_ptr(), 700, 70000, out.data_ptr(), 3, 100, 700, 2, c, 5, 1e-7,
                                         ws.data_ptr(), need, torch.cuda.current_stream().cuda_stream)
    assert status == 0 and torch.equal(out[:210000].view(3, 100, 700), want)
    assert (out[210000:] == 5).all() and (ws[need:] == 77).all()


@pytest.mark.parametrize("m,n", [(20, 30), (100, 300), (300, 100)])
def test_without_steps_or_norm(m, n):
    # no steps: the normed matrix itself, where an infinity stays at its place; 0 / 0 with eps 0
    g = rnd(8, m, n)
    g[3, 4] = float("inf")
    got = gr.orthogonalize(g, 0)
    assert torch.isnan(got[3, 4]) and int(torch.isnan(got).sum()) == 1 and int(got.count_nonzero()) == 1
    zero = torch.zeros(m, n, device="cuda")
    assert not gr.orthogonalize(zero).any() and torch.isnan(gr.orthogonalize(zero, eps=0.0)).all()


def test_empty_sizes():
    for shape in ((0, 5), (5, 0), (0, 4, 5), (3, 0, 5)):
        assert gr.orthogonalize(torch.zeros(shape, device="cuda")).shape == shape


@pytest.mark.parametrize("batch,m,n,names", [
    (1, 2900, 2890, "d128x128x64_s4_i16w8/d64x64x64_s4"), (2, 2880, 3000, "d128x128x64_s2w8/d64x64x64_s4"),
    (3, 3300, 3264, "d256x256x32_s4_i16w8/d128x128x64_s4_i16w8"), (1, 5900, 5800, "d256x256x32_s4_i16w8/d64x64x64_s4")])
def test_diagonal_tiles_in_a_launch_of_their_own(batch, m, n, names):
    # exact as in test_exact_step: the products' tiles below the diagonal and those on it, the
    # last ones past the edge
    assert names in gr.library().gemm_relu_orthogonalize_plan(batch, m, n).decode()
    k = 6
    g = torch.stack([scattered(m, n, k, 7 * i) for i in range(batch)])
    for a, b, c in ((1.5, -0.5, 0.0), (1.0, 0.0, 4.0 ** k)):
        got = gr.orthogonalize(g.to(BF16), 1, (a, b, c), 0.0)
        for x, y in zip(g.to(F64) / 2 ** k, got.to(F64)):
            x, y = (x.t(), y.t()) if m > n else (x, y)
            gram = x @ x.t()
            assert ((gram * 4 ** k) @ (gram * 4 ** k)).abs().max() < 2 ** 9
            assert torch.equal(y, (a * x + (b * gram + c * gram @ gram) @ x).to(BF16).to(F64))
    want = torch.stack([gr.orthogonalize(v) for v in rnd(1, batch, m, n)])
    if batch == 1:
        ref, err = steps_of(rnd(1, batch, m, n)[0], 5, QUINTIC)
        assert (want[0].to(F64) - ref).norm() <= (1e-3 + 2.0 ** -8) * ref.norm()
