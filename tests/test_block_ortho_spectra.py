"""The orthogonalisation's accuracy, for matrices whose singular values lie far apart too.

What is documented (include/gemm_relu_block.h) is stated for the result before its rounding
to bfloat16, in shares of its Frobenius norm.  An element's rounding is at most half a step
of bfloat16 at its magnitude, so what an element is off beyond that is at most its error
before the rounding: the norm of these excesses is held to the documented share.

That the documented shares follow from the roundings the header names is shown on the CPU:
`rounded` carries the steps out in binary64 with those roundings only.  A and B = b A + c A^2
are rounded as operands, X as a whole meets B; so a rounding is a factor on X's left, and
what it does to a singular direction is a share of that direction.
"""
import pytest
import torch

import dense_tiled_gemm_relu_amd as gr

F16, BF16, F32, F64 = torch.float16, torch.bfloat16, torch.float32, torch.float64
QUINTIC = (3.4445, -4.7750, 2.0315)
CUBIC, CONVERGING = (1.5, -0.5, 0.0), (1.875, -1.25, 0.375)


def documented(p, coefficients, steps):
    """The share of the norm that a result of shorter side p may be off before its rounding."""
    if coefficients == QUINTIC:
        if p >= 16:
            return 3e-3 if steps <= 6 else 1.2e-2
        return 1e-2
    return 1.5e-3


def schedules(p):
    yield QUINTIC, 5
    if p >= 16:
        yield QUINTIC, 4
        yield QUINTIC, 6
        yield QUINTIC, 10
    yield CUBIC, 12
    yield CONVERGING, 12


def matrices(m, n, seed, device):
    """Noise, few directions over noise that is ever smaller, and singular values over decades."""
    gen = torch.Generator().manual_seed(seed)

    def randn(*shape):
        return torch.randn(*shape, generator=gen, dtype=F64)
    p = min(m, n)
    few = max(1, p // 16)
    yield "noise", randn(m, n).to(device)
    for noise in (1e-2, 1e-3, 1e-4):
        low = randn(m, few) @ randn(few, n) * few ** -0.5
        yield "%d directions over %g" % (few, noise), (low + noise * randn(m, n)).to(device)
    u, v = torch.linalg.qr(randn(m, p))[0], torch.linalg.qr(randn(n, p))[0]
    for decades in (2, 4, 6):
        yield "%d decades" % decades, ((u * torch.logspace(0, -decades, p, dtype=F64)) @ v.t()).to(device)


def exact(g, coefficients, steps, eps=1e-7):
    x = g.to(F64)
    tall = x.shape[0] > x.shape[1]
    x = (x.t() if tall else x) / (x.norm() + eps)
    a, b, c = coefficients
    for _ in range(steps):
        gram = x @ x.t().contiguous()
        x = a * x + (b * gram + c * gram @ gram) @ x
    return x.t() if tall else x


def half(v, scale):
    """v as float16 under a scale, and 2048 times what that loses as another."""
    v = (v * scale).float().to(F64)
    hi = v.to(F16).to(F64)
    return hi / scale, ((v - hi) * 2048).to(F16).to(F64) / 2048 / scale


def rounded(g, coefficients, steps, eps=1e-7):
    """The steps with the roundings that the header names, sums exact."""
    x = g.to(F64)
    x = x.t() if x.shape[0] > x.shape[1] else x
    x = x / (x.norm() + eps)
    a, b, c = coefficients
    for _ in range(steps):
        hi, lo = half(x, 256.0)
        gram = hi @ hi.t()
        d = gram.diag().float().to(F64)
        off, _ = half(gram - torch.diag(gram.diag()), 1024.0)
        square = off @ off
        poly = b * off + c * (square + (d[:, None] + d[None, :]) * off)
        on = (b * d + c * (square.diag() + d * d)).float().to(F64)
        poly, _ = half(poly - torch.diag(poly.diag()), 256.0)
        x = ((a + on)[:, None] * (hi + lo) + poly @ (hi + lo)).float().to(F64)
    return x.t() if g.shape[0] > g.shape[1] else x


@pytest.mark.parametrize("m,n", [(1, 5), (3, 4), (6, 2), (9, 40), (16, 16), (17, 60), (33, 200), (64, 64), (130, 90), (200, 200)])
def test_documented_shares_follow_from_the_roundings(m, n):
    for name, g in matrices(m, n, 31 * m + n, "cpu"):
        for coefficients, steps in schedules(min(m, n)):
            want = exact(g, coefficients, steps)
            off = (rounded(g, coefficients, steps) - want).norm() / want.norm()
            assert off <= documented(min(m, n), coefficients, steps), (name, coefficients, steps, float(off))


def excess(got, want):
    """The norm of what elements are off beyond half a step of bfloat16 (eps 2^-7) at their magnitude."""
    v = got.to(F64)
    _, exponent = torch.frexp(v)                             # v = m 2^exponent, 0.5 <= m < 1
    step = torch.ldexp(torch.ones_like(v), exponent.clamp(min=-125) - 8)
    return ((v - want).abs() - step / 2).clamp(min=0).norm()


# (one launch), (one launch a step), (tiles), tall ones of each
SHAPES = [(1, 1), (3, 4), (6, 2), (7, 100), (16, 16), (17, 40), (40, 17), (33, 300), (64, 64), (64, 512), (100, 200), (256, 128),
          (16, 5000), (33, 4100), (5000, 33), (64, 1024), (100, 700), (700, 128), (128, 2048),
          (200, 200), (130, 300), (1000, 200), (200, 1000), (129, 2050), (513, 512), (100, 4500)]


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("m,n", SHAPES)
def test_far_apart_singular_values(m, n, dtype):
    for name, g in matrices(m, n, 31 * m + n, "cuda"):
        g = (1e-2 * g).to(dtype)
        for coefficients, steps in schedules(min(m, n)):
            want = exact(g, coefficients, steps)
            off = excess(gr.orthogonalize(g, steps, coefficients), want) / want.norm()
            assert off <= documented(min(m, n), coefficients, steps), (name, coefficients, steps, float(off))


@pytest.mark.gpu
@pytest.mark.parametrize("m,n", [(33, 300), (64, 1024), (200, 300), (300, 200)])
def test_far_apart_singular_values_in_a_batch(m, n):
    g = torch.stack([g for _, g in matrices(m, n, 7, "cuda")]).float()
    got = gr.orthogonalize(g)
    for one, result in zip(g, got):
        want = exact(one, QUINTIC, 5)
        assert excess(result, want) <= documented(min(m, n), QUINTIC, 5) * want.norm()


@pytest.mark.gpu
@pytest.mark.parametrize("steps", [0, 5])
@pytest.mark.parametrize("dtype,least", [(F16, 2.0 ** -24), (BF16, 2.0 ** -133), (F32, 2.0 ** -149)])
@pytest.mark.parametrize("m,n", [(5, 7), (60, 100), (100, 60), (100, 250), (64, 1024), (700, 100), (200, 300), (300, 200)])
def test_values_below_the_normal_range(m, n, dtype, least, steps):
    # a power of two times whole numbers, all of them multiples of the type's smallest value:
    # with eps 0 X is the same as without the factor, to the bit
    gen = torch.Generator().manual_seed(m + n)
    whole = torch.randint(-9, 10, (m, n), generator=gen).float()
    tiny = (whole.to(F64) * least).to(dtype)
    assert torch.equal(tiny.to(F64), whole.to(F64) * least)
    got = gr.orthogonalize(tiny.cuda(), steps, eps=0.0)
    assert torch.equal(got, gr.orthogonalize(whole.to(dtype).cuda(), steps, eps=0.0)) and got.any()
