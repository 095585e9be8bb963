"""Paths of the operators around the half layer that few sizes take: each is asserted by the
plan before its results are."""
import pytest
import torch

import dense_tiled_gemm_relu_amd as gr
from tests.block_helpers import ACTS, BF16, F16, F32, F64, U, act_ref, close, ints, rnd, shifted, strided


def act_plan(rows, n, k):
    return gr.library().gemm_relu_act_plan(rows, n, k, gr.BF16).decode()


# odd rows, columns and K: the residual's, the bias's and K's ends inside a tile
TILE_48X32 = [(37, 6837, 789), (226, 1628, 127), (134, 2649, 3846)]


def test_the_sizes_take_these_paths():
    assert all(act_plan(*size) == "k48x32x64_s3" for size in TILE_48X32)


@pytest.mark.gpu
@pytest.mark.parametrize("act", ACTS)
@pytest.mark.parametrize("dtype,bias_dtype", [(F16, F32), (BF16, BF16)])
@pytest.mark.parametrize("rows,n,k", TILE_48X32)
def test_48x32_tiles(rows, n, k, dtype, bias_dtype, act):
    x, w = rnd(1, rows, k).to(dtype), (rnd(2, n, k) * k ** -0.5).to(dtype)
    b, r = (0.5 * rnd(3, n)).to(bias_dtype), (4 * rnd(4, rows, n)).to(dtype)
    y, z = gr.matmul_act(x, w, b, act, r, save=True)
    sums = x.to(F64) @ w.to(F64).t() + b.to(F64)
    off = (k + 2) * U * (x.to(F64).abs() @ w.to(F64).abs().t() + b.to(F64).abs())
    value, _ = act_ref(sums, act)
    # as in test_block_act: slopes below 1.2; the tails' relative steps; the sum with the residual
    own = 0.0 if act == "none" else (16 + 4 * sums * sums).clamp(max=1e4) * U * value.abs()
    close(y, value + r.to(F64), 1.2 * off + own + U * (value.abs() + r.to(F64).abs()))
    if act != "none":
        close(z, sums, off)
    for args in ((strided(x, 3), strided(w, 5), shifted(b), act, strided(r, 1)), (shifted(x), shifted(w), b, act, shifted(r))):
        assert torch.equal(gr.matmul_act(*args), y)


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", [F16, BF16])
@pytest.mark.parametrize("rows,n,k", TILE_48X32)
def test_48x32_tiles_on_integers(rows, n, k, dtype):
    # sums of at most 8 bits: each result has exactly one right value
    x, w = ints(1, -1, 1, rows, k), ints(2, -1, 1, n, k) * (ints(3, 0, max(15, k // 8), n, k) == 0)
    b, r = ints(4, -8, 8, n), ints(5, -64, 64, rows, n)
    z = x.to(F64) @ w.to(F64).t() + b
    assert z.abs().max() <= 128
    for act, v in (("none", z), ("relu", z.clamp(min=0))):
        y = gr.matmul_act(x.to(dtype), w.to(dtype), b.to(dtype), act, r.to(dtype))
        assert torch.equal(y.to(F64), v + r)
