"""Paths of the operators around the half layer that few sizes take: each is asserted by the
plan before its results are."""
import pytest
import torch

import dense_tiled_gemm_relu_amd as gr
from tests.block_helpers import ACTS, BF16, F16, F32, F64, U, act_ref, close, ints, rnd, shifted, strided


def act_plan(rows, n, k):
    return gr.library().gemm_relu_act_plan(rows, n, k, gr.BF16).decode()


def ortho_plan(batch, m, n):
    return gr.library().gemm_relu_orthogonalize_plan(batch, m, n).decode()


# odd rows, columns and K: the residual's, the bias's and K's ends inside a tile
TILE_48X32 = [(37, 6837, 789), (226, 1628, 127), (134, 2649, 3846)]
# batch, rows, columns, parts of A's K
CUT = [(1, 300, 900, 3), (1, 1001, 300, 4), (3, 256, 1024, 4), (1, 320, 1600, 5), (1, 512, 2048, 7), (1, 129, 5000, 8),
       (1, 16385, 64, 8), (1, 1000, 3001, 3)]


def test_the_sizes_take_these_paths():
    assert all(act_plan(*size) == "k48x32x64_s3" for size in TILE_48X32)
    assert all("*" not in ortho_plan(*size) for size in ((1, 129, 300), (1, 2100, 2100), (8, 1024, 2048)))
    for batch, m, n, parts in CUT:
        assert ortho_plan(batch, m, n).startswith("d64x64x64_s4*%d," % parts), (m, n, ortho_plan(batch, m, n))


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


def scattered(m, n, k, seed):
    """4^k entries of +-1, the others 0, so that the norm is 2^k."""
    gen = torch.Generator().manual_seed(seed)
    g = torch.zeros(m * n)
    g[torch.randperm(m * n, generator=gen)[:4 ** k]] = (2 * torch.randint(0, 2, (4 ** k,), generator=gen) - 1).float()
    return g.view(m, n).cuda()


@pytest.mark.gpu
@pytest.mark.parametrize("batch,m,n,parts", CUT)
def test_products_cut_along_k(batch, m, n, parts):
    # A and A^2 are whole numbers of at most 9 bits times a power of two, and B is a multiple
    # of one of them: exactly one right result
    k = 5 if min(m, n) > 64 else 4
    g = torch.stack([scattered(m, n, k, 3 * i) for i in range(batch)])
    g = g if batch > 1 else g[0]
    for a, b, c in ((1.5, -0.5, 0.0), (1.0, 0.0, 4.0 ** k)):
        got = gr.orthogonalize(g, 1, (a, b, c), 0.0)
        for x, y in zip(g.view(batch, m, n).to(F64) / 2 ** k, got.view(batch, m, n).to(F64)):
            x, y = (x.t(), y.t()) if m > n else (x, y)
            gram = x @ x.t()
            assert ((gram * 4 ** k) @ (gram * 4 ** k)).abs().max() < 2 ** 9
            assert torch.equal(y, (a * x + (b * gram + c * gram @ gram) @ x).to(BF16).to(F64))


@pytest.mark.gpu
@pytest.mark.parametrize("batch,m,n,parts", CUT)
def test_products_cut_along_k_in_a_graph_and_on_two_streams(batch, m, n, parts):
    # the arrival counters stand in each call's own workspace and are left cleared
    shape = (batch, m, n) if batch > 1 else (m, n)
    g, other = rnd(1, *shape).to(BF16), rnd(2, *shape).to(BF16)
    want, want2 = gr.orthogonalize(g), gr.orthogonalize(other)
    streams = torch.cuda.Stream(), torch.cuda.Stream()
    torch.cuda.synchronize()
    for _ in range(3):
        a, b = gr.orthogonalize(g, stream=streams[0]), gr.orthogonalize(other, stream=streams[1])
        torch.cuda.synchronize()
        assert torch.equal(a, want) and torch.equal(b, want2)
    graph, kept = torch.cuda.CUDAGraph(), g.clone()
    with torch.cuda.graph(graph, stream=streams[0]):
        out = gr.orthogonalize(g)
    for k in range(4):
        g.copy_(other if k % 2 else kept)
        out.zero_()
        gr.orthogonalize(other)
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, want2 if k % 2 else want), k


@pytest.mark.gpu
@pytest.mark.parametrize("m,n", [(20001, 60001), (60001, 20001)])
def test_matrices_past_32_bits(m, n):
    # X's two halves are one operand of 2.4e9 values, 4.8 GB.  g is zero but for some rows and
    # columns, the first and the last among them: exact there as above, and zero elsewhere
    if torch.cuda.mem_get_info()[0] < 40 << 30:
        pytest.skip("needs 40 GB")
    gen = torch.Generator().manual_seed(5)
    rows = torch.cat([torch.tensor([0, m - 1]), 1 + torch.randperm(m - 2, generator=gen)[:62]]).sort().values.cuda()
    cols = torch.cat([torch.tensor([0, n - 1]), 1 + torch.randperm(n - 2, generator=gen)[:298]]).sort().values.cuda()
    part = scattered(64, 300, 4, 11)
    part[0, 0] = part[0, 299] = part[63, 0] = part[63, 299] = 0
    at = part.view(-1).nonzero()[:4, 0]                      # four entries move to the corners
    part.view(-1)[at] = 0
    part[0, 0] = part[0, 299] = part[63, 0] = part[63, 299] = 1
    assert part.norm() == 16
    g = torch.zeros(m, n, dtype=BF16, device="cuda")
    g[rows[:, None], cols[None, :]] = part.to(BF16)
    x = part.to(F64) / 16
    gram = x @ x.t()
    assert ((256 * gram) @ (256 * gram)).abs().max() < 2 ** 9
    for a, b, c in ((1.5, -0.5, 0.0), (1.0, 0.0, 256.0)):
        got = gr.orthogonalize(g, 1, (a, b, c), 0.0)
        inside = got[rows[:, None], cols[None, :]]
        want = (a * x + (b * gram + c * gram @ gram) @ x).to(BF16)
        assert torch.equal(inside, want)
        assert int(got.count_nonzero()) == int(want.count_nonzero())
