"""Which kernel configuration the feed-forward products take, on the host."""
import itertools

import dense_tiled_gemm_relu_amd as gr

SIZES = (1, 3, 16, 40, 64, 100, 300, 1000, 2048, 4096, 8192)


def test_every_configuration_is_reached():
    lib = gr.library()
    gated = {lib.gemm_relu_gated_plan(m, n, k, gr.F16) for m, n, k in itertools.product(SIZES, SIZES, SIZES)}
    i8 = {lib.gemm_relu_i8_plan(m, n, k, gr.F16) for m, n, k in itertools.product(SIZES, SIZES, SIZES)}
    for sizes in ((100, 3000, 3000), (40, 7000, 3000)):           # just over a round of 32 x 32 tiles
        i8.add(lib.gemm_relu_i8_plan(*sizes, gr.F16))
        gated.add(lib.gemm_relu_gated_plan(sizes[0], sizes[1] // 2, sizes[2], gr.F16))
    tiles = {b"d256x256x32_s4_i16w8", b"d128x128x64_s4_i16w8", b"d128x128x64_s2w8", b"d64x64x64_s4"}
    assert gated == i8 == tiles | {b"k16x16x64_s4", b"k32x32x64_s4", b"k32x48x64_s3", b"k48x32x64_s3"}
    back = set()
    for m, n, k in itertools.product(SIZES, SIZES, SIZES):
        back.update(lib.gemm_relu_gated_backward_plan(m, n, k, gr.BF16).split(b","))
    assert back == tiles | {b"g64x64x64"}                    # columns fewer than a tile's
    # rows too far apart for 32-bit copy offsets inside a tile
    far = 2 ** 22 + 8
    assert lib.gemm_relu_gated_plan(300, 300, far, gr.F16) in (b"g64x64x64", b"k16x16x64_s4", b"k32x32x64_s4")
    assert lib.gemm_relu_gated_plan(4000, 4000, 2 ** 30, gr.F16) == b"g64x64x64"


def test_one_token_of_a_long_row_takes_the_smallest_tile():
    lib = gr.library()
    for n, k in itertools.product((64, 1000, 8192), (1000, 8192)):
        assert lib.gemm_relu_gated_plan(1, n, k, gr.BF16) == b"k16x16x64_s4"
        assert lib.gemm_relu_i8_plan(1, n, k, gr.BF16) == b"k16x16x64_s4"


def test_workspace_covers_every_plan():
    # strided rows never need more than dense ones, which the workspace function assumes
    lib = gr.library()
    for m, n, k in itertools.product((1, 34, 320, 4096), (1, 64, 2816), (64, 119, 4096)):
        both = 2 * (m * 2 * n) * 2
        assert lib.gemm_relu_gated_backward_workspace(m, n, k) >= both


def test_a_few_rows_past_a_tile_take_a_launch_of_their_own():
    lib = gr.library()
    assert lib.gemm_relu_gated_plan(1027, 2003, 1501, gr.F16) == b"d128x128x64_s4_i16w8+k16x16x64_s4"
    assert lib.gemm_relu_gated_plan(1024, 2003, 1501, gr.F16) == b"d128x128x64_s4_i16w8"
    assert lib.gemm_relu_i8_plan(1027, 4006, 1501, gr.F16) == b"d128x128x64_s4_i16w8+k16x16x64_s4"
    # no round is saved: 17 x 24 tiles are two rounds, and so are 16 x 24
    assert lib.gemm_relu_gated_plan(4097, 3000, 2000, gr.BF16) == b"d256x256x32_s4_i16w8"
