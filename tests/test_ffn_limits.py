"""Size limits of the products: refused on the host, before any launch."""
import dense_tiled_gemm_relu_amd as gr

# fake, well-aligned and disjoint addresses: validation inspects, never dereferences
A, B, C, D, E, G, W = (i << 56 for i in range(1, 8))
K_LIMIT = 2 ** 31 - 128


def test_k_whose_last_step_passes_31_bits():
    # a step of 64 (8-bit inputs: 128) elements past the last one must still be counted in 31 bits
    lib = gr.library()
    for k in (K_LIMIT + 1, 2 ** 31 - 63, 2 ** 31 - 1):
        for dt in (gr.F16, gr.F8E4M3):
            assert gr.gemm_relu_status(A, B, C, 1, 1, k, dt, gr.F16, 1, stream=0) == gr.EUNSUPPORTED
            assert gr.gemm_relu_plan(A, B, C, 1, 1, k, dt, gr.F16, 1) == "unsupported"
            assert gr.gemm_relu_noalloc_status(A, B, C, 1, 1, k, dt, gr.F16, 1, stream=0) == gr.EUNSUPPORTED
            assert gr.gemm_relu_ws_status(A, B, C, 1, 1, k, dt, gr.F16, 1, None, 0, stream=0) == gr.EUNSUPPORTED
            assert gr.gemm_relu_status(A, B, C, 0, 1, k, dt, gr.F16, 1, stream=0) == gr.OK      # nothing to do
        assert lib.gemm_relu_gated(A, k, B, k, C, D, 1, 1, k, gr.F16, 0, 0) == gr.EUNSUPPORTED
        assert lib.gemm_relu_gated_plan(1, 1, k, gr.F16) == b"unsupported"
        assert lib.gemm_relu_gated_plan(0, 1, k, gr.F16) == b"none"
    assert gr.gemm_relu_plan(A, B, C, 1, 1, K_LIMIT, gr.F16, gr.F16, 1) == "g64x64x64"
    assert lib.gemm_relu_gated_plan(1, 1, K_LIMIT, gr.F16) == b"g64x64x64"


TILES = {"d256x256x32_s4_i16w8": (256, 256), "d128x128x64_s4_i16w8": (128, 128), "d128x128x64_s2w8": (128, 128),
         "d64x64x64_s4": (64, 64), "g64x64x64": (64, 64), "k16x16x64_s4": (16, 16), "k32x32x64_s4": (32, 32),
         "k32x48x64_s3": (32, 48), "k48x32x64_s3": (48, 32)}


def workgroups(name, m, n):
    bm, bn = TILES[name]
    return -(-m // bm) * -(-n // bn)


def test_both_launches_of_a_product_fit_the_device():
    # a launch of 2^23 workgroups of 512 threads has 2^32 work-items, one more than there may be
    lib = gr.library()
    for rows in (1, 16, 129, 140, 257, 270, 520):
        for n in (2 ** 20, 2 ** 27 - 2, 2 ** 28, 2 ** 29, 2 ** 30 - 2, 2 ** 30):
            for k in (16, 64, 5000):
                for plan, status in (
                        (lib.gemm_relu_i8_plan(rows, n, k, gr.F16),
                         lambda: lib.gemm_relu_i8(A, k, B, C, k, D, E, rows, n, k, gr.F16, 0)),
                        (lib.gemm_relu_gated_plan(rows, n // 2, k, gr.F16),
                         lambda: lib.gemm_relu_gated(A, k, B, k, C, 0, rows, n // 2, k, gr.F16, 0, 0))):
                    parts = plan.decode().split("+")
                    if len(parts) == 2:                  # the first launch has no rows of the second
                        top = rows - rows % TILES[parts[0]][0]
                        assert workgroups(parts[0], top, n) <= 2 ** 22 and workgroups(parts[1], rows - top, n) <= 2 ** 22
                    elif workgroups(parts[0], rows, n) > 2 ** 22:
                        assert status() == gr.EUNSUPPORTED


def test_gradients_too_large_for_a_launch():
    lib = gr.library()

    def backward(rows, hidden, cols):
        return lib.gemm_relu_gated_backward(A, hidden, B, C, cols, D, cols, E, G, rows, hidden, cols, gr.F16, 0, W, 1 << 62, 0)
    # 2^11 x 2^12 tiles of the element-wise gradient: 2^32 work-items
    assert backward(64 << 11, 64 << 12, 8) == gr.EUNSUPPORTED
    # more rows of dx or dweight than the largest tiles cover; a size that would wrap a 64-bit workspace
    for rows, hidden in ((2 ** 30 + 1, 1), (1, 2 ** 29 + 1), (2 ** 31 - 1, 2 ** 30 - 1)):
        assert backward(rows, hidden, 1) == gr.EUNSUPPORTED
        assert lib.gemm_relu_gated_backward_workspace(rows, hidden, 1) == gr.EUNSUPPORTED
    assert lib.gemm_relu_gated_backward_workspace(2 ** 30, 2 ** 29, 1) >= 2 ** 62
