"""Size limits of the products: refused on the host, before any launch."""
import dense_tiled_gemm_relu_amd as gr

# fake, well-aligned and disjoint addresses: validation inspects, never dereferences
A, B, C, D, E, G, W = (i << 40 for i in range(1, 8))
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
