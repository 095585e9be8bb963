"""A plan's name stays what it was when other plans are asked for."""
import ctypes

import dense_tiled_gemm_relu_amd as gr


def test_names_outlive_later_queries():
    lib = ctypes.CDLL(gr.LIB_PATH)
    i64, code = ctypes.c_int64, ctypes.c_int
    kept = []
    for name in ("gemm_relu_gated_plan", "gemm_relu_i8_plan", "gemm_relu_gated_backward_plan"):
        fn = getattr(lib, name)
        fn.argtypes, fn.restype = [i64, i64, i64, code], ctypes.c_void_p
        for sizes in ((1027, 2003, 1501), (2050, 2000, 1003), (64, 64, 64), (4096, 7168, 4096), (1027, 4006, 1501), (130, 70, 63)):
            at = fn(*sizes, gr.F16)
            kept.append((at, ctypes.string_at(at)))
    assert len({text for _, text in kept}) > 6 and any(b"+" in text for _, text in kept)
    assert all(ctypes.string_at(at) == text for at, text in kept)
