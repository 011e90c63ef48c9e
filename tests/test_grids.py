"""A shape that would take a grid of 2^32 threads is refused, on the CPU."""
import ctypes

import quantized_linear_layer_amd as qll

PTR = ctypes.c_void_p(0x10000)


def test_f32_gemv_of_more_columns_than_one_grid_holds():
    L = qll.load()
    assert L.qll_sgemm(PTR, PTR, PTR, 1, 1 << 30, 4, PTR, 1 << 62, None) == -2
    assert qll.qll_workspace_bytes(qll.QLL_OP_SGEMM, 1, 1 << 30, 4) == 2 ** 64 - 1
    assert qll.qll_workspace_bytes(qll.QLL_OP_SGEMM, 1, (1 << 30) - 1, 4) < 2 ** 64 - 1
    assert qll.qll_workspace_bytes(qll.QLL_OP_SGEMM, 2, 1 << 30, 4) == 0
