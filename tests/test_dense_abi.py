"""Host-side checks of the dense operators (no GPU): shapes of launches and refusals before any."""
import ctypes

import pytest

from token_sparse_long_b200 import _lib


@pytest.fixture(scope="module")
def lib():
    from token_sparse_long_b200 import build
    build.build()
    return _lib.load()


def test_rows_pass_stage_belongs_to_one_group(lib):
    # 8 / G groups of G warps take the rows of w in turn, row i from stage i % stages: only with a
    # whole number of stages per group is a stage always the same group's
    for M in (1, 2):
        for K in range(8, 16385, 8):
            g, s = ctypes.c_int(), ctypes.c_int()
            assert lib.jenga_test_linear_rows_shape(M, K, ctypes.byref(g), ctypes.byref(s)) == 0
            groups = 8 // g.value
            assert g.value in (1, 2, 4, 8) and s.value >= groups and s.value % groups == 0, (M, K, g.value, s.value)
            assert s.value <= 64 and s.value * K * 2 <= 192 * 1024
    assert lib.jenga_test_linear_rows_shape(3, 64, ctypes.byref(g), ctypes.byref(s)) == _lib.EINVAL
