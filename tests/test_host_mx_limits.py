"""Sizes that the microscaled products refuse before any CUDA call."""

import ctypes

import pytest

UNSUPPORTED = 2


@pytest.fixture(scope="module")
def lib():
    from block_causal_linear_relu_b200 import build
    build.build()
    import block_causal_linear_relu_b200 as sv
    return sv.load()


@pytest.mark.parametrize("fmt", [0, 1])
def test_columns_whose_sum_outlasts_the_waits(lib, fmt):
    # a tile of 2^31 - 32 columns takes seconds, and the warps that wait for it give up after two
    from block_causal_linear_relu_b200 import SvMx

    def call(cols):
        x = SvMx(1 << 20, 1 << 21, None, 1, cols, fmt)
        w = SvMx(1 << 46, 1 << 47, None, 8, cols, fmt)
        return lib.sv_mx_projection(ctypes.byref(x), ctypes.byref(w), 1 << 48, 1 << 49, 256, None)

    for cols in ((1 << 26) + 32, (1 << 31) - 32):
        assert call(cols) == UNSUPPORTED and b"cols" in lib.sv_last_error()
    assert not (call(1 << 26) == UNSUPPORTED and b"cols" in lib.sv_last_error())
