"""Host-side checks of the microscaled entry points that need no GPU: sizes, and arguments that must be
refused before any CUDA call."""

import ctypes

import pytest

INVALID, UNSUPPORTED = 1, 2


@pytest.fixture(scope="module")
def lib():
    from block_causal_linear_relu_b200 import build
    build.build()
    import block_causal_linear_relu_b200 as sv
    return sv.load()


def mx(codes=1 << 20, scales=1 << 20, g=None, rows=128, cols=256, fmt=0):
    from block_causal_linear_relu_b200 import SvMx
    return ctypes.byref(SvMx(codes, scales, g, rows, cols, fmt))


FAKE = ctypes.c_void_p(1 << 20)
G = 1 << 20


def test_sizes(lib):
    assert lib.sv_mx_code_bytes(0, 130, 2592) == 130 * 2592
    assert lib.sv_mx_code_bytes(1, 130, 2592) == lib.sv_mx_code_bytes(2, 130, 2592) == 130 * 1296
    # 130 rows -> 256; 2592 columns -> 21 runs of 128 (e4m3) or 11 runs of 256 (e2m1)
    assert lib.sv_mx_scale_bytes(0, 130, 2592) == 256 * 21 * 4
    assert lib.sv_mx_scale_bytes(1, 130, 2592) == 256 * 11 * 8
    assert lib.sv_mx_scale_bytes(2, 130, 2592) == 256 * 11 * 16
    assert lib.sv_mx_scale_bytes(2, 1, 32) == 128 * 16
    assert lib.sv_mx_code_bytes(0, 1 << 30, 4096) == 1 << 42  # past 32 bits
    for bad in ((0, 0, 64), (0, 1 << 31, 64), (0, 4, 0), (0, 4, 48), (3, 4, 64), (-1, 4, 64)):
        assert lib.sv_mx_code_bytes(*bad) == 0 and lib.sv_mx_scale_bytes(*bad) == 0
        assert lib.sv_last_error()


def test_python_shapes_agree_with_the_library(lib):
    from block_causal_linear_relu_b200 import _native as n
    for fmt in range(3):
        for rows, cols in ((1, 32), (128, 128), (129, 160), (331, 2592)):
            shape = n._mx_scale_shape(rows, cols, fmt)
            size = 1
            for d in shape:
                size *= d
            assert size == lib.sv_mx_scale_bytes(fmt, rows, cols)


def test_descriptor_is_checked(lib):
    f = lib.sv_mx_dequantize
    assert f(None, FAKE, 0, None) == INVALID and b"in is NULL" in lib.sv_last_error()
    assert f(mx(codes=None), FAKE, 0, None) == INVALID
    assert f(mx(codes=(1 << 20) + 8), FAKE, 0, None) == INVALID and b"16-byte" in lib.sv_last_error()
    assert f(mx(scales=(1 << 20) + 4), FAKE, 0, None) == INVALID
    assert f(mx(fmt=2), FAKE, 0, None) == INVALID and b"gscale" in lib.sv_last_error()
    assert f(mx(g=G), FAKE, 0, None) == INVALID
    assert f(mx(fmt=2, g=G + 2), FAKE, 0, None) == INVALID
    assert f(mx(fmt=7), FAKE, 0, None) == UNSUPPORTED
    assert f(mx(rows=0), FAKE, 0, None) == INVALID
    assert f(mx(cols=40), FAKE, 0, None) == UNSUPPORTED
    assert f(mx(), None, 0, None) == INVALID
    assert f(mx(), ctypes.c_void_p((1 << 20) + 8), 0, None) == INVALID
    assert f(mx(), FAKE, 2, None) == UNSUPPORTED


def test_quantize_arguments(lib):
    f = lib.sv_mx_quantize
    assert f(FAKE, 1, 1, 128, 256, 9, mx(), None) == UNSUPPORTED
    assert f(FAKE, 1, 1, 128, 256, 0, None, None) == INVALID
    assert f(FAKE, 0, 1, 128, 256, 0, mx(), None) == INVALID
    assert f(FAKE, 1, 1, 127, 256, 0, mx(), None) == INVALID and b"rows" in lib.sv_last_error()
    assert f(FAKE, 1, 2, 128, 256, 0, mx(), None) == INVALID
    assert f(FAKE, 1, 64, 128, 4, 0, mx(), None) == UNSUPPORTED  # D = 4
    assert f(None, 1, 1, 128, 256, 0, mx(), None) == INVALID
    assert f(ctypes.c_void_p((1 << 20) + 2), 1, 1, 128, 256, 0, mx(), None) == INVALID


def test_global_scale_arguments(lib):
    f = lib.sv_mx_global_scale
    assert f(FAKE, 0, 0, FAKE, None) == INVALID
    assert f(None, 5, 0, FAKE, None) == INVALID
    assert f(FAKE, 5, 0, None, None) == INVALID
    assert f(FAKE, 5, 0, ctypes.c_void_p((1 << 20) + 1), None) == INVALID
    assert f(FAKE, 5, 4, FAKE, None) == UNSUPPORTED


def test_rmsnorm_arguments(lib):
    f = lib.sv_rmsnorm
    other = ctypes.c_void_p(1 << 21)
    assert f(FAKE, None, None, FAKE, 0, 256, 0, 1e-6, other, None, None) == INVALID
    assert f(FAKE, None, None, FAKE, 1 << 31, 256, 0, 1e-6, other, None, None) == INVALID
    assert f(FAKE, None, None, FAKE, 4, 252, 0, 1e-6, other, None, None) == UNSUPPORTED
    assert f(FAKE, None, None, FAKE, 4, 32776, 0, 1e-6, other, None, None) == UNSUPPORTED
    assert f(FAKE, None, None, FAKE, 4, 0, 0, 1e-6, other, None, None) == UNSUPPORTED
    assert f(FAKE, None, None, FAKE, 4, 256, 5, 1e-6, other, None, None) == UNSUPPORTED
    for eps in (-1e-6, float("nan"), float("inf")):
        assert f(FAKE, None, None, FAKE, 4, 256, 0, eps, other, None, None) == INVALID
    assert f(None, None, None, FAKE, 4, 256, 0, 1e-6, other, None, None) == INVALID
    assert f(FAKE, None, None, None, 4, 256, 0, 1e-6, other, None, None) == INVALID
    assert f(FAKE, FAKE, None, FAKE, 4, 256, 0, 1e-6, other, None, None) == INVALID and b"residual" in lib.sv_last_error()
    assert f(FAKE, None, None, FAKE, 4, 256, 0, 1e-6, None, None, None) == INVALID and b"exactly one" in lib.sv_last_error()
    assert f(FAKE, None, None, FAKE, 4, 256, 0, 1e-6, other, mx(rows=4), None) == INVALID
    assert f(FAKE, FAKE, other, FAKE, 4, 256, 0, 1e-6, other, None, None) == INVALID  # y is h
    assert f(FAKE, None, None, FAKE, 4, 256, 0, 1e-6, None, mx(rows=5), None) == INVALID
    assert f(FAKE, None, None, FAKE, 4, 264, 0, 1e-6, None, mx(rows=4, cols=264), None) == UNSUPPORTED
    assert f(ctypes.c_void_p((1 << 20) + 8), None, None, FAKE, 4, 256, 0, 1e-6, other, None, None) == INVALID


def test_product_arguments(lib):
    f = lib.sv_mx_projection
    ws = (FAKE, 256)
    assert f(None, mx(), FAKE, *ws, None) == INVALID
    assert f(mx(), None, FAKE, *ws, None) == INVALID
    assert f(mx(), mx(rows=12), FAKE, *ws, None) == UNSUPPORTED  # 12 output features
    assert f(mx(), mx(fmt=1), FAKE, *ws, None) == INVALID and b"format" in lib.sv_last_error()
    assert f(mx(), mx(cols=512), FAKE, *ws, None) == INVALID and b"columns" in lib.sv_last_error()
    assert f(mx(), mx(), None, *ws, None) == INVALID
    assert f(mx(), mx(), ctypes.c_void_p((1 << 20) + 8), *ws, None) == INVALID
    assert f(mx(), mx(), FAKE, None, 256, None) == INVALID
    assert f(mx(), mx(), FAKE, ctypes.c_void_p((1 << 20) + 16), 256, None) == INVALID
    assert f(mx(), mx(), FAKE, FAKE, 255, None) == INVALID
    g = lib.sv_mx_qkv_projection
    w = mx(rows=384)
    assert g(mx(), w, FAKE, FAKE, FAKE, 1, 128, 1, 96, *ws, None) == UNSUPPORTED
    assert g(mx(), w, FAKE, FAKE, FAKE, 1, 127, 1, 128, *ws, None) == INVALID and b"rows" in lib.sv_last_error()
    assert g(mx(), w, FAKE, FAKE, FAKE, 1, 128, 2, 128, *ws, None) == INVALID
    assert g(mx(), w, FAKE, None, FAKE, 1, 128, 1, 128, *ws, None) == INVALID
    assert g(mx(), w, FAKE, FAKE, FAKE, 0, 128, 1, 128, *ws, None) == INVALID


def test_binding_refuses_host_tensors():
    import torch

    import block_causal_linear_relu_b200 as sv
    x, w = torch.zeros(4, 64), torch.ones(64)
    with pytest.raises(ValueError):
        sv.sv_rmsnorm(x, w)
    with pytest.raises(ValueError):
        sv.sv_mx_quantize(x, sv.SV_MXFP8)
    with pytest.raises(ValueError):
        sv.sv_mx_global_scale(x)
    with pytest.raises(ValueError):
        sv.MxTensor(torch.zeros(4, 64, dtype=torch.uint8), torch.zeros(1, 1, 32, 4, 4, dtype=torch.uint8), 4, 64, sv.SV_MXFP8)
