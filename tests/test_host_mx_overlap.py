"""Outputs of the microscaled calls that overlap an input or one another are refused before any CUDA call."""

import ctypes

import pytest

INVALID = 1
MB = 1 << 20


@pytest.fixture(scope="module")
def lib():
    from block_causal_linear_relu_b200 import build
    build.build()
    import block_causal_linear_relu_b200 as sv
    return sv.load()


def mx(codes, scales, rows=128, cols=256):
    from block_causal_linear_relu_b200 import SvMx
    return ctypes.byref(SvMx(codes, scales, None, rows, cols, 0))


def refused(lib, status):
    return status == INVALID and b"overlap" in lib.sv_last_error()


def test_norm(lib):
    n = 4 * 256 * 2  # bytes of a [4, 256] bf16 matrix

    def f(x=MB, res=2 * MB, h=3 * MB, w=4 * MB, y=5 * MB, yq=None):
        return lib.sv_rmsnorm(x, res, h, w, 4, 256, 0, 1e-6, y, yq, None)

    for at in (-n + 16, -512, 512, n - 16):
        assert refused(lib, f(h=MB + at)) and refused(lib, f(h=2 * MB + at))
        assert refused(lib, f(y=MB + at)) and refused(lib, f(y=2 * MB + at)) and refused(lib, f(y=3 * MB + at))
    for at in (-1024 + 16, 512, n - 16):  # the codes and the scales have 1024 bytes each
        assert refused(lib, f(y=None, yq=mx(MB + at, 6 * MB, rows=4)))
        assert refused(lib, f(y=None, yq=mx(7 * MB, 3 * MB + at, rows=4)))
    assert refused(lib, f(y=4 * MB + 1008)) and refused(lib, f(h=4 * MB + 1008))
    assert refused(lib, f(res=None, h=4 * MB + 1008))  # h takes a copy of x
    assert refused(lib, f(y=None, yq=mx(MB, 6 * MB, rows=4)))  # quantised in place: other rows' bytes
    for ok in (dict(), dict(h=MB), dict(h=2 * MB), dict(y=MB), dict(y=2 * MB), dict(h=MB + n), dict(y=MB - n), dict(res=MB),
               dict(y=None, yq=mx(MB + n, MB + n + 1024, rows=4))):
        assert not refused(lib, f(**ok))


def test_quantise_and_values(lib):
    q = lambda x, out: lib.sv_mx_quantize(x, 1, 1, 128, 256, 0, out, None)
    d = lambda m, y: lib.sv_mx_dequantize(m, y, 0, None)
    n = 128 * 256 * 2
    for at in (-128 * 256 + 16, 0, n - 16):
        assert refused(lib, q(MB, mx(MB + at, 4 * MB))) and refused(lib, d(mx(MB + at, 4 * MB), MB))
    for at in (-1024 + 16, 0, n - 16):
        assert refused(lib, q(MB, mx(4 * MB, MB + at))) and refused(lib, d(mx(4 * MB, MB + at), MB))
    assert not refused(lib, q(MB, mx(MB + n, 4 * MB))) and not refused(lib, d(mx(MB + n, 4 * MB), MB))


def test_products(lib):
    ws = (8 * MB, 256)
    y = lambda y: lib.sv_mx_projection(mx(MB, 2 * MB), mx(3 * MB, 4 * MB), y, *ws, None)
    for at in (MB, 2 * MB, 3 * MB, 4 * MB, MB - 128 * 128 * 2 + 16, 4 * MB + 1024 - 16):
        assert refused(lib, y(at))
    assert not refused(lib, y(6 * MB))
    n = 128 * 128 * 2

    def qkv(q=5 * MB, k=6 * MB, v=7 * MB):
        return lib.sv_mx_qkv_projection(mx(MB, 2 * MB), mx(3 * MB, 4 * MB, rows=384), q, k, v, 1, 128, 1, 128, *ws, None)

    for bad in (dict(q=6 * MB), dict(k=7 * MB), dict(v=5 * MB), dict(v=5 * MB + n - 16), dict(q=MB), dict(k=2 * MB), dict(v=3 * MB + 64)):
        assert refused(lib, qkv(**bad))
    assert not refused(lib, qkv()) and not refused(lib, qkv(k=5 * MB + n, v=5 * MB + 2 * n))
