"""The binding of the microscaled operators where it needs no GPU: its own checks and fields, on host memory."""

import pytest
import torch


@pytest.fixture(scope="module")
def native():
    from block_causal_linear_relu_b200 import _native
    return _native


def matrix(native, rows=3, cols=64, fmt=None, gscale=None):
    return native.MxTensor._new(rows, cols, native.SV_MXFP8 if fmt is None else fmt, gscale, torch.device("cpu"))


def test_fields_cannot_be_assigned(native):
    # a call reads the descriptor, which would keep the old values and the old tensor scale's address
    g = torch.ones(1)
    m = matrix(native, fmt=native.SV_NVFP4, gscale=g)
    for name, value in (("rows", 5), ("cols", 32), ("fmt", native.SV_MXFP8), ("gscale", torch.zeros(1)), ("device", None),
                        ("codes", None), ("scales", None)):
        with pytest.raises(AttributeError):
            setattr(m, name, value)
    with pytest.raises(AttributeError):
        m.other = 1
    assert (m.rows, m.cols, m.fmt, m.device) == (3, 64, native.SV_NVFP4, torch.device("cpu")) and m.gscale is g
    assert (m._c.rows, m._c.cols, m._c.fmt, m._c.gscale) == (3, 64, native.SV_NVFP4, g.data_ptr())
    assert m.codes.shape == (3, 32) and m.codes.data_ptr() == m._c.codes
    assert m.scales.shape == (1, 4, 32, 4, 4) and m.scales.data_ptr() == m._c.scales


def test_sizes_that_a_c_int_cannot_hold_are_refused(native):
    for cols in (2**31, 2**32 + 32):
        with pytest.raises(ValueError):
            native._mx_check(1, cols, native.SV_MXFP8, None, torch.device("cpu"))
    native._mx_check(1, 2**31 - 32, native.SV_MXFP8, None, torch.device("cpu"))


def test_a_workspace_on_another_device_is_refused(native):
    # a kernel would read and write its status word through a pointer that its device may not reach
    class Elsewhere:
        buf = type("Buffer", (), {"device": torch.device("cuda", 1)})()

    with pytest.raises(ValueError, match="workspace"):
        native._mx_workspace(Elsewhere(), torch.device("cuda", 0), 0, None)
