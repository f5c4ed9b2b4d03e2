"""Arguments of the microscaled calls that are right, or wrong, only on a device."""

import pytest
import torch

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def sv():
    if not torch.cuda.is_available():
        pytest.fail("GPU tests need a CUDA device")
    from block_causal_linear_relu_b200 import build
    build.build()
    import block_causal_linear_relu_b200 as m
    m.load()
    return m


@pytest.mark.parametrize("device", ["cuda", torch.device("cuda"), "cuda:0", None])
def test_empty_takes_a_device_without_an_index(sv, device):
    g = torch.full((1,), 0.01, device="cuda")
    x = torch.randn(130, 96, device="cuda")
    out = sv.MxTensor.empty(130, 96, sv.SV_NVFP4, gscale=g, device=device)
    assert out.device == x.device
    assert sv.sv_mx_quantize(x, sv.SV_NVFP4, gscale=g, out=out) is out
    assert torch.equal(out.codes, sv.sv_mx_quantize(x, sv.SV_NVFP4, gscale=g).codes)


def test_columns_past_32_bits_are_refused(sv):
    # a C int would take 2^32 + 32 columns for 32 of them
    x = torch.empty(1, 2**32 + 32, dtype=torch.bfloat16, device="cuda")
    for fmt in (sv.SV_MXFP8, sv.SV_MXFP4):
        with pytest.raises(ValueError):
            sv.sv_mx_quantize(x, fmt)
    with pytest.raises(ValueError):
        sv.sv_rmsnorm(x, torch.empty(2**32 + 32, device="cuda"))
    with pytest.raises(ValueError):
        sv.MxTensor.empty(1, 2**31, sv.SV_MXFP8)


def test_the_widest_rows_are_quantised_whole(sv):
    cols = 2**31 - 32  # the last group of columns ends below 2^31
    x = torch.zeros(1, cols, dtype=torch.bfloat16, device="cuda")
    x[0, -40:] = torch.arange(40, device="cuda").bfloat16() - 20
    x[0, :32] = 1
    q = sv.sv_mx_quantize(x, sv.SV_MXFP4)
    y = sv.sv_mx_dequantize(q)
    small = sv.sv_mx_dequantize(sv.sv_mx_quantize(x[:, -96:].contiguous(), sv.SV_MXFP4))
    assert torch.equal(y[:, -96:], small) and bool((y[0, :32] == 1).all()) and not bool(y[0, 32:-96].any())
