"""The norm in place, and where its scale factor leaves the range of fp32."""

import numpy as np
import pytest
import torch

from oracle import microscale as M

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


@pytest.mark.parametrize("R,C", [(1, 2560), (70, 320), (700, 2592)])
def test_in_place_without_a_residual(sv, R, C):
    x = torch.randn(R, C, generator=torch.Generator("cuda").manual_seed(1), device="cuda").bfloat16()
    w = torch.randn(C, generator=torch.Generator("cuda").manual_seed(2), device="cuda")
    want, h = sv.sv_rmsnorm(x, w)
    assert h is x
    inplace = x.clone()
    y, h = sv.sv_rmsnorm(inplace, w, y=inplace)
    assert y is inplace and torch.equal(y, want)
    assert h is None  # its place holds y
    view = x.clone()  # the same memory through another tensor
    y, h = sv.sv_rmsnorm(view, w, y=view.view(R, C))
    assert h is None and torch.equal(y, want)
    other = torch.empty_like(x)
    y, h = sv.sv_rmsnorm(x, w, y=other)
    assert h is x and y is other and torch.equal(y, want)
