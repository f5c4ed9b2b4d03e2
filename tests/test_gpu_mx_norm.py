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


# Tolerances as for the norm elsewhere: three fp32 roundings, 3 * 2^-24 relative, one bf16 rounding, 2^-8 at most, and
# 1e-40 where a product is subnormal.
@pytest.mark.parametrize("dt", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("R,C", [(1, 32), (5, 2560), (700, 544), (3, 16384)])
@pytest.mark.parametrize("size,eps", [(1e-39, 0.0), (1e-41, 0.0), (1e-36, 0.0), (1.2e38, 1e-6), (6e37, 0.0)])
def test_rows_at_the_ends_of_the_range(sv, dt, R, C, size, eps):
    gen = torch.Generator("cuda").manual_seed(3)
    x = (torch.rand(R, C, generator=gen, device="cuda") * 4 - 2).double() * size
    x[:, 0] = size
    x = x.to(dt)
    w = 1 + torch.rand(C, generator=gen, device="cuda")
    y, _ = sv.sv_rmsnorm(x, w, eps=eps)
    xd = x.double().cpu().numpy()
    with np.errstate(invalid="ignore"):
        ref = M.rms_norm(xd, w.double().cpu().numpy(), float(np.float32(eps)))
    tol = 3.01 * 2.0**-24 + (2.0**-8 if dt == torch.bfloat16 else 0)
    y = y.double().cpu().numpy()
    zero = ~xd.any(axis=1)  # 1e-41 is zero in bf16, and zero rows without an eps are 0 / 0
    assert np.isfinite(ref[~zero]).all() and np.isnan(y[zero]).all() and np.isnan(ref[zero]).all()
    assert np.all(np.abs(y - ref)[~zero] <= tol * np.abs(ref[~zero]) + 1e-40)
    y32, _ = sv.sv_rmsnorm(x.float(), w, eps=eps)
    for name, fmt in (("mxfp8", sv.SV_MXFP8), ("mxfp4", sv.SV_MXFP4), ("nvfp4", sv.SV_NVFP4)):
        g = torch.full((1,), 0.002, device="cuda") if name == "nvfp4" else None
        q, _ = sv.sv_rmsnorm(x, w, eps=eps, fmt=fmt, gscale=g)
        c, s = M.quantize(y32.double().cpu().numpy(), name, float(g.item()) if g is not None else None)
        assert np.array_equal(q.scales.cpu().numpy(), M.tile_scales(s, name))
        assert np.array_equal(M.elements(M.unpack(q.codes.cpu().numpy(), name), name), M.elements(c, name))
