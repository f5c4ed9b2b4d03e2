"""Products whose tensor scales multiply to numbers far outside fp32's range, and results that lie inside it.

Tolerance: that of the products (a rounding of every K step's sum and of the accumulation, (cols / 32 + 8) * 2^-22 of the
sum of magnitudes), the bf16 rounding (2^-8 of the result), two fp32 roundings of the scaling (inside the 8 above), and
half of the smallest bf16 number, 2^-134, with one fp32 subnormal rounding, 2^-150, where results are subnormal."""

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


def operand(sv, rows, cols, seed, size, g):
    """A matrix of elements near `size` with zero rows among them, and the tensor scale g; its values in fp64."""
    x = torch.randn(rows, cols, generator=torch.Generator("cuda").manual_seed(seed), device="cuda") * size
    x[::5] = 0
    q = sv.sv_mx_quantize(x, sv.SV_NVFP4, gscale=torch.ones(1, device="cuda"))
    q = sv.MxTensor(q.codes, q.scales, rows, cols, sv.SV_NVFP4, torch.tensor([g], dtype=torch.float32, device="cuda"))
    c, s = M.unpack(q.codes.cpu().numpy(), "nvfp4"), M.untile_scales(q.scales.cpu().numpy(), rows, cols // 16)
    return q, M.values(c, s, "nvfp4", float(q.gscale.item()))


# (rows, columns, features): K split over a cluster, single CTAs, CTA pairs
@pytest.mark.parametrize("R,K,F", [(3, 1024, 136), (160, 128, 640), (2900, 96, 3336)])
@pytest.mark.parametrize("ga,gb,size", [
    (2.0**-70 * 1.1, 2.0**-62 * 1.3, 1.0),   # 2^-132: results about 2^-130
    (2.0**-75, 2.0**-78, 2600.0),            # 2^-153
    (1e-45, 3e36, 1.0),                      # a subnormal scale
    (2.0**66 * 1.3, 2.0**64 * 1.7, 2.0**-8), # 2^131: results about 2^117, and zeros
    (2.0**90, 2.0**90, 0.0),                 # 2^180 times zeros
    (3e38, 3e38, 0.0),
    (1e30, 1e-30, 1.0),
])
def test_products_of_extreme_tensor_scales(sv, R, K, F, ga, gb, size):
    xq, xv = operand(sv, R, K, 1, size, ga)
    wq, wv = operand(sv, F, K, 2, size, gb)
    y = sv.sv_mx_projection(xq, wq).double().cpu().numpy()
    ref, mag = xv @ wv.T, np.abs(xv) @ np.abs(wv).T
    assert mag.max() < 2.0**127
    tol = (K / 32 + 8) * 2.0**-22 * mag
    assert np.all(np.abs(y - ref) <= tol + 2.0**-8 * (np.abs(ref) + tol) + 2.0**-134 + 2.0**-150)
    assert not y[::5].any() and not y[:, ::5].any()
    if size:
        assert np.abs(y).max() > 0


def test_qkv_of_extreme_tensor_scales(sv):
    B, N, H, D, K = 2, 700, 4, 64, 128
    xq, xv = operand(sv, B * N, K, 3, 2.0**-8, 2.0**66)
    wq, wv = operand(sv, 3 * H * D, K, 4, 2.0**-8, 2.0**65)
    ref, mag = xv @ wv.T, np.abs(xv) @ np.abs(wv).T
    tol = (K / 32 + 8) * 2.0**-22 * mag
    for t, y in enumerate(sv.sv_mx_qkv_projection(xq, wq, B, N, H, D)):
        rows = y.permute(0, 2, 1, 3).reshape(B * N, H * D).double().cpu().numpy()
        r, e = ref[:, t * H * D:(t + 1) * H * D], tol[:, t * H * D:(t + 1) * H * D]
        r = np.maximum(r, 0) if t < 2 else r
        assert np.all(np.abs(rows - r) <= e + 2.0**-8 * (np.abs(r) + e))
