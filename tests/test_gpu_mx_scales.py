"""Quantisation to NVFP4 with tensor scales outside the range in which fp32 quotients are accurate, with values that
neither saturate nor vanish, and a token's layer inside a graph. Quantisation is exact: no tolerance."""

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


def check(q, x, g):
    rc, rs = M.quantize(x.double().cpu().numpy(), "nvfp4", g)
    assert np.array_equal(q.scales.cpu().numpy(), M.tile_scales(rs, "nvfp4"))
    e = M.elements(M.unpack(q.codes.cpu().numpy(), "nvfp4"), "nvfp4")
    assert np.array_equal(e, M.elements(rc, "nvfp4"))
    return e, rs


@pytest.mark.parametrize("R,C", [(20, 64), (33, 544), (600, 2560)])
@pytest.mark.parametrize("dt", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("g", [1e-36, 2.0**-95, 2.0**-90, 2.0**-89 * 1.25, 2.0**89 * 1.5, 2.0**92, 3e30])
def test_extreme_tensor_scales(sv, g, dt, R, C):
    gen = torch.Generator("cuda").manual_seed(1)
    x = torch.randn(R, C, generator=gen, device="cuda") * torch.exp(2 * torch.randn(R, 1, generator=gen, device="cuda"))
    x[0] = torch.round(x[0] * 4) / 4  # ties
    gt = torch.tensor([g], dtype=torch.float32, device="cuda")
    x = (x.double() * 300 * gt.double()).to(dt)
    e, s = check(sv.sv_mx_quantize(x, sv.SV_NVFP4, gscale=gt), x, float(gt.item()))
    assert np.unique(e).size == 15 and np.unique(s).size > 20  # every element value (zero is one), and many scales


@pytest.mark.parametrize("dt", [torch.bfloat16, torch.float32])
def test_a_tensor_scale_of_zero_gives_zero_elements(sv, dt):
    x = torch.randn(140, 96, generator=torch.Generator("cuda").manual_seed(2), device="cuda").to(dt)
    q = sv.sv_mx_quantize(x, sv.SV_NVFP4, gscale=torch.zeros(1, device="cuda"))
    assert not q.codes.any()
    assert not sv.sv_mx_dequantize(q).any()
    x[3, 5] = float("nan")  # its block is NaN all the same
    v = sv.sv_mx_dequantize(sv.sv_mx_quantize(x, sv.SV_NVFP4, gscale=torch.zeros(1, device="cuda")), torch.float32)
    assert torch.isnan(v[3, :16]).all() and not v[3, 16:].any() and not v[4:].any()


@pytest.mark.parametrize("fmt", ["mxfp8", "nvfp4"])
def test_a_tokens_layer_captured_and_replayed(sv, fmt):
    C, H, D = 256, 4, 64
    f = {"mxfp8": sv.SV_MXFP8, "nvfp4": sv.SV_NVFP4}[fmt]
    gen = torch.Generator("cuda").manual_seed(3)
    rand = lambda *shape: torch.randn(*shape, generator=gen, device="cuda")
    scale = lambda t: sv.sv_mx_global_scale(t) if fmt == "nvfp4" else None
    weight = lambda t: sv.sv_mx_quantize(t, f, gscale=scale(t))
    x, r, w = rand(1, 1, C).bfloat16(), rand(1, 1, C).bfloat16(), rand(C)
    w_qkv, w_o = weight(rand(3 * C, C) / 16), weight(rand(C, C) / 16)
    g = torch.full((1,), 0.01, device="cuda") if fmt == "nvfp4" else None

    def token():
        yq, h = sv.sv_rmsnorm(x, w, residual=r, fmt=f, gscale=g)
        q, k, v = sv.sv_mx_qkv_projection(yq, w_qkv, 1, 1, H, D)
        oq = sv.sv_mx_quantize(v, f, gscale=g)
        return h, q, k, v, sv.sv_mx_projection(oq, w_o)

    token()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = token()
    for _ in range(3):
        x.copy_(rand(1, 1, C).bfloat16())
        graph.replay()
        torch.cuda.synchronize()
        for a, b in zip(out, token()):
            assert torch.equal(a, b)
