"""Products of the most columns that they take, sums of 2^26 terms; tensor scales and heads past 32 bits.

Operands are zero but for 16384 places at most. In the MX formats they are powers of two, whose sums fp32 holds
exactly, so the result has no tolerance. In NVFP4 they stand for 6 * e4m3(a / 6) in place of a: the sums take 16384
roundings of at most 2^-22 (a step's own and the accumulation's), 2^-8, and bf16 half a step, 2^-9."""

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


@pytest.mark.parametrize("fmt", ["mxfp8", "mxfp4", "nvfp4"])
@pytest.mark.parametrize("R", [2, 200])
def test_the_longest_sums(sv, fmt, R):
    cols, F = 1 << 26, 16
    f = {"mxfp8": sv.SV_MXFP8, "mxfp4": sv.SV_MXFP4, "nvfp4": sv.SV_NVFP4}[fmt]
    g = torch.ones(1, device="cuda") if fmt == "nvfp4" else None
    if R > 2 and fmt == "mxfp8":
        R = 130  # 9 GB of codes
    x = torch.zeros(2, cols, dtype=torch.bfloat16, device="cuda")
    x[0, ::4096] = 1
    x[1, 31::8192] = 2
    x[1, -1] = 4
    two = sv.sv_mx_quantize(x, f, gscale=g)
    xq = sv.MxTensor.empty(R, cols, f, gscale=g)
    xq.codes.zero_(), xq.scales.zero_()
    xq.codes[-2:].copy_(two.codes)
    r = torch.arange(R - 2, R)
    xq.scales[r // 128, :, r % 32, r // 32 % 4] = two.scales[0, :, :2, 0].permute(1, 0, 2)
    w = torch.ones(F, cols, dtype=torch.bfloat16, device="cuda")
    w[1::2] = -1
    wq = sv.sv_mx_quantize(w, f, gscale=g)
    del w, x
    ws = sv.Workspace(256, xq.device)
    y = sv.sv_mx_projection(xq, wq, ws=ws)
    torch.cuda.synchronize()
    assert ws.status() == 0
    one, minus = sv.sv_mx_dequantize(sv.sv_mx_quantize(torch.tensor([[1.0], [-1.0]], device="cuda").repeat(1, 32), f, gscale=g),
                                     torch.float32)[:, 0].tolist()
    v = sv.sv_mx_dequantize(two, torch.float32)
    want = torch.zeros(R, F, dtype=torch.float64, device="cuda")
    for i in range(2):
        total = v[i].double().sum()
        want[R - 2 + i, 0::2], want[R - 2 + i, 1::2] = total * one, total * minus
    if fmt == "nvfp4":
        assert ((y.double() - want).abs() <= (2.0**-8 + 2.0**-9) * want.abs()).all()
    else:
        assert want[-2, 0] == 16384 and want[-1, 0] == 2 * 8192 + 4 and torch.equal(y, want.bfloat16())


def test_tensor_scale_and_heads_past_32_bits(sv):
    # 2.2e9 values: the largest one at either end, and the last rows of a call equal a call on those rows alone
    B, H, N, D, last = 1, 2, 1_100_003, 1024, 131
    x = torch.ones(B, H, N, D, dtype=torch.bfloat16, device="cuda")
    tail = torch.randn(B, H, last, D, generator=torch.Generator("cuda").manual_seed(5), device="cuda").bfloat16()
    x[:, :, -last:] = tail
    for at, value in (((0, 0, 0, 0), 2688.0), ((0, 1, N - 1, D - 1), -5376.0), ((0, 1, N // 2, 3), 8064.0)):
        kept = x[at].item()
        x[at] = value
        assert sv.sv_mx_global_scale(x).item() == abs(value) / 2688
        x[at] = kept
    g = torch.full((1,), 0.002, device="cuda")
    for fmt in (sv.SV_MXFP8, sv.SV_NVFP4):
        gs = g if fmt == sv.SV_NVFP4 else None
        q = sv.sv_mx_quantize(x, fmt, gscale=gs)
        part = sv.sv_mx_quantize(tail, fmt, gscale=gs)
        assert torch.equal(q.codes[-last:], part.codes)
        r, p = torch.arange(N - last, N), torch.arange(last)
        assert torch.equal(q.scales[r // 128, :, r % 32, r // 32 % 4], part.scales[p // 128, :, p % 32, p // 32 % 4])
