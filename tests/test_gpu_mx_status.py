"""The status word of the microscaled products' workspaces: a word that another call has raised does not stop
a product. The word is raised by the host; no wait runs out."""

import pytest
import torch

pytestmark = pytest.mark.gpu

WORD = -0x7FFF9F00  # 0x80006100 as int32: a timeout, raised by the products' copying warp


@pytest.fixture(scope="module")
def sv():
    if not torch.cuda.is_available():
        pytest.fail("GPU tests need a CUDA device")
    from block_causal_linear_relu_b200 import build
    build.build()
    import block_causal_linear_relu_b200 as m
    m.load()
    return m


def operand(sv, rows, cols, seed):
    x = torch.randn(rows, cols, generator=torch.Generator("cuda").manual_seed(seed), device="cuda")
    return sv.sv_mx_quantize(x, sv.SV_MXFP8)


def raise_word(ws):
    ws.view[:4].copy_(torch.tensor([WORD], dtype=torch.int32).view(torch.uint8))


@pytest.mark.parametrize("R,K,F", [(1, 2560, 2560), (300, 1024, 640), (2900, 640, 3336)])  # K split, tiles of a CTA, of a pair
def test_a_raised_word_does_not_stop_a_product(sv, R, K, F):
    xq, wq = operand(sv, R, K, 1), operand(sv, F, K, 2)
    want = sv.sv_mx_projection(xq, wq)
    ws = sv.Workspace(256, want.device)
    raise_word(ws)
    y = sv.sv_mx_projection(xq, wq, y=torch.full_like(want, 7), ws=ws)
    torch.cuda.synchronize()
    assert torch.equal(y, want)
    assert ws.status() == 0x80006100  # still there for the caller to read
    assert ws.status() == 0
