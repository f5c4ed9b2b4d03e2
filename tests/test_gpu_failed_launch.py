"""A launch that the runtime refuses fails its own call and no later one.

The refusal is made on the host: while a blocking stream is being captured, nothing may be launched on the legacy
default stream, and the runtime says so (cudaErrorStreamCaptureImplicit)."""

import ctypes

import pytest
import torch

import oracle

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


def refused(call, sv):
    """Runs `call`, whose launch on the default stream is refused."""
    cu = ctypes.CDLL("libcuda.so.1")
    stream, graph = ctypes.c_void_p(), ctypes.c_void_p()
    assert cu.cuStreamCreate(ctypes.byref(stream), 0) == 0
    assert cu.cuStreamBeginCapture_v2(stream, 2) == 0  # relaxed
    try:
        with pytest.raises(sv.SvError) as err:
            call()
        assert err.value.status == 3  # SV_ERR_CUDA
    finally:
        cu.cuStreamEndCapture(stream, ctypes.byref(graph))
        if graph.value:
            cu.cuGraphDestroy(graph)
        cu.cuStreamDestroy_v2(stream)


def test_a_refused_launch_does_not_fail_the_next_call(sv):
    gen = torch.Generator("cuda").manual_seed(1)
    q, k, v = (torch.randn(1, 2, 200, 32, generator=gen, device="cuda") for _ in range(3))
    x = torch.randn(130, 96, generator=gen, device="cuda")
    out, y = sv.sv_mx_quantize(x, sv.SV_MXFP8), torch.empty_like(x)
    w = torch.ones(96, device="cuda")
    wq = sv.sv_mx_quantize(x[:128].contiguous(), sv.SV_MXFP8)
    p = sv.sv_mx_projection(out, wq)
    ws = sv.make_workspace(sv.SV_OP_LINATTN_FWD, q)
    want = oracle.linattn_fwd(*(t.double().cpu().numpy() for t in (q, k, v)), 1e-6)
    torch.cuda.synchronize()
    for call in (lambda: sv.sv_mx_quantize(x, sv.SV_MXFP8, out=out), lambda: sv.sv_rmsnorm(x, w, y=y),
                 lambda: sv.sv_mx_dequantize(out, y=y), lambda: sv.sv_mx_projection(out, wq, y=p)):
        refused(call, sv)
        o = sv.sv_linattn_fwd(q, k, v, eps=1e-6, ws=ws)  # fp32: asks the runtime for the last error
        torch.cuda.synchronize()
        assert oracle.max_rel_err(o.double().cpu().numpy(), want) < 1e-5
