"""The microscaled operators on streams: memory that a call on another stream allocates."""

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
    torch.cuda._sleep(1000)  # the tests' own kernels are loaded: loading one waits for those that run
    for dt in (torch.bfloat16, torch.float32, torch.uint8):
        torch.empty(8, device="cuda", dtype=dt).fill_(7).clone()
    return m


def normal(shape, seed, dtype=torch.bfloat16):
    return torch.randn(shape, generator=torch.Generator("cuda").manual_seed(seed), device="cuda").to(dtype)


def buffers(out):
    """The device memory behind a call's outputs: one byte view per allocation."""
    ts = out if isinstance(out, tuple) else (out,)
    return [(t._buf if hasattr(t, "_buf") else t).contiguous().view(torch.uint8) for t in ts]


def calls(sv):
    R, C, H, D = 1536, 640, 5, 64  # outputs of more than 1 MB: a block of memory each
    x, r, w = normal((R, C), 1), normal((R, C), 2), normal((C,), 3, torch.float32)
    xq = sv.sv_mx_quantize(x, sv.SV_MXFP8)
    wq = sv.sv_mx_quantize(normal((3 * H * D, C), 4), sv.SV_MXFP8)
    torch.cuda.synchronize()  # the inputs are there for every stream
    return {
        "norm": lambda s: sv.sv_rmsnorm(x, w, residual=r, stream=s),
        "norm to mxfp8": lambda s: sv.sv_rmsnorm(x, w, residual=r, fmt=sv.SV_MXFP8, stream=s),
        "quantise": lambda s: sv.sv_mx_quantize(x, sv.SV_MXFP8, stream=s),
        "values": lambda s: sv.sv_mx_dequantize(xq, stream=s),
        "tensor scale": lambda s: sv.sv_mx_global_scale(x, stream=s),
        "projection": lambda s: sv.sv_mx_projection(xq, wq, stream=s),
        "qkv projection": lambda s: sv.sv_mx_qkv_projection(xq, wq, 1, R, H, D, stream=s),
    }


@pytest.mark.parametrize("name", ["norm", "norm to mxfp8", "quantise", "values", "tensor scale", "projection", "qkv projection"])
def test_outputs_do_not_take_memory_that_another_stream_still_uses(sv, name):
    call = calls(sv)[name]
    side = torch.cuda.Stream()
    want = [b.clone() for b in buffers(call(None))]
    call(side)
    torch.cuda.synchronize()
    torch.cuda.empty_cache()
    # temporaries of the outputs' sizes, written late by kernels queued on the current stream, and dropped
    temps = [torch.empty_like(b) for b in want for _ in range(3)]
    copies = [torch.empty_like(t) for t in temps]
    torch.cuda._sleep(200_000_000)  # about 0.1 s
    for t, c in zip(temps, copies):
        t.fill_(7)
        c.copy_(t)
    del t, c, temps
    got = call(side)
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(buffers(got), want))
    assert all(bool((c == 7).all()) for c in copies)


@pytest.mark.parametrize("name", ["norm", "quantise", "projection"])
def test_outputs_may_be_dropped_while_the_current_stream_reads_them(sv, name):
    call = calls(sv)[name]
    side = torch.cuda.Stream()
    want = [b.clone() for b in buffers(call(None))]
    call(side)
    torch.cuda.synchronize()
    got = call(side)
    torch.cuda.current_stream().wait_stream(side)
    torch.cuda._sleep(200_000_000)
    copies = [b.clone() for b in buffers(got)]  # read late on the current stream
    del got
    with torch.cuda.stream(side):
        trash = [torch.full_like(b, 3) for b in want for _ in range(2)]  # takes what is free on the side stream
    torch.cuda.synchronize()
    assert len(trash) == 2 * len(want) and all(torch.equal(a, b) for a, b in zip(copies, want))


@pytest.mark.parametrize("name", ["norm to mxfp8", "tensor scale", "qkv projection"])
def test_a_stream_may_be_any_object_with_a_handle(sv, name):
    call = calls(sv)[name]
    want = [b.clone() for b in buffers(call(None))]
    side = torch.cuda.Stream()

    class Handle:
        cuda_stream = side.cuda_stream

    torch.cuda.synchronize()
    got = call(Handle())
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(buffers(got), want))
