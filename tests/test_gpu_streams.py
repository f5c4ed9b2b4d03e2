"""Calls on a given stream: the outputs, workspaces and tables that they allocate do not take memory that
kernels queued on the current stream still use."""

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


def calls(sv):
    B, H, N, D, L = 1, 4, 2100, 128, 700  # outputs of 2.1 MB: a block of memory each
    q, k, v = (normal((B, H, N, D), i) for i in range(3))
    S, z = torch.zeros(B, H, D, D, device="cuda"), torch.zeros(B, H, D, device="cuda")
    x, w = normal((B, 3, N, 256), 4), normal((256, 3), 5, torch.float32)
    carry = normal((B, N, 256), 6)
    rows, w_qkv, w_o = normal((B, N, 512), 7), normal((3 * H * D, 512), 8), normal((512, H * D), 9)
    table = sv.sv_rope3d_table(3, 20, 35, D, sv.rope_pairs(D))
    torch.cuda.synchronize()  # the inputs are there for every stream
    return {
        "linattn_fwd": lambda s: sv.sv_linattn_fwd(q, k, v, stream=s),
        "block_causal_attn": lambda s: sv.sv_block_causal_attn(q, k, v, L, stream=s),
        "cache_step": lambda s: sv.sv_cache_step(q, k, v, S, z, commit=False, stream=s),
        "cache_step_noalloc": lambda s: sv.sv_cache_step_noalloc(q, k, v, S, z, commit=False, stream=s),
        "block_causal_attn_rope": lambda s: sv.sv_block_causal_attn_rope(q, k, v, L, table, stream=s),
        "temporal_conv": lambda s: sv.sv_temporal_conv(x, w, 3, stream=s),
        "temporal_conv_step": lambda s: sv.sv_temporal_conv_step(x, w, carry, commit=False, stream=s),
        "qkv_projection": lambda s: sv.sv_qkv_projection(rows, w_qkv, H, D, stream=s),
        "out_projection": lambda s: sv.sv_out_projection(q, w_o, stream=s),
        "rope3d_table": lambda s: sv.sv_rope3d_table(60, 23, 40, D, sv.rope_pairs(D), stream=s).table,
    }


def outputs(out):
    return out if isinstance(out, tuple) else (out,)


@pytest.mark.parametrize("name", ["linattn_fwd", "block_causal_attn", "cache_step", "cache_step_noalloc",
                                  "block_causal_attn_rope", "temporal_conv", "temporal_conv_step", "qkv_projection",
                                  "out_projection", "rope3d_table"])
def test_outputs_do_not_take_memory_that_another_stream_still_uses(sv, name):
    call = calls(sv)[name]
    side = torch.cuda.Stream()
    want = [t.clone() for t in outputs(call(None))]
    call(side)  # the side stream has its workspace
    torch.cuda.synchronize()
    torch.cuda.empty_cache()
    temps = [torch.empty_like(t) for t in want for _ in range(8)]
    copies = [torch.empty_like(t) for t in temps]
    torch.cuda._sleep(200_000_000)  # about 0.1 s
    for t, c in zip(temps, copies):  # written late on the current stream, and dropped
        t.fill_(7)
        c.copy_(t)
    del t, c, temps
    got = call(side)
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(outputs(got), want))
    assert all(bool((c == 7).all()) for c in copies)


def test_a_workspace_does_not_take_memory_that_another_stream_still_uses(sv):
    side = torch.cuda.Stream()
    sv.Workspace(3 << 20, torch.device("cuda:0"), side)
    torch.cuda.synchronize()
    torch.cuda.empty_cache()
    temps = [torch.empty((3 << 20) + 256, dtype=torch.uint8, device="cuda") for _ in range(16)]
    torch.cuda._sleep(200_000_000)
    for t in temps:
        t.fill_(7)
    del t, temps
    ws = sv.Workspace(3 << 20, torch.device("cuda:0"), side)
    torch.cuda.synchronize()
    assert ws.status() == 0 and not bool(ws.view[48:].any())  # zero behind the status and mirror words


@pytest.mark.parametrize("name", ["linattn_fwd", "temporal_conv", "qkv_projection"])
def test_a_stream_may_be_any_object_with_a_handle(sv, name):
    call = calls(sv)[name]
    want = [t.clone() for t in outputs(call(None))]
    side = torch.cuda.Stream()

    class Handle:
        cuda_stream = side.cuda_stream

    torch.cuda.synchronize()
    got = outputs(call(Handle()))
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(got, want))
