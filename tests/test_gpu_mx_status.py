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


def report_timeout(ws):
    """What a kernel does whose wait runs out: the device's word and its mirror on the host."""
    raise_word(ws)
    ws._mirror_np[0] = WORD
    torch.cuda.synchronize()


def test_a_timeout_is_reported_to_its_own_stream(sv):
    from block_causal_linear_relu_b200 import _native
    xq, wq = operand(sv, 300, 640, 3), operand(sv, 640, 640, 4)
    torch.cuda.synchronize()
    a, b = torch.cuda.Stream(), torch.cuda.Stream()
    want = sv.sv_mx_projection(xq, wq)
    for s in (a, b):
        sv.sv_mx_projection(xq, wq, stream=s)
    torch.cuda.synchronize()
    report_timeout(_native._mx_ws[0, a.cuda_stream])
    for s in (b, None):  # the other streams' products run, and their calls do not take the report
        y = sv.sv_mx_projection(xq, wq, stream=s)
        q, k, v = sv.sv_mx_qkv_projection(xq, operand(sv, 384, 640, 5), 1, 300, 2, 64, stream=s)
        torch.cuda.synchronize()
        assert torch.equal(y, want)
    with torch.cuda.stream(a), pytest.raises(sv.SvError) as err:
        sv.sv_mx_projection(xq, wq)
    assert err.value.status == 4  # SV_ERR_TIMEOUT
    y = sv.sv_mx_projection(xq, wq, stream=a)  # reported once
    torch.cuda.synchronize()
    assert torch.equal(y, want)


def test_a_captured_calls_timeout_is_reported_by_the_next_call(sv):
    from block_causal_linear_relu_b200 import _native
    xq, wq = operand(sv, 300, 640, 6), operand(sv, 640, 640, 7)
    want = sv.sv_mx_projection(xq, wq)
    torch.cuda.synchronize()
    graphs = []
    for _ in range(2):  # both captures use the same word
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, stream=torch.cuda.Stream()):
            y = sv.sv_mx_projection(xq, wq)
        graphs.append((g, y))
    raise_word(_native._mx_ws[0])  # one graph's kernel raises it before the host reads its mirror
    torch.cuda.synchronize()
    for g, y in graphs:
        y.fill_(7)
        torch.cuda.synchronize()
        with torch.cuda.stream(torch.cuda.Stream()):
            g.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(y, want) for _, y in graphs)
    report_timeout(_native._mx_ws[0])
    with pytest.raises(sv.SvError):
        sv.sv_mx_projection(xq, wq)
    assert torch.equal(sv.sv_mx_projection(xq, wq), want)


def test_a_call_on_a_capturing_stream_makes_no_workspace(sv):
    from block_causal_linear_relu_b200 import _native
    xq, wq = operand(sv, 16, 64, 8), operand(sv, 16, 64, 9)
    sv.sv_mx_projection(xq, wq)
    torch.cuda.synchronize()
    kept = dict(_native._mx_ws)
    _native._mx_ws.clear()
    try:  # the capture is on the call's stream, which is not the current one
        side, graph = torch.cuda.Stream(), torch.cuda.CUDAGraph()
        y = torch.empty(16, 16, dtype=torch.bfloat16, device="cuda")
        with torch.cuda.stream(side):
            graph.capture_begin(capture_error_mode="relaxed")
        try:
            with pytest.raises(RuntimeError, match="before a capture"):
                sv.sv_mx_projection(xq, wq, y=y, stream=side)
        finally:
            with torch.cuda.stream(side):
                graph.capture_end()
        assert not _native._mx_ws
    finally:
        _native._mx_ws.update(kept)


def test_threads_that_make_the_first_call_share_one_workspace(sv):
    import threading

    from block_causal_linear_relu_b200 import _native
    xq, wq = operand(sv, 300, 640, 10), operand(sv, 640, 640, 11)
    want = sv.sv_mx_projection(xq, wq)
    torch.cuda.synchronize()
    kept = dict(_native._mx_ws)
    _native._mx_ws.clear()
    made, start, ys = [], threading.Barrier(4), [None] * 4
    real = _native.Workspace

    class Counted(real):
        def __init__(self, *args):
            made.append(self)
            super().__init__(*args)

    def first(i):
        start.wait()
        ys[i] = sv.sv_mx_projection(xq, wq)

    try:
        _native.Workspace = Counted
        threads = [threading.Thread(target=first, args=(i,)) for i in range(4)]
        for t in threads:
            t.start()
        for t in threads:
            t.join()
        torch.cuda.synchronize()
        assert all(torch.equal(y, want) for y in ys)
        assert len(made) == 2 and set(made) == set(_native._mx_ws.values())
    finally:
        _native.Workspace = real
        _native._mx_ws.update(kept)
