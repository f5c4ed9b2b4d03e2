"""GPU parity of the microscaled operators (quantisation, values, tensor scale, norm, products) against
the fp64 oracle (oracle/microscale.py), through the C ABI.

Tolerances. Quantisation is exact: the scales and element values of the oracle, bit for bit. The norm
in fp32 rounds three times (1 / sqrt, and two products): 3 * 2^-24 relative, and a bf16 output once more,
2^-8 at most. A product sums exact products of the operands' values in fp32: every K step of at least 32
columns adds one rounded sum to the accumulator, so its error is at most (cols / 32 + 8) * 2^-22 of the sum of
magnitudes (a step's own sum and the accumulation may each truncate), and the bf16 rounding adds 2^-8 of
the result.
"""

import numpy as np
import pytest
import torch

from oracle import microscale as M

pytestmark = pytest.mark.gpu

FMTS = ["mxfp8", "mxfp4", "nvfp4"]
DT = {"bf16": torch.bfloat16, "f32": torch.float32}


@pytest.fixture(scope="module")
def sv():
    if not torch.cuda.is_available():
        pytest.fail("GPU tests need a CUDA device")
    from block_causal_linear_relu_b200 import build
    build.build()
    import block_causal_linear_relu_b200 as m
    m.load()
    return m


def fid(sv, fmt):
    return {"mxfp8": sv.SV_MXFP8, "mxfp4": sv.SV_MXFP4, "nvfp4": sv.SV_NVFP4}[fmt]


def f64(t):
    return t.double().cpu().numpy()


def make(shape, dt, seed, scale=1.0, odd=True):
    """Values of both signs over a wide range, with the blocks that quantisation can get wrong."""
    rng = np.random.default_rng(seed)
    x = rng.standard_normal(shape).astype(np.float32) * scale
    x *= np.exp(rng.standard_normal(shape[:-1] + (1,))).astype(np.float32)
    r = x.reshape(-1, shape[-1])
    if odd:
        r[0] = np.round(r[0] * 4) / 4                        # exact ties
        if r.shape[0] > 8:
            r[1, :32] = 0                                     # an empty block
            r[2, 3], r[3, 5], r[4, 7] = np.inf, np.nan, -np.inf
            r[5] *= 1e-30
            r[6] *= 1e30
            r[7] *= 1e-42                                     # subnormal
            r[8] = -0.0
    return torch.from_numpy(x).to(DT[dt]).cuda()


def scale_for(sv, fmt, value=None):
    if fmt != "nvfp4":
        return None
    return torch.tensor([0.0123 if value is None else value], device="cuda")


def read(xq, fmt):
    """(element values, scale bytes, matrix values) of an MxTensor."""
    c = M.unpack(xq.codes.cpu().numpy(), fmt)
    s = M.untile_scales(xq.scales.cpu().numpy(), xq.rows, xq.cols // M.BLOCK[fmt])
    g = float(xq.gscale.item()) if fmt == "nvfp4" else None
    return M.elements(c, fmt), s, M.values(c, s, fmt, g)


def same(a, b):
    return np.array_equal(a, b, equal_nan=True)


@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("dt", ["bf16", "f32"])
@pytest.mark.parametrize("R,C", [(1, 32), (9, 64), (128, 128), (129, 160), (331, 2592), (40, 256 * 5 + 32)])
def test_quantize_is_exact(sv, fmt, dt, R, C):
    x = make((R, C), dt, R + C)
    g = scale_for(sv, fmt)
    xq = sv.sv_mx_quantize(x, fid(sv, fmt), gscale=g)
    torch.cuda.synchronize()
    e, s, v = read(xq, fmt)
    rc, rs = M.quantize(f64(x), fmt, float(g.item()) if g is not None else None)
    assert np.array_equal(s, rs)
    assert same(e, M.elements(rc, fmt))
    # the places of the tiles without a block are zero
    assert np.array_equal(xq.scales.cpu().numpy(), M.tile_scales(rs, fmt))
    for t in DT.values():
        y = sv.sv_mx_dequantize(xq, t)
        assert same(y.float().cpu().numpy(), torch.from_numpy(v).float().to(t).float().numpy())


@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("B,H,N,D", [(1, 20, 3, 128), (2, 4, 77, 8), (3, 2, 130, 112), (1, 4, 5, 24), (2, 3, 33, 32)])
def test_quantize_heads(sv, fmt, B, H, N, D):
    x = make((B, H, N, D), "bf16", 5, odd=False)
    g = scale_for(sv, fmt)
    xq = sv.sv_mx_quantize(x, fid(sv, fmt), gscale=g)
    e, s, _ = read(xq, fmt)
    rc, rs = M.quantize(M.heads_to_rows(f64(x)), fmt, float(g.item()) if g is not None else None)
    assert np.array_equal(s, rs) and same(e, M.elements(rc, fmt))


@pytest.mark.parametrize("g", [1e-36, 2.0**-10, 1.0, 3.0e30, 0.0, float("inf"), float("nan")])
def test_nvfp4_tensor_scales(sv, g):
    x = make((20, 64), "f32", 6, odd=False)
    gt = torch.tensor([g], device="cuda")
    xq = sv.sv_mx_quantize(x, sv.SV_NVFP4, gscale=gt)
    _, s, v = read(xq, "nvfp4")
    if g == 0.0:
        assert same(v, np.zeros_like(v))
        return
    g32 = float(gt.item())
    rc, rs = M.quantize(f64(x), "nvfp4", g32)
    assert np.array_equal(s, rs) and same(v, M.values(rc, rs, "nvfp4", g32))


def test_nvfp4_borders_of_a_measured_scale(sv):
    # bf16 values and g = amax / 2688 lie on borders between elements in exact arithmetic or one rounding off
    x = make((512, 512), "bf16", 7, odd=False)
    g = sv.sv_mx_global_scale(x)
    assert float(g.item()) == float(np.float32(f64(x.abs().max())) / np.float32(2688))
    e, s, _ = read(sv.sv_mx_quantize(x, sv.SV_NVFP4, gscale=g), "nvfp4")
    rc, rs = M.quantize(f64(x), "nvfp4", float(g.item()))
    assert np.array_equal(s, rs) and same(e, M.elements(rc, "nvfp4"))


@pytest.mark.parametrize("dt", ["bf16", "f32"])
def test_nvfp4_tensor_scales_next_to_nice_numbers(sv, dt):
    # s * g a few last places from a number whose borders are bf16 values: on, just below and just above ties
    x = make((24, 256), dt, 50, odd=False)
    for base in (1.0, 0.0625, 1.0 / 3.0, 5.0 / 7.0, 1.9921875):
        for k in range(-9, 10):
            g = torch.tensor([base], dtype=torch.float32).view(torch.int32).add(k).view(torch.float32).cuda()
            e, s, _ = read(sv.sv_mx_quantize(x, sv.SV_NVFP4, gscale=g), "nvfp4")
            rc, rs = M.quantize(f64(x), "nvfp4", float(g.item()))
            assert np.array_equal(s, rs) and same(e, M.elements(rc, "nvfp4")), (base, k)


@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("heads", [False, True])
def test_large_inputs_equal_their_slices(sv, fmt, heads):
    # 11 million values: the kernels chosen for large inputs, against small calls on slices
    B, H, N, D = (3, 20, 1411, 128) if heads else (1, 1, 4233, 2560)
    g = scale_for(sv, fmt)
    x = make((B, H, N, D), "bf16", 51, odd=False)
    big = sv.sv_mx_quantize(x if heads else x.view(N, D), fid(sv, fmt), gscale=g)
    values = sv.sv_mx_dequantize(big)
    R = B * N
    codes, scales = big.codes, M.untile_scales(big.scales.cpu().numpy(), R, H * D // M.BLOCK[fmt])
    for b in range(B):
        for n0 in (0, 640, N - 300):
            part = x[b:b + 1, :, n0:n0 + 300].contiguous()
            q = sv.sv_mx_quantize(part if heads else part.view(300, D), fid(sv, fmt), gscale=g)
            at = slice(b * N + n0, b * N + n0 + 300)
            assert torch.equal(q.codes, codes[at])
            assert np.array_equal(M.untile_scales(q.scales.cpu().numpy(), 300, H * D // M.BLOCK[fmt]), scales[at])
            assert torch.equal(sv.sv_mx_dequantize(q), values[at])
    pad = big.scales.cpu().numpy().copy()
    pad[np.arange(R)[:, None] // 128, np.arange(scales.shape[1]) // 4, np.arange(R)[:, None] % 32,
        np.arange(R)[:, None] // 32 % 4, np.arange(scales.shape[1]) % 4] = 0
    assert not pad.any()


def test_offsets_past_32_bits(sv):
    # 2.2e9 values: the last rows of one call equal a call on those rows alone
    R, C, last = 68001, 32768, 257
    x = torch.empty(R, C, dtype=torch.bfloat16, device="cuda")
    x[:-last] = 1.0
    x[-last:] = make((last, C), "bf16", 52, odd=False)
    tail = x[-last:].clone()
    q, t = sv.sv_mx_quantize(x, sv.SV_MXFP8), sv.sv_mx_quantize(tail, sv.SV_MXFP8)
    assert torch.equal(q.codes[-last:], t.codes)
    v = sv.sv_mx_dequantize(q)
    assert torch.equal(v[-last:], sv.sv_mx_dequantize(t)) and (v[:3] == 1).all()
    del v
    w = make((C,), "f32", 53, odd=False)
    y, h = sv.sv_rmsnorm(x, w, residual=x)
    y2, h2 = sv.sv_rmsnorm(tail, w, residual=tail)
    assert torch.equal(y[-last:], y2) and torch.equal(h[-last:], h2)
    del y, h, q, x
    R, C, F = 300001, 32, 8192
    xq, _ = operand(sv, R, C, "mxfp4", 54)
    wq, _ = operand(sv, F, C, "mxfp4", 55)
    y = sv.sv_mx_projection(xq, wq)  # 2.5e9 outputs
    xv = sv.sv_mx_dequantize(xq, torch.float32)
    tail = sv.sv_mx_quantize(xv[-257:].contiguous(), sv.SV_MXFP4)  # already representable: the same operand
    assert torch.equal(y[-257:], sv.sv_mx_projection(tail, wq))


@pytest.mark.parametrize("dt", ["bf16", "f32"])
@pytest.mark.parametrize("n", [1, 7, 8, 2049, 100003, 700001])
def test_global_scale(sv, dt, n):
    x = make((n,), dt, n, odd=False)
    assert float(sv.sv_mx_global_scale(x).item()) == float(np.float32(f64(x.abs().max())) / np.float32(2688))
    x[-1] = float("nan")
    assert np.isnan(sv.sv_mx_global_scale(x).item())
    x.zero_()
    assert sv.sv_mx_global_scale(x).item() == 0.0


# ---- norm ----

NORM = [(1, 32), (1, 2560), (3, 8), (130, 104), (257, 2592), (5, 520), (9, 1024), (11, 5120), (7, 16384), (2, 32768),
        (700, 264), (601, 2592), (650, 5120), (600, 8192)]  # many rows: two groups of columns per thread


@pytest.mark.parametrize("dt", ["bf16", "f32"])
@pytest.mark.parametrize("res", [True, False])
@pytest.mark.parametrize("R,C", NORM)
def test_rmsnorm(sv, dt, res, R, C):
    x, r = make((R, C), dt, 1, odd=False), make((R, C), dt, 2, odd=False) if res else None
    w = make((C,), "f32", 3, odd=False)
    y, h = sv.sv_rmsnorm(x, w, residual=r, eps=1e-5)
    rh = x if r is None else (x.float() + r.float()).to(x.dtype)
    assert torch.equal(h, rh)
    ref = M.rms_norm(f64(rh), f64(w), float(np.float32(1e-5)))
    tol = 3.01 * 2.0**-24 + (2.0**-8 if dt == "bf16" else 0)
    assert np.all(np.abs(f64(y) - ref) <= tol * np.abs(ref) + 1e-40)


@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("dt", ["bf16", "f32"])
@pytest.mark.parametrize("R,C", [(1, 32), (1, 2560), (130, 96), (257, 2592), (5, 544), (9, 1024), (11, 5120), (300, 7680), (3, 32768),
                                 (700, 544), (601, 2592), (600, 8224)])
def test_rmsnorm_quantised(sv, fmt, dt, R, C):
    x, r = make((R, C), dt, 4, odd=False), make((R, C), dt, 5, odd=False)
    w = make((C,), "f32", 6, odd=False)
    g = scale_for(sv, fmt, 0.02)
    yq, h = sv.sv_rmsnorm(x, w, residual=r, fmt=fid(sv, fmt), gscale=g)
    # what the unquantised fp32 norm of the stored h gives, quantised apart: the same bits
    y32, _ = sv.sv_rmsnorm(h.float(), w)
    e, s, v = read(yq, fmt)
    rc, rs = M.quantize(f64(y32), fmt, float(g.item()) if g is not None else None)
    assert np.array_equal(yq.scales.cpu().numpy(), M.tile_scales(rs, fmt))
    assert same(e, M.elements(rc, fmt))
    ref = M.rms_norm(f64(h), f64(w), float(np.float32(1e-6)))
    assert np.all(np.abs(f64(y32) - ref) <= 3.01 * 2.0**-24 * np.abs(ref) + 1e-40)


def test_rmsnorm_rows_with_nan_and_infinity(sv):
    x = make((6, 256), "bf16", 8, odd=False)
    x[1, 9], x[2, 200], x[3] = float("nan"), float("inf"), 0.0
    w = torch.ones(256, device="cuda")
    y, _ = sv.sv_rmsnorm(x, w)
    # an infinity makes its row's 1 / rms zero: inf * 0 is NaN there, the row's other values are zero
    assert torch.isnan(y[1]).all() and torch.isnan(y[2, 200]) and (y[2, :200] == 0).all() and (y[3] == 0).all()
    assert torch.isfinite(y[[0, 3, 4, 5]].float()).all()
    for fmt in FMTS:
        yq, _ = sv.sv_rmsnorm(x, w, fmt=fid(sv, fmt), gscale=scale_for(sv, fmt))
        v = sv.sv_mx_dequantize(yq, torch.float32)
        b = M.BLOCK[fmt]
        assert torch.isnan(v[1]).all() and torch.isnan(v[2, 200 // b * b:(200 // b + 1) * b]).all()
        assert (v[2, :200 // b * b] == 0).all() and torch.isfinite(v[[0, 3, 4, 5]]).all()


def test_rmsnorm_in_place_and_into_given_outputs(sv):
    x, r = make((70, 320), "bf16", 9, odd=False), make((70, 320), "bf16", 10, odd=False)
    w = make((320,), "f32", 11, odd=False)
    y0, h0 = sv.sv_rmsnorm(x, w, residual=r)
    for place in ("x", "residual"):
        x1, r1 = x.clone(), r.clone()
        y1, h1 = sv.sv_rmsnorm(x1, w, residual=r1, h=x1 if place == "x" else r1)
        assert h1 is (x1 if place == "x" else r1) and torch.equal(h1, h0) and torch.equal(y1, y0)
        assert torch.equal(r1 if place == "x" else x1, r if place == "x" else x)
    x2 = x.clone()
    y2, h2 = sv.sv_rmsnorm(x2, w, residual=r, y=x2)
    assert torch.equal(y2, y0) and torch.equal(h2, h0) and y2 is x2
    out = sv.MxTensor.empty(70, 320, sv.SV_MXFP8, device=x.device)
    y3, _ = sv.sv_rmsnorm(x, w, residual=r, fmt=sv.SV_MXFP8, y=out)
    y4, _ = sv.sv_rmsnorm(x, w, residual=r, fmt=sv.SV_MXFP8)
    assert y3 is out and torch.equal(y3.codes, y4.codes) and torch.equal(y3.scales, y4.scales)


# ---- products ----


def operand(sv, rows, cols, fmt, seed, scale=1.0):
    x = make((rows, cols), "f32", seed, scale, odd=False)
    g = sv.sv_mx_global_scale(x) if fmt == "nvfp4" else None
    q = sv.sv_mx_quantize(x, fid(sv, fmt), gscale=g)
    return q, read(q, fmt)[2]


def check_product(y, xv, wv, cols, relu=False):
    ref, mag = xv @ wv.T, np.abs(xv) @ np.abs(wv).T
    tol = (cols / 32 + 8) * 2.0**-22 * mag
    if relu:
        ref = np.maximum(ref, 0)
    err = np.abs(f64(y) - ref)
    assert np.all(err <= tol + 2.0**-8 * (np.abs(ref) + tol)), float(np.max(err - tol - 2.0**-8 * np.abs(ref)))


SIZES = [(1, 32, 8), (1, 2560, 2560), (5, 64, 16), (128, 128, 128), (127, 256, 136), (129, 288, 264), (300, 1024, 640),
         (333, 2592, 200), (16, 10240, 96), (700, 96, 1000), (2, 5120, 7680)]


@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("R,C,F", SIZES)
def test_projection(sv, fmt, R, C, F):
    xq, xv = operand(sv, R, C, fmt, 21)
    wq, wv = operand(sv, F, C, fmt, 22, C**-0.5)
    y = sv.sv_mx_projection(xq, wq)
    torch.cuda.synchronize()
    check_product(y, xv, wv, C)


@pytest.mark.parametrize("fmt", FMTS)
def test_projection_over_many_tiles_per_block(sv, fmt):
    # more tiles than SMs: both accumulators and the stage ring wrap around several times
    xq, xv = operand(sv, 2900, 640, fmt, 23)
    wq, wv = operand(sv, 3336, 640, fmt, 24, 0.04)
    y = sv.sv_mx_projection(xq, wq)
    check_product(y, xv, wv, 640)
    assert torch.equal(y, sv.sv_mx_projection(xq, wq))


@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("R,C,F", [(18900, 64, 128), (18900, 96, 192), (18900, 64, 256), (18700, 320, 248), (9400, 576, 376)])
def test_projection_column_tiles(sv, fmt, R, C, F):
    # one wave of 256-row tiles: each width of the column tile is the best one for some of these
    xq, xv = operand(sv, R, C, fmt, 70)
    wq, wv = operand(sv, F, C, fmt, 71, C**-0.5)
    check_product(sv.sv_mx_projection(xq, wq), xv, wv, C)


@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("B,N,C,H,D", [(700, 3, 96, 20, 64), (90, 33, 64, 20, 128), (9, 300, 128, 24, 64), (1, 5000, 64, 4, 128)])
def test_qkv_projection_of_many_short_batches(sv, fmt, B, N, C, H, D):
    # rows of several batches in the 32 rows of one store
    xq, xv = operand(sv, B * N, C, fmt, 72)
    wq, wv = operand(sv, 3 * H * D, C, fmt, 73, C**-0.5)
    for t, y in enumerate(sv.sv_mx_qkv_projection(xq, wq, B, N, H, D)):
        rows = y.permute(0, 2, 1, 3).reshape(B * N, H * D)
        check_product(rows, xv, wv[t * H * D:(t + 1) * H * D], C, relu=t < 2)


@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("B,N,C,H,D", [(1, 1, 64, 1, 64), (2, 77, 256, 2, 128), (3, 130, 288, 5, 64), (5, 3, 160, 3, 128),
                                       (1, 1000, 2560, 20, 128)])
def test_qkv_projection(sv, fmt, B, N, C, H, D):
    xq, xv = operand(sv, B * N, C, fmt, 25)
    wq, wv = operand(sv, 3 * H * D, C, fmt, 26, C**-0.5)
    qkv = sv.sv_mx_qkv_projection(xq, wq, B, N, H, D)
    for t, y in enumerate(qkv):
        assert y.shape == (B, H, N, D)
        rows = y.permute(0, 2, 1, 3).reshape(B * N, H * D)
        check_product(rows, xv, wv[t * H * D:(t + 1) * H * D], C, relu=t < 2)
        if t < 2:
            assert (y >= 0).all()


@pytest.mark.parametrize("fmt", FMTS)
def test_one_elements_find_their_place(sv, fmt):
    # a single one in row r, column c of X picks column c of W: every code and scale position is hit
    C, F = 512, 128
    w = torch.randint(1, 4, (F, C), device="cuda").float() * torch.exp2(torch.randint(-3, 4, (F, C // 32), device="cuda").float()).repeat_interleave(32, 1)
    g = torch.ones(1, device="cuda") if fmt == "nvfp4" else None
    wq = sv.sv_mx_quantize(w, fid(sv, fmt), gscale=g)
    wv = sv.sv_mx_dequantize(wq, torch.float32)
    x = torch.eye(C, device="cuda") * torch.exp2((torch.arange(C, device="cuda") % 5).float() - 2)[:, None]
    xq = sv.sv_mx_quantize(x, fid(sv, fmt), gscale=g)
    y = sv.sv_mx_projection(xq, wq)
    assert torch.equal(y.float(), (sv.sv_mx_dequantize(xq, torch.float32).double() @ wv.double().T).float().bfloat16().float())


@pytest.mark.parametrize("fmt", FMTS)
def test_nan_blocks_stay_in_their_rows(sv, fmt):
    x = make((200, 320), "f32", 27, odd=False)
    x[3, 40], x[150, 319] = float("nan"), float("inf")
    g = scale_for(sv, fmt)
    xq = sv.sv_mx_quantize(x, fid(sv, fmt), gscale=g)
    wq, _ = operand(sv, 256, 320, fmt, 28)
    y = sv.sv_mx_projection(xq, wq)
    bad = torch.zeros(200, dtype=torch.bool, device="cuda")
    bad[3] = bad[150] = True
    assert torch.isnan(y[bad]).all() and torch.isfinite(y[~bad].float()).all()
    q, k, v = sv.sv_mx_qkv_projection(xq, operand(sv, 384, 320, fmt, 29)[0], 1, 200, 2, 64)
    for t in (q, k, v):  # ReLU keeps a NaN
        assert torch.isnan(t[0, :, bad]).all() and torch.isfinite(t[0, :, ~bad].float()).all()


@pytest.mark.parametrize("fmt", FMTS)
def test_layer_in_microscaled_operands(sv, fmt):
    # residual + norm -> Q/K/V -> linear attention -> heads quantised -> output projection, stage by stage
    # against the oracle fed with the GPU's own intermediate values
    import oracle

    B, N, H, D = 2, 333, 4, 64
    C = H * D
    x, r = make((B, N, C), "bf16", 30, odd=False), make((B, N, C), "bf16", 31, odd=False)
    w = make((C,), "f32", 32, odd=False)
    wqkv, wqkv_v = operand(sv, 3 * C, C, fmt, 33, C**-0.5)
    wo, wo_v = operand(sv, C, C, fmt, 34, C**-0.5)
    g = scale_for(sv, fmt, 0.01)
    yq, h = sv.sv_rmsnorm(x, w, residual=r, fmt=fid(sv, fmt), gscale=g)
    q, k, v = sv.sv_mx_qkv_projection(yq, wqkv, B, N, H, D)
    o = sv.sv_linattn_fwd(q, k, v, eps=1e-6)
    oq = sv.sv_mx_quantize(o, fid(sv, fmt), gscale=sv.sv_mx_global_scale(o) if fmt == "nvfp4" else None)
    y = sv.sv_mx_projection(oq, wo, y=torch.empty(B, N, C, dtype=torch.bfloat16, device="cuda"))
    torch.cuda.synchronize()
    xv = read(yq, fmt)[2]
    for t, got in enumerate((q, k, v)):
        check_product(got.permute(0, 2, 1, 3).reshape(B * N, C), xv, wqkv_v[t * C:(t + 1) * C], C, relu=t < 2)
    assert oracle.max_rel_err(f64(o), oracle.linattn_fwd(f64(q), f64(k), f64(v), 1e-6)) < 2e-2
    check_product(y.reshape(B * N, C), read(oq, fmt)[2], wo_v, C)


def test_captured_and_replayed(sv):
    x, r = make((1, 300, 256), "bf16", 35, odd=False), make((1, 300, 256), "bf16", 36, odd=False)
    w = make((256,), "f32", 37, odd=False)
    wq, _ = operand(sv, 384, 256, "nvfp4", 38)
    g = scale_for(sv, "nvfp4")

    def layer():
        yq, h = sv.sv_rmsnorm(x, w, residual=r, fmt=sv.SV_NVFP4, gscale=g)
        q, k, v = sv.sv_mx_qkv_projection(yq, wq, 1, 300, 2, 64)
        return (h, q, k, v, sv.sv_mx_global_scale(q))

    layer()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = layer()
    for seed in (39, 40):
        x.copy_(make((1, 300, 256), "bf16", seed, odd=False))
        graph.replay()
        torch.cuda.synchronize()
        for a, b in zip(out, layer()):
            assert torch.equal(a, b)


def test_captured_weight_conversion(sv):
    # the two launches of a large tensor scale are replayed, also when the new maximum is smaller
    x = make((600, 2560), "f32", 62, odd=False)
    sv.sv_mx_quantize(x, sv.SV_NVFP4, gscale=sv.sv_mx_global_scale(x))
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        g = sv.sv_mx_global_scale(x)
        q = sv.sv_mx_quantize(x, sv.SV_NVFP4, gscale=g)
        y = sv.sv_mx_dequantize(q)
    for factor in (1.0, 0.01, 3.0):
        x.copy_(make((600, 2560), "f32", 63, factor, odd=False))
        graph.replay()
        torch.cuda.synchronize()
        g2 = sv.sv_mx_global_scale(x)
        assert torch.equal(g, g2)
        q2 = sv.sv_mx_quantize(x, sv.SV_NVFP4, gscale=g2)
        assert torch.equal(q.codes, q2.codes) and torch.equal(q.scales, q2.scales)
        assert torch.equal(y, sv.sv_mx_dequantize(q2))


def test_slices_of_whole_row_tiles(sv):
    # 128 rows are one tile of scales: a matrix can be cut there without a copy
    for fmt in FMTS:
        xq, xv = operand(sv, 384, 320, fmt, 64)
        wq, wv = operand(sv, 256, 320, fmt, 65)
        part = sv.MxTensor(xq.codes[128:256], xq.scales[1:2], 128, 320, xq.fmt, xq.gscale)
        half = sv.MxTensor(wq.codes[128:], wq.scales[1:], 128, 320, wq.fmt, wq.gscale)
        y = sv.sv_mx_projection(part, half)
        check_product(y, xv[128:256], wv[128:], 320)
        assert same(f64(sv.sv_mx_dequantize(part, torch.float32)), np.float32(xv[128:256]).astype(np.float64))


def test_first_call_inside_a_capture_is_refused(sv):
    from block_causal_linear_relu_b200 import _native
    xq, _ = operand(sv, 16, 64, "mxfp8", 60)
    wq, _ = operand(sv, 16, 64, "mxfp8", 61)
    sv.sv_mx_projection(xq, wq)
    torch.cuda.synchronize()
    kept = dict(_native._mx_ws)
    _native._mx_ws.clear()
    try:
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph), pytest.raises(RuntimeError):
            sv.sv_mx_projection(xq, wq)
    finally:
        _native._mx_ws.update(kept)
    y = torch.empty(16, 16, dtype=torch.bfloat16, device="cuda")
    ws = sv.Workspace(256, y.device)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        sv.sv_mx_projection(xq, wq, y=y, ws=ws)
    y.zero_()
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(y, sv.sv_mx_projection(xq, wq))


def test_two_streams_at_once(sv):
    wq, wv = operand(sv, 512, 512, "mxfp8", 41)
    xs = [operand(sv, 3000, 512, "mxfp8", 42 + i) for i in range(2)]
    sv.sv_mx_projection(xs[0][0], wq)
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in xs]
    ys = []
    for s, (xq, _) in zip(streams, xs):
        with torch.cuda.stream(s):
            ys.append([sv.sv_mx_projection(xq, wq) for _ in range(5)][-1])
    torch.cuda.synchronize()
    for y, (_, xv) in zip(ys, xs):
        check_product(y, xv, wv, 512)


def test_calls_on_a_given_stream(sv):
    # every call on a stream that is not the current one, its outputs dropped early
    side = torch.cuda.Stream()
    x, r = make((900, 256), "bf16", 46, odd=False), make((900, 256), "bf16", 47, odd=False)
    w = make((256,), "f32", 48, odd=False)
    wq, _ = operand(sv, 384, 256, "nvfp4", 49)

    def chain(stream):
        g = sv.sv_mx_global_scale(x, stream=stream)
        yq, h = sv.sv_rmsnorm(x, w, residual=r, fmt=sv.SV_NVFP4, gscale=g, stream=stream)
        q, k, v = sv.sv_mx_qkv_projection(yq, wq, 3, 300, 2, 64, stream=stream)
        oq = sv.sv_mx_quantize(q, sv.SV_MXFP8, stream=stream)
        return h, q, k, v, sv.sv_mx_dequantize(oq, stream=stream), sv.sv_mx_projection(yq, wq, stream=stream)

    want = chain(None)
    torch.cuda.synchronize()
    for _ in range(3):
        got = chain(side)
        trash = [torch.full((900, 256), 3.0, device="cuda") for _ in range(8)]  # takes what the chain has freed
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(got, want)) and len(trash) == 8


def test_rows_past_the_end_are_left_as_they_were(sv):
    xq, xv = operand(sv, 130, 128, "mxfp4", 44)
    wq, wv = operand(sv, 72, 128, "mxfp4", 45)
    buf = torch.full((134, 72), 7.0, dtype=torch.bfloat16, device="cuda")
    sv.sv_mx_projection(xq, wq, y=buf[2:132])
    assert (buf[:2] == 7).all() and (buf[132:] == 7).all()
    check_product(buf[2:132], xv, wv, 128)


def test_bad_arguments_raise(sv):
    x = torch.zeros(4, 64, dtype=torch.bfloat16, device="cuda")
    g = torch.ones(1, device="cuda")
    with pytest.raises(ValueError):
        sv.sv_mx_quantize(x, sv.SV_NVFP4)                       # no tensor scale
    with pytest.raises(ValueError):
        sv.sv_mx_quantize(x, sv.SV_MXFP8, gscale=g)
    with pytest.raises(ValueError):
        sv.sv_mx_quantize(x.t(), sv.SV_MXFP8)                   # not contiguous
    with pytest.raises(ValueError):
        sv.sv_mx_quantize(x[:, :48].contiguous(), sv.SV_MXFP8)  # 48 columns
    with pytest.raises(TypeError):
        sv.sv_mx_quantize(x.half(), sv.SV_MXFP8)
    with pytest.raises(ValueError):
        sv.sv_mx_quantize(x[:0], sv.SV_MXFP8)
    with pytest.raises(ValueError):
        sv.sv_mx_quantize(x, 5)
    a, b = sv.sv_mx_quantize(x, sv.SV_MXFP8), sv.sv_mx_quantize(x, sv.SV_MXFP4)
    with pytest.raises(ValueError):
        sv.sv_mx_projection(a, b)
    with pytest.raises(sv.SvError):
        sv.sv_mx_projection(a, sv.sv_mx_quantize(x[:3].contiguous(), sv.SV_MXFP8))  # 3 output features
    with pytest.raises(ValueError):
        sv.sv_mx_qkv_projection(a, a, 1, 3, 1, 64)
    with pytest.raises(ValueError):
        sv.sv_rmsnorm(x, torch.ones(32, device="cuda"))
    with pytest.raises(sv.SvError):
        sv.sv_rmsnorm(x, torch.ones(64, device="cuda"), eps=-1.0)
    with pytest.raises(sv.SvError):
        sv.sv_rmsnorm(x, torch.ones(64, device="cuda"), residual=x, h=x, y=x)
