"""Cases of the microscaled layer: root-mean-square norm with the residual's addition, quantisation to
block-scaled 8- and 4-bit floating point, and the projections on such operands.

Formats (value = element x block scale x tensor scale):

    mxfp8   e4m3 elements, 32 to a block, scale a power of two (e8m0)
    mxfp4   e2m1 elements, 32 to a block, scale a power of two (e8m0)
    nvfp4   e2m1 elements, 16 to a block, scale e4m3, and one fp32 scale g for the tensor

Quantisation of a block with largest magnitude a: mxfp8 / mxfp4 take the smallest power of two s >=
2^-127 with a <= s * (448 | 6); nvfp4 takes s = e4m3(a / (6 g)). Elements are x / (s g); both quotients are
rounded once, to nearest, ties to even, and stop at the type's largest value. A block whose a or g is not finite gets the scale NaN and zero elements.

Scales lie in tiles of 128 rows x 4 blocks: [rows / 128][blocks / 4][row % 32][row / 32 % 4][block % 4]
bytes, rows rounded up to 128 and columns to 128 bytes of elements, the rest zero. 4-bit elements lie two to
a byte, the even column low.
"""

import torch

own = False  # set by the measuring tools: run() then calls this repository's kernels

BLOCK = {"mxfp8": 32, "mxfp4": 32, "nvfp4": 16}
PAD = {"mxfp8": 4, "mxfp4": 8, "nvfp4": 16}  # blocks in 128 bytes of elements
EPS = 1e-6


def listed():
    return [
        # one token's pre-norm, its output in 8 bits: latency of a token-by-token caller
        {"name": "norm_token_mxfp8", "op": "norm", "B": 1, "N": 1, "C": 2560, "dt": "bf16", "fmt": "mxfp8", "res": True},
        # the pre-norm of one 720p streaming block (3 frames of 23 x 40 tokens), output in 8 bits
        {"name": "norm_block_mxfp8", "op": "norm", "B": 1, "N": 2760, "C": 2560, "dt": "bf16", "fmt": "mxfp8", "res": True},
        # the pre-norm of a whole 720p prefill with an unquantised output (the bf16 projections)
        {"name": "norm_prefill_bf16", "op": "norm", "B": 1, "N": 55200, "C": 2560, "dt": "bf16", "fmt": "none", "res": True},
        # fp32 activations, ragged rows and an odd hidden size
        {"name": "norm_odd_f32", "op": "norm", "B": 2, "N": 1013, "C": 2592, "dt": "f32", "fmt": "none", "res": False},
        # the attention output of a 2.0 layer, heads gathered into rows, to 4 bits with a calibrated g
        {"name": "quant_heads_nvfp4", "op": "quant", "B": 2, "H": 20, "N": 10120, "D": 128, "dt": "bf16", "fmt": "nvfp4", "dynamic": False},
        # converting an fp32 weight (fused Q/K/V, hidden 2560) to 4 bits, its tensor scale measured
        {"name": "quant_weight_nvfp4", "op": "quant", "B": 1, "H": 1, "N": 7680, "D": 2560, "dt": "f32", "fmt": "nvfp4", "dynamic": True},
        # the output projection of one token
        {"name": "linear_token_nvfp4", "op": "linear", "B": 1, "H": 20, "N": 1, "D": 128, "Nout": 2560, "dt": "bf16", "fmt": "nvfp4"},
        # the output projection of a 720p streaming block, 8 bits
        {"name": "linear_block_mxfp8", "op": "linear", "B": 1, "H": 20, "N": 2760, "D": 128, "Nout": 2560, "dt": "bf16", "fmt": "mxfp8"},
        # ragged sizes of every dimension
        {"name": "linear_odd_mxfp4", "op": "linear", "B": 3, "H": 1, "N": 331, "D": 2592, "Nout": 2568, "dt": "bf16", "fmt": "mxfp4"},
        # norm and Q/K/V projection of one streaming block with 4-bit operands
        {"name": "qkv_block_nvfp4", "op": "qkv", "B": 1, "N": 2760, "C": 2560, "H": 20, "D": 128, "fmt": "nvfp4"},
        # the same for a 2.0 layer (2 x 11 frames) in 8 bits
        {"name": "qkv_layer_mxfp8", "op": "qkv", "B": 2, "N": 10120, "C": 2560, "H": 20, "D": 128, "fmt": "mxfp8"},
        # the same for a whole 720p prefill in 4 bits
        {"name": "qkv_prefill_nvfp4", "op": "qkv", "B": 1, "N": 55200, "C": 2560, "H": 20, "D": 128, "fmt": "nvfp4"},
    ]


def _log(rng, lo, hi):
    return int(round(lo * (hi / lo) ** rng.random()))


def draw(rng):
    op = rng.choice(["norm", "quant", "linear", "qkv"])
    fmt = rng.choice(["mxfp8", "mxfp4", "nvfp4"])
    dt = rng.choice(["bf16", "bf16", "f32"])
    B = rng.choice([1, 1, 2, 3])
    N = max(1, _log(rng, 1, 20000) // B)
    C = 32 * _log(rng, 1, 160)
    if op == "norm":
        return {"op": op, "B": B, "N": N, "C": C, "dt": dt, "fmt": rng.choice([fmt, "none"]), "res": rng.random() < 0.7}
    heads = rng.random() < 0.5
    D = rng.choice([32, 64, 96, 128]) if heads else C
    H = _log(rng, 1, 24) if heads else 1
    if op == "quant":
        return {"op": op, "B": B, "H": H, "N": N, "D": D, "dt": dt, "fmt": fmt, "dynamic": fmt == "nvfp4" and rng.random() < 0.5}
    if op == "linear":
        return {"op": op, "B": B, "H": H, "N": N, "D": D, "Nout": 8 * _log(rng, 1, 1280), "dt": dt, "fmt": fmt}
    return {"op": op, "B": B, "N": N, "C": C, "H": _log(rng, 1, 24), "D": rng.choice([64, 128]), "fmt": fmt}


# ---- inputs ----

DT = {"bf16": torch.bfloat16, "f32": torch.float32}


def _activations(gen, rows, C, dt):
    """Residual-stream values: channels of different size, a few of them large, rows of different size."""
    x = torch.randn(rows, C, generator=gen, device="cuda")
    ch = torch.exp(0.4 * torch.randn(C, generator=gen, device="cuda"))
    ch *= torch.where(torch.rand(C, generator=gen, device="cuda") < 0.01, 12.0, 1.0)
    return (x * ch * torch.exp(0.3 * torch.randn(rows, 1, generator=gen, device="cuda"))).to(DT[dt])


def _calibrated(gen, largest):
    """A tensor scale from calibration: the mean of the largest values of some batches, near `largest`."""
    return (largest * (0.9 + 0.2 * torch.rand(8, generator=gen, device="cuda"))).mean().reshape(1) / (6.0 * 448.0)


def _weight(gen, rows, C, fmt):
    """A weight that the program holds quantised: its elements, scales and tensor scale."""
    w = torch.randn(rows, C, generator=gen, device="cuda") / C**0.5
    g = w.abs().amax().reshape(1) / (6.0 * 448.0) if fmt == "nvfp4" else None
    e, s = _quantise(w, fmt, g)
    return {"codes": _pack(e, fmt), "scales": _tile(_scale_bytes(s, fmt), fmt), "g": g, "rows": rows, "C": C, "fmt": fmt}


def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    op, fmt = case["op"], case["fmt"]
    st = dict(case)
    if op in ("norm", "qkv"):
        rows, C = case["B"] * case["N"], case["C"]
        dt = case.get("dt", "bf16")
        st["x"] = _activations(gen, rows, C, dt).reshape(case["B"], case["N"], C)
        st["r"] = _activations(gen, rows, C, dt).reshape(case["B"], case["N"], C) if case.get("res", True) else None
        st["nw"] = 1.0 + 0.2 * torch.randn(C, generator=gen, device="cuda")
        st["g"] = _calibrated(gen, 24.0) if fmt == "nvfp4" else None
        if op == "qkv":
            st["w"] = _weight(gen, 3 * case["H"] * case["D"], C, fmt)
    else:
        B, H, N, D = case["B"], case["H"], case["N"], case["D"]
        x = _activations(gen, B * H * N, D, "f32") * 0.05  # attention outputs and weights are small
        st["x"] = x.to(DT[case["dt"]]).reshape((B, H, N, D) if H > 1 else (B, N, D))
        st["g"] = _calibrated(gen, 3.0) if fmt == "nvfp4" and not case.get("dynamic") else None
        if op == "linear":
            st["w"] = _weight(gen, case["Nout"], H * D, fmt)
    if own:
        import block_causal_linear_relu_b200 as sv

        st["fmt_id"] = {"none": None, "mxfp8": sv.SV_MXFP8, "mxfp4": sv.SV_MXFP4, "nvfp4": sv.SV_NVFP4}[fmt]
        if "w" in st:
            w = st["w"]
            st["wq"] = sv.MxTensor(w["codes"], w["scales"], w["rows"], w["C"], st["fmt_id"], w["g"])
    return st


# ---- plain form: elementary torch operations in 32 bits (the norm's sum in 64) ----


def _e2m1(v):
    """|v| rounded to 0, 0.5, 1, 1.5, 2, 3, 4, 6 (ties to the even code), with v's sign."""
    a = v.abs()
    r = 0.5 * (a > 0.25) + 0.5 * (a >= 0.75) + 0.5 * (a > 1.25) + 0.5 * (a >= 1.75) + 1.0 * (a > 2.5) + 1.0 * (a >= 3.5) + 2.0 * (a > 5.0)
    return torch.where(v < 0, -r, r)


def _e4m3(v):
    """v >= 0 in 64 bits to the nearest e4m3 value up to 448, ties to the even code, still in 64 bits."""
    t = torch.arange(127, dtype=torch.uint8, device=v.device).view(torch.float8_e4m3fn).double()
    i = torch.searchsorted(t, v.clamp(max=448.0), right=True).clamp(max=126) - 1  # t[i] <= v <= t[i + 1]
    mid = (t[i] + t[i + 1]) / 2
    return t[i + ((v > mid) | ((v == mid) & (i % 2 == 1))).long()]


def _pow2(k):
    """2^k in fp32 for whole k in [-127, 127], from its bits."""
    return torch.where(k > -127, (k + 127) << 23, 1 << 22).to(torch.int32).view(torch.float32)


def _quantise(x, fmt, g):
    """x [R, C] fp32 -> element values [R, C] fp32 and scales [R, C / block] fp32."""
    b = x.reshape(x.shape[0], -1, BLOCK[fmt])
    a = b.abs().amax(-1)
    if fmt == "nvfp4":  # the quotients in 64 bits: bf16 values often lie on a border between two elements
        fine = torch.isfinite(a) & torch.isfinite(g)
        s = _e4m3(torch.where(fine, a, 0.0).double() / (6.0 * g.double()))
        d = (s * g.double())[..., None]
        q = _e2m1(torch.where(d > 0, b.double() / d, 0.0)).float()
        s = s.float()
    else:
        m, e = torch.frexp(a)  # a = m 2^e, 0.5 <= m < 1
        top_m, top_e = (0.875, 9) if fmt == "mxfp8" else (0.75, 3)
        k = (e - top_e + (m > top_m)).clamp(min=-127)
        k = torch.where(a > 0, k, -127)
        fine = torch.isfinite(a)
        k = torch.where(fine, k, 0)
        s = _pow2(k)
        q = b * _pow2(-k)[..., None]
        q = q.clamp(-448.0, 448.0).to(torch.float8_e4m3fn).float() if fmt == "mxfp8" else _e2m1(q)
    s = torch.where(fine, s, float("nan"))
    q = torch.where(fine[..., None], q, 0.0)
    return q.reshape(x.shape), s


def _scale_bytes(s, fmt):
    if fmt == "nvfp4":
        return s.to(torch.float8_e4m3fn).view(torch.uint8)
    m, e = torch.frexp(s)
    return torch.where(torch.isnan(s), 255, e + 126).to(torch.uint8)


def _tile(s, fmt):
    """[R, S] scale bytes -> [R / 128, S / 4, 32, 4, 4], rounded up with zeros."""
    R, S = s.shape
    Rb, Sp = -(-R // 128), -(-S // PAD[fmt]) * PAD[fmt]
    full = torch.zeros(Rb * 128, Sp, dtype=torch.uint8, device=s.device)
    full[:R, :S] = s
    return full.reshape(Rb, 4, 32, Sp // 4, 4).permute(0, 3, 2, 1, 4).contiguous()


def _pack(q, fmt):
    if fmt == "mxfp8":
        return q.to(torch.float8_e4m3fn).view(torch.uint8)
    a = q.abs()
    code = torch.where(a < 2, 2 * a, torch.where(a < 4, a + 2, a / 2 + 4)).to(torch.uint8)
    code = code | (torch.signbit(q).to(torch.uint8) << 3)
    return (code[:, 0::2] | (code[:, 1::2] << 4)).contiguous()


def _unpack(w):
    """The fp32 values of a packed weight."""
    fmt, R, C = w["fmt"], w["rows"], w["C"]
    if fmt == "mxfp8":
        q = w["codes"].view(torch.float8_e4m3fn).float()
    else:
        table = torch.tensor([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0], device="cuda")
        table = torch.cat([table, -table])
        c = w["codes"].long()
        q = torch.stack([table[c & 15], table[c >> 4]], -1).reshape(R, C)
    t = w["scales"].permute(0, 3, 2, 1, 4).reshape(w["scales"].shape[0] * 128, -1)[:R, : C // BLOCK[fmt]].contiguous()
    s = t.view(torch.float8_e4m3fn).float() if fmt == "nvfp4" else _pow2(t.int() - 127)
    v = (q.reshape(R, -1, BLOCK[fmt]) * s[..., None]).reshape(R, C)
    return v * w["g"] if fmt == "nvfp4" else v


def _values(q, s, fmt, g):
    v = (q.reshape(q.shape[0], -1, BLOCK[fmt]) * s[..., None]).reshape(q.shape)
    return v * g if fmt == "nvfp4" else v


def _norm(st):
    """(h, y): h = x + r in x's type, y = h / rms(h) * w in fp32."""
    x, r = st["x"], st["r"]
    h = x if r is None else (x.float() + r.float()).to(x.dtype)
    h = h.reshape(-1, x.shape[-1])
    rstd = (1.0 / torch.sqrt(h.double().square().mean(-1, keepdim=True) + EPS)).float()
    return h, h.float() * rstd * st["nw"]


def _rows(st):
    """x as rows: [B, N, C], or [B, H, N, D] with the heads side by side in a row."""
    x = st["x"]
    return x.permute(0, 2, 1, 3).reshape(x.shape[0] * x.shape[2], -1) if x.dim() == 4 else x.reshape(-1, x.shape[-1])


def _plain(st):
    op, fmt = st["op"], st["fmt"]
    if op == "norm":
        h, y = _norm(st)
        out = {"h": h} if st["r"] is not None else {}
        if fmt == "none":
            return {**out, "y": y.to(st["x"].dtype)}
        q, s = _quantise(y, fmt, st["g"])
        if fmt == "mxfp8":
            return {**out, "y": q.to(torch.float8_e4m3fn), "s": _tile(_scale_bytes(s, fmt), fmt).view(torch.float8_e8m0fnu)}
        return {**out, "y": _values(q, s, fmt, st["g"]).to(torch.bfloat16)}
    if op == "qkv":
        h, y = _norm(st)
        v = _values(*_quantise(y, fmt, st["g"]), fmt, st["g"])
        B, N, H, D = st["B"], st["N"], st["H"], st["D"]
        p = (v @ _unpack(st["w"]).t()).reshape(B, N, 3, H, D).permute(2, 0, 3, 1, 4)
        return {"h": h, "q": p[0].clamp(min=0).to(torch.bfloat16), "k": p[1].clamp(min=0).to(torch.bfloat16), "v": p[2].to(torch.bfloat16)}
    x = _rows(st).float()
    g = x.abs().amax().reshape(1) / torch.full((1,), 6.0 * 448.0, device="cuda") if st.get("dynamic") else st["g"]
    q, s = _quantise(x, fmt, g)
    if op == "quant":
        if fmt == "mxfp8":
            return {"y": q.to(torch.float8_e4m3fn), "s": _tile(_scale_bytes(s, fmt), fmt).view(torch.float8_e8m0fnu)}
        return {"y": _values(q, s, fmt, g).to(torch.bfloat16)}
    return {"y": (_values(q, s, fmt, g) @ _unpack(st["w"]).t()).to(torch.bfloat16)}


# ---- the framework's calls ----


def _own(st):
    import block_causal_linear_relu_b200 as sv

    op, fmt = st["op"], st["fmt_id"]
    if op in ("norm", "qkv"):
        y, h = sv.sv_rmsnorm(st["x"], st["nw"], residual=st["r"], eps=EPS, fmt=fmt, gscale=st["g"])
        if op == "qkv":
            q, k, v = sv.sv_mx_qkv_projection(y, st["wq"], st["B"], st["N"], st["H"], st["D"])
            return {"h": h.view(-1, st["C"]), "q": q, "k": k, "v": v}
        out = {"h": h.view(-1, st["C"])} if st["r"] is not None else {}
        if fmt is None:
            return {**out, "y": y.view(-1, st["C"])}
        if st["fmt"] == "mxfp8":
            return {**out, "y": y.codes.view(torch.float8_e4m3fn), "s": y.scales.view(torch.float8_e8m0fnu)}
        return {**out, "y": sv.sv_mx_dequantize(y)}
    g = sv.sv_mx_global_scale(st["x"]) if st.get("dynamic") else st["g"]
    xq = sv.sv_mx_quantize(st["x"], fmt, gscale=g)
    if op == "quant":
        if st["fmt"] == "mxfp8":
            return {"y": xq.codes.view(torch.float8_e4m3fn), "s": xq.scales.view(torch.float8_e8m0fnu)}
        return {"y": sv.sv_mx_dequantize(xq)}
    return {"y": sv.sv_mx_projection(xq, st["wq"])}


def run(state):
    return _own(state) if own else _plain(state)


# ---- the work that a pass cannot do without ----


def _mx_bytes(R, C, fmt):
    return R * C * (1 if fmt == "mxfp8" else 0.5) + R * C / BLOCK[fmt]


def work(case):
    op, fmt = case["op"], case["fmt"]
    if op in ("norm", "qkv"):
        R, C = case["B"] * case["N"], case["C"]
        e = 4 if case.get("dt") == "f32" else 2
        read = R * C * e * (2 if case.get("res", True) else 1) + 4 * C
        wrote = R * C * e if case.get("res", True) else 0
        flops = 4 * R * C
        if op == "qkv":
            F = 3 * case["H"] * case["D"]
            return {"bytes": read + wrote + _mx_bytes(F, C, fmt) + 2 * R * F, "flops": flops + 2 * R * C * F}
        wrote += R * C * e if fmt == "none" else _mx_bytes(R, C, fmt) if fmt == "mxfp8" else 2 * R * C
        return {"bytes": read + wrote, "flops": flops}
    R, C = case["B"] * case["N"], case["H"] * case["D"]
    read = R * C * (4 if case["dt"] == "f32" else 2)
    if op == "quant":
        return {"bytes": read + (_mx_bytes(R, C, fmt) if fmt == "mxfp8" else 2 * R * C), "flops": 2 * R * C}
    F = case["Nout"]
    return {"bytes": read + _mx_bytes(F, C, fmt) + 2 * R * F, "flops": 2 * R * C * F}


# ---- the definition in 64 bits, apart from the plain form ----


def _two_to(k):
    """2^k in 64 bits for whole k, from its bits."""
    return ((k.long() + 1023) << 52).view(torch.float64)


def _mini(v, mantissa, lowest, top):
    """v (64 bits) to the nearest value of a small float type: `mantissa` bits behind the point, lowest exponent, largest value."""
    _, e = torch.frexp(v)
    step = _two_to((e - 1).clamp(min=lowest) - mantissa)
    return (torch.round(v / step) * step).clamp(-top, top)


def _exact_quantise(x, fmt, g):
    n = 16 if fmt == "nvfp4" else 32
    blocks = x.view(x.shape[0], x.shape[1] // n, n)
    top = blocks.abs().max(dim=2).values
    if fmt == "nvfp4":
        scale = _mini(top / (g * 6), 3, -6, 448.0)
        unit = scale * g
    else:
        limit = 448.0 if fmt == "mxfp8" else 6.0
        scale = _two_to(torch.ceil(torch.log2((top / limit).clamp(min=2.0**-127))))
        scale = torch.where(top > scale * limit, 2 * scale, scale)
        scale = torch.where((top <= scale / 2 * limit) & (scale > 2.0**-127), scale / 2, scale)
        unit = scale
    ratio = blocks / unit.masked_fill(unit == 0, float("inf")).unsqueeze(2)
    elements = _mini(ratio, 3, -6, 448.0) if fmt == "mxfp8" else _mini(ratio, 1, 0, 6.0)
    return elements.view(x.shape), scale, (elements * unit.unsqueeze(2)).view(x.shape)


def _exact_scales(scale, fmt):
    """The scales in their tiles; places that hold none are bytes of zero, 2^-127 in e8m0."""
    R, S = scale.shape
    rows, blocks = (R + 127) // 128 * 128, (S + PAD[fmt] - 1) // PAD[fmt] * PAD[fmt]
    out = torch.full((rows // 128, blocks // 4, 32, 4, 4), 2.0**-127, dtype=torch.float64, device=scale.device)
    r = torch.arange(R, device=scale.device).unsqueeze(1)
    b = torch.arange(S, device=scale.device).unsqueeze(0)
    out[r // 128, b // 4, r % 32, r // 32 % 4, b % 4] = scale
    return out


def _exact_weight(w):
    """The values of a packed weight from the bits of its bytes."""
    R, C, fmt = w["rows"], w["C"], w["fmt"]
    byte = w["codes"].int()
    if fmt == "mxfp8":
        sign, e, m = byte >> 7, (byte >> 3) & 15, (byte & 7).double()
        v = torch.where(e > 0, (1 + m / 8) * _two_to(e - 7), m / 8 * 2.0**-6)
    else:
        code = torch.stack([byte % 16, byte // 16], dim=2).view(R, C)
        sign, e, m = code >> 3, (code >> 1) & 3, (code & 1).double()
        v = torch.where(e > 0, (1 + m / 2) * _two_to(e - 1), m / 2)
    v = torch.where(sign > 0, -v, v)
    r = torch.arange(R, device="cuda").unsqueeze(1)
    b = torch.arange(C // BLOCK[fmt], device="cuda").unsqueeze(0)
    t = w["scales"][r // 128, b // 4, r % 32, r // 32 % 4, b % 4].int()
    if fmt == "nvfp4":
        e, m = (t >> 3) & 15, (t & 7).double()
        s = torch.where(e > 0, (1 + m / 8) * _two_to(e - 7), m / 8 * 2.0**-6) * w["g"].double()
    else:
        s = _two_to(t - 127)
    return v * s.repeat_interleave(BLOCK[fmt], dim=1)


def exact(case, seed):
    st = prepare(case, seed)
    op, fmt = case["op"], case["fmt"]
    g = st["g"].double() if st["g"] is not None else None
    out = {}
    if op in ("norm", "qkv"):
        x = st["x"].double().flatten(0, 1)
        if st["r"] is not None:
            out["h"] = x + st["r"].double().flatten(0, 1)
            x = out["h"].to(st["x"].dtype).double()  # the norm is of the stored h
        x = x * torch.rsqrt((x * x).sum(1, keepdim=True) / x.shape[1] + EPS) * st["nw"].double()
        if fmt == "none":
            return {**out, "y": x}
    else:
        x = st["x"].double()
        x = torch.cat([x[:, i] for i in range(x.shape[1])], dim=2) if x.dim() == 4 else x
        x = x.flatten(0, 1)
        if case.get("dynamic"):
            g = (x.abs().max() / 2688).float().double()  # the tensor scale is held in 32 bits
    elements, scale, values = _exact_quantise(x, fmt, g)
    if op in ("norm", "quant"):
        return {**out, "y": elements, "s": _exact_scales(scale, fmt)} if fmt == "mxfp8" else {**out, "y": values}
    y = values @ _exact_weight(st["w"]).T
    if op == "linear":
        return {"y": y}
    B, N, H, D = case["B"], case["N"], case["H"], case["D"]
    q, k, v = (t.reshape(B, N, H, D).transpose(1, 2) for t in y.split(H * D, dim=1))
    return {**out, "q": torch.relu(q), "k": torch.relu(k), "v": v}
