"""Microscaled operands in plain fp64: quantisation, layout, values, norm and products.

Shares no code with the GPU path. Formats (OCP Microscaling 1.0; NVFP4 of the deployment that the
SANA-Video abstract names): 'mxfp8' e4m3 elements, 32 to a power-of-two (e8m0) scale; 'mxfp4' e2m1, 32,
e8m0; 'nvfp4' e2m1, 16, an e4m3 scale, and one fp32 scale g for the tensor.

Rounding is done by comparison with the borders between neighbouring codes, border * unit being exact in
fp64 (at most 5 + 4 + 24 bits), so no quotient is ever rounded: a value on a border goes to the even code.
"""

from __future__ import annotations

import numpy as np

BLOCK = {"mxfp8": 32, "mxfp4": 32, "nvfp4": 16}
RUN = {"mxfp8": 128, "mxfp4": 256, "nvfp4": 256}  # columns in 128 bytes of codes


def _decode(bits: np.ndarray, mant: int, bias: int) -> np.ndarray:
    """Non-negative codes of a small float type with `mant` fraction bits."""
    e = bits >> mant
    m = (bits & ((1 << mant) - 1)).astype(np.float64)
    return np.where(e > 0, np.ldexp(1.0 + m / (1 << mant), e - bias), np.ldexp(m / (1 << mant), 1 - bias))


E2M1 = _decode(np.arange(8), 1, 1)      # 0, 0.5, 1, 1.5, 2, 3, 4, 6
E4M3 = _decode(np.arange(127), 3, 7)    # 0 .. 448; code 127 is NaN


def _codes(a: np.ndarray, unit: np.ndarray, values: np.ndarray) -> np.ndarray:
    """The code whose value * unit is nearest to a >= 0 (ties to the even code, the last code at most)."""
    lo = np.zeros(a.shape, dtype=np.int64)
    hi = np.full(a.shape, len(values) - 1, dtype=np.int64)
    while np.any(lo < hi):  # the largest code c with a above (or, for even c, on) the border below it
        mid = (lo + hi + 1) // 2
        border = (values[mid - 1] + values[mid]) / 2 * unit
        above = (a > border) | ((a == border) & (mid % 2 == 0))
        lo, hi = np.where(above & (lo < hi), mid, lo), np.where(~above & (lo < hi), mid - 1, hi)
    return lo


def quantize(x: np.ndarray, fmt: str, g: float | None = None):
    """x [R, C] fp64 -> (element codes [R, C] with the sign in the top bit, scale bytes [R, C / block])."""
    R, C = x.shape
    blk = x.reshape(R, -1, BLOCK[fmt])
    a = np.abs(blk).max(axis=2)
    bad = ~np.isfinite(a) | (~np.isfinite(g) if g is not None else False)
    a = np.where(bad, 0.0, a)
    v = np.where(bad[..., None], 0.0, blk)
    if fmt == "nvfp4":
        sc = _codes(a, np.full(a.shape, 6.0 * g if np.isfinite(g) else 1.0), E4M3)
        unit = E4M3[sc] * (g if np.isfinite(g) else 0.0)
    else:
        top = 448.0 if fmt == "mxfp8" else 6.0
        k = np.full(a.shape, -127)
        for e in range(-127, 128):  # the smallest power of two with a <= s * top
            k = np.where((k == e) & (a > top * 2.0**e), e + 1, k)
        sc, unit = k + 127, 2.0 ** k.astype(np.float64)
    values = E4M3 if fmt == "mxfp8" else E2M1
    u = unit[..., None] * np.ones(v.shape)
    c = np.where(u > 0, _codes(np.abs(v), u, values), 0)
    c = np.where((v < 0) & (c > 0), c | (128 if fmt == "mxfp8" else 8), c)
    sc = np.where(bad, 127 if fmt == "nvfp4" else 255, sc)
    return c.reshape(R, C).astype(np.uint8), sc.astype(np.uint8)


def elements(codes: np.ndarray, fmt: str) -> np.ndarray:
    """Element values of codes [R, C]."""
    if fmt == "mxfp8":
        mag = codes & 127
        return np.where(codes & 128, -1.0, 1.0) * np.where(mag == 127, np.nan, E4M3[np.minimum(mag, 126)])
    return np.where(codes & 8, -1.0, 1.0) * E2M1[codes & 7]


def scale_values(sc: np.ndarray, fmt: str) -> np.ndarray:
    if fmt == "nvfp4":
        mag = sc & 127
        return np.where(mag == 127, np.nan, np.where(sc & 128, -1.0, 1.0) * E4M3[np.minimum(mag, 126)])
    return np.where(sc == 255, np.nan, 2.0 ** (sc.astype(np.float64) - 127))


def values(codes: np.ndarray, sc: np.ndarray, fmt: str, g: float | None = None) -> np.ndarray:
    """The matrix that codes and scales stand for, exact in fp64."""
    v = elements(codes, fmt) * np.repeat(scale_values(sc, fmt), BLOCK[fmt], axis=1)
    return v * g if fmt == "nvfp4" else v


def pack(codes: np.ndarray, fmt: str) -> np.ndarray:
    """Codes as stored: a byte each, or two to a byte, the even column low."""
    if fmt == "mxfp8":
        return codes
    return (codes[:, 0::2] | (codes[:, 1::2] << 4)).astype(np.uint8)


def unpack(stored: np.ndarray, fmt: str) -> np.ndarray:
    if fmt == "mxfp8":
        return stored
    return np.stack([stored & 15, stored >> 4], axis=2).reshape(stored.shape[0], -1)


def tile_scales(sc: np.ndarray, fmt: str) -> np.ndarray:
    """[R, S] -> [ceil(R / 128), P / 4, 32, 4, 4], zeros where there is no block."""
    R, S = sc.shape
    per_run = RUN[fmt] // BLOCK[fmt]
    P = -(-S // per_run) * per_run
    out = np.zeros((-(-R // 128), P // 4, 32, 4, 4), dtype=np.uint8)
    for r in range(R):
        for j in range(S):
            out[r // 128, j // 4, r % 32, (r // 32) % 4, j % 4] = sc[r, j]
    return out


def untile_scales(t: np.ndarray, R: int, S: int) -> np.ndarray:
    r, j = np.arange(R)[:, None], np.arange(S)[None, :]
    return t[r // 128, j // 4, r % 32, (r // 32) % 4, j % 4]


def rms_norm(h: np.ndarray, w: np.ndarray, eps: float) -> np.ndarray:
    """h [R, C] (the stored sum of x and the residual) -> h / sqrt(mean(h^2) + eps) * w."""
    return h / np.sqrt((h * h).mean(axis=1, keepdims=True) + eps) * w


def heads_to_rows(x: np.ndarray) -> np.ndarray:
    """[B, H, N, D] -> [B * N, H * D]."""
    B, H, N, D = x.shape
    return np.stack([np.concatenate([x[b, h, n] for h in range(H)]) for b in range(B) for n in range(N)])
