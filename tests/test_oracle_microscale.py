"""Pins of the microscaled oracle: code tables, hand-worked blocks, exhaustive rounding against the nearest
value, layout round trips."""

import numpy as np
import pytest

from oracle import microscale as M


def test_code_tables():
    assert M.E2M1.tolist() == [0, 0.5, 1, 1.5, 2, 3, 4, 6]
    assert M.E4M3[1] == 2.0**-9 and M.E4M3[8] == 2.0**-6 and M.E4M3[56] == 1.0 and M.E4M3[126] == 448.0
    assert np.all(np.diff(M.E4M3) > 0)


def test_hand_worked_blocks():
    x = np.zeros((1, 32))
    x[0, :4] = [6.0, 2.5, -5.0, 0.25]      # ties: 2.5 -> 2, 5 -> 4, 0.25 -> 0
    c, s = M.quantize(x, "mxfp4")
    assert s.tolist() == [[127]] and M.elements(c, "mxfp4")[0, :4].tolist() == [6, 2, -4, 0]
    x[0, 0] = 6.0000001                      # above 6: the scale doubles, nothing saturates
    c, s = M.quantize(x, "mxfp4")
    assert s.tolist() == [[128]] and M.elements(c, "mxfp4")[0, :3].tolist() == [3, 1, -2]  # 1.25 is a tie -> 1
    x = np.zeros((1, 32))
    x[0, 16] = 448 * 6.0
    c, s = M.quantize(x, "nvfp4", 1.0)
    assert s.tolist() == [[0, 126]] and M.values(c, s, "nvfp4", 1.0)[0, 16] == 2688
    x[0, 3], x[0, 20] = np.nan, np.inf
    c, s = M.quantize(x, "nvfp4", 1.0)
    assert s.tolist() == [[127, 127]] and not c.any() and np.isnan(M.values(c, s, "nvfp4", 1.0)).all()
    c, s = M.quantize(x, "mxfp8")
    assert s.tolist() == [[255]] and not c.any()
    assert M.quantize(np.zeros((1, 32)), "mxfp8")[1].tolist() == [[0]]


@pytest.mark.parametrize("fmt", ["mxfp8", "mxfp4", "nvfp4"])
def test_rounding_is_to_the_nearest_value(fmt):
    rng = np.random.default_rng(1)
    x = rng.standard_normal((40, 256)) * np.exp(3 * rng.standard_normal((40, 1)))
    g = float(np.float32(np.abs(x).max() / 2688)) if fmt == "nvfp4" else None
    c, s = M.quantize(x, fmt, g)
    unit = np.repeat(M.scale_values(s, fmt), M.BLOCK[fmt], axis=1) * (g or 1.0)
    grid = M.E4M3 if fmt == "mxfp8" else M.E2M1
    best = np.abs(np.abs(x)[..., None] - grid * unit[..., None]).min(axis=2)
    assert np.all(np.abs(M.values(c, s, fmt, g) - x) <= best * (1 + 1e-12))
    if fmt != "nvfp4":  # no saturation, and half the scale would saturate
        a = np.abs(x.reshape(40, -1, 32)).max(axis=2)
        top, sv = grid[-1], M.scale_values(s, fmt)
        assert np.all(a <= sv * top) and np.all(a > sv / 2 * top)


@pytest.mark.parametrize("fmt", ["mxfp8", "mxfp4", "nvfp4"])
def test_layout_round_trip(fmt):
    rng = np.random.default_rng(2)
    c = rng.integers(0, 256 if fmt == "mxfp8" else 16, (150, 96), dtype=np.uint8)
    assert np.array_equal(M.unpack(M.pack(c, fmt), fmt), c)
    S = 96 // M.BLOCK[fmt]
    s = rng.integers(1, 255, (150, S), dtype=np.uint8)
    t = M.tile_scales(s, fmt)
    assert t.shape == (2, {"mxfp8": 1, "mxfp4": 2, "nvfp4": 4}[fmt], 32, 4, 4)
    assert np.array_equal(M.untile_scales(t, 150, S), s)
    assert np.count_nonzero(t) == s.size


def test_norm_and_heads():
    h = np.array([[3.0, 4.0]])
    assert np.allclose(M.rms_norm(h, np.array([1.0, 2.0]), 0.0), [[3 / np.sqrt(12.5), 8 / np.sqrt(12.5)]], rtol=1e-15)
    x = np.arange(2 * 3 * 4 * 5, dtype=float).reshape(2, 3, 4, 5)
    r = M.heads_to_rows(x)
    assert r.shape == (8, 15) and np.array_equal(r[1 * 4 + 2, 2 * 5:3 * 5], x[1, 2, 2])
