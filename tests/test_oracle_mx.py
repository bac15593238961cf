"""Pins of the microscaled 4-bit oracle: brute force against the list of
values, constructed halves and borders, the layout by hand."""
import math

import numpy as np
import pytest

from oracle import hadamard, mx


def _decode(codes, byte):
    return mx.values(codes, byte)


def test_grid_is_e2m1():
    for c, g in enumerate(mx.GRID):
        e, m = c >> 1, c & 1
        assert g == (m * 0.5 if e == 0 else 2.0 ** (e - 1) * (1 + m / 2))


def test_every_step_by_brute_force():
    a = np.concatenate([np.arange(0, 8, 1 / 64), [0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0, 7.99]])
    x = np.zeros((len(a), 32), np.float32)
    x[:, 0] = 4.0                        # A in [4, 8): one unit
    x[:, 1] = a
    x[:, 2] = -a
    codes, byte = mx.quantize(x)
    assert np.all(byte == 127)
    for i, v in enumerate(a):
        want = mx.nearest_code(v)
        assert codes[i, 1] == want and codes[i, 2] == (want + 8 if want else 0), v


def test_halves_go_to_even_codes():
    halves = {0.25: 0.0, 0.75: 1.0, 1.25: 1.0, 1.75: 2.0, 2.5: 2.0, 3.5: 4.0, 5.0: 4.0}
    for v, want in halves.items():
        assert mx.GRID[mx.nearest_code(v)] == want, v


def test_powers_and_borders():
    x = np.zeros((7, 32), np.float32)
    x[0, 3] = 7.999                     # saturates at 6 units of 1
    x[1, 3] = 8.0                       # the next power
    x[2, 3] = 2.0 ** -126               # the smallest normal: byte clamped at 0
    x[3, 3] = 2.0 ** -130
    x[4, 3] = 3.0e38
    x[6, :] = -0.0
    codes, byte = mx.quantize(x)
    assert byte[:, 0].tolist() == [127, 128, 0, 0, 127 + 125, 0, 0]
    assert mx.GRID[codes[0, 3]] == 6 and mx.GRID[codes[1, 3]] == 4
    assert mx.GRID[codes[2, 3]] == 2 and mx.GRID[codes[3, 3]] == 0       # 2^-126 = 2 units of 2^-127; 2^-3 of a unit
    assert not codes[5].any() and not codes[6].any()
    x[0, 5], x[1, 6] = np.inf, np.nan
    codes, byte = mx.quantize(x)
    assert byte[0, 0] == 255 and byte[1, 0] == 255 and not codes[:2].any()
    assert np.isnan(_decode(codes, byte)[0]).all()


@pytest.mark.parametrize("rot", [0, 16, 64, 256, 1024])
def test_error_and_rotation(rot):
    g = np.random.default_rng(rot)
    x = g.standard_normal((5, 1024)).astype(np.float32)
    codes, byte = mx.quantize(x, rot)
    v = hadamard.rotate(x, rot).astype(np.float64) / math.sqrt(rot) if rot else x.astype(np.float64)
    got = mx.values(codes, byte)
    unit = np.repeat(np.exp2(byte.astype(np.float64) - 127), 32, axis=1)
    # steps are half a unit below 2, one below 4, two above; beyond 6 up to 8 the value is 6
    assert np.all(np.abs(got - v) <= unit * np.where(np.abs(v) < 2 * unit, 0.25, np.where(np.abs(v) < 4 * unit, 0.5, 2)))
    top = np.abs(v).reshape(5, -1, 32).max(-1)
    u = np.exp2(byte.astype(np.float64) - 127)
    assert np.all((top >= 4 * u) & (top < 8 * u))
    back = mx.dequantize(codes, byte, rot)
    assert np.linalg.norm(back - x) < 0.15 * np.linalg.norm(x)
    # the product of two operands in the same rotated basis is that of the unrotated values
    w = g.standard_normal((3, 1024)).astype(np.float32)
    wc, wb = mx.quantize(w, rot)
    y, _ = mx.gemm(got, mx.values(wc, wb))
    assert np.allclose(y, back @ mx.dequantize(wc, wb, rot).T, rtol=0, atol=1e-9 * np.abs(y).max())


def test_layout_by_hand():
    g = np.random.default_rng(3)
    codes, byte = g.integers(0, 16, (3, 160)).astype(np.uint8), g.integers(0, 255, (3, 5)).astype(np.uint8)
    c, b = mx.pack(codes, byte)
    assert c.shape == (2, 3, 64) and b.shape == (2, 3, 4)
    assert c[0, 1, 7] == codes[1, 14] + 16 * codes[1, 15]
    assert c[1, 2, 15] == codes[2, 158] + 16 * codes[2, 159] and not c[1, :, 16:].any()
    assert b[0, 2].tolist() == byte[2, :4].tolist() and b[1, 1].tolist() == [byte[1, 4], 0, 0, 0]
    back = mx.unpack(c, b, 160)
    assert np.array_equal(back[0], codes) and np.array_equal(back[1], byte)
