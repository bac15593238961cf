"""Pins of the layer norm and AdamW oracle: closed forms, finite differences,
brute force, and what the 8-bit codes have to keep."""
import math

import numpy as np
import pytest

from oracle import training as tr


def test_norm_closed_form():
    x = np.array([[1.0, 3.0], [-2.0, -2.0]])
    y, mean, rstd = tr.norm_forward(x, eps=0.0 + 1e-30)
    assert np.allclose(mean, [2, -2]) and np.allclose(y[0], [-1, 1]) and np.allclose(y[1], 0)
    y, _, _ = tr.norm_forward(x, w=[[2.0, 4.0]], b=[[1.0, -1.0]], plus=1.0, eps=0.0 + 1e-30)
    assert np.allclose(y[0], [-3 + 1, 5 - 1]) and np.allclose(y[1], [1, -1])


def test_norm_gradients_by_differences():
    g = np.random.default_rng(1)
    M, C, S = 7, 6, 3
    x, dy = g.standard_normal((M, C)), g.standard_normal((M, C))
    w, b = g.standard_normal((S, C)), g.standard_normal((S, C))
    rows = np.array([0, 0, 0, 2, 2, 2, 2])
    f = lambda x, w, b: (tr.norm_forward(x, w, b, rows, 1.0)[0] * dy).sum()  # noqa: E731
    _, mean, rstd = tr.norm_forward(x, w, b, rows, 1.0)
    dx, dw, db = tr.norm_backward(dy, x, mean, rstd, w, rows, 1.0, S)
    h = 1e-6
    for grad, arg in ((dx, 0), (dw, 1), (db, 2)):
        for i in np.ndindex(grad.shape):
            at = [x.copy(), w.copy(), b.copy()]
            at[arg][i] += h
            hi = f(*at)
            at[arg][i] -= 2 * h
            assert abs((hi - f(*at)) / (2 * h) - grad[i]) < 1e-7, (arg, i)
    assert not dw[1].any() and not db[1].any()


def test_sequences():
    assert tr.sequences([1, 3, 3, 6], 8).tolist() == [-1, 0, 0, 2, 2, 2, -1, -1]
    assert tr.sequences([0, 5, 3, 7], 8).tolist() == [0, 0, 0, 0, 0, 2, 2, -1]
    assert tr.sequences([-4, 2, 20], 4).tolist() == [0, 0, 1, 1]


def test_adamw_first_step_and_decay():
    p, g = np.array([1.0, -2.0]), np.array([0.5, -0.25])
    z = np.zeros(2)
    p1, m, v = tr.adamw(p, g, z, z, 1, 0.1, 0.9, 0.999, 1e-8, 0.0)
    assert np.allclose(p1, p - 0.1 * np.sign(g), atol=1e-7) and np.allclose(m, 0.1 * g) and np.allclose(v, 0.001 * g * g)
    p2, _, _ = tr.adamw(p, z, z, z, 5, 0.1, 0.9, 0.999, 1e-8, 0.5)
    assert np.allclose(p2, p * 0.95)
    a, _, _ = tr.adamw(p, g * 4, z, z, 3, 0.1, 0.9, 0.999, 1e-8, 0.01, grad_scale=0.25)
    b, _, _ = tr.adamw(p, g, z, z, 3, 0.1, 0.9, 0.999, 1e-8, 0.01)
    assert np.allclose(a, b)


@pytest.mark.parametrize("most", [127, 255])
def test_codes_keep_what_they_must(most):
    g = np.random.default_rng(most)
    x = (g.standard_normal(700) * np.exp2(g.uniform(-30, 0, 700))).astype(np.float32)
    x[300:310] = 0
    if most == 255:
        x = np.abs(x)
    u = g.random(700).astype(np.float32)
    codes, scales = tr.encode(x, u, most)
    back = tr.decode(codes, scales, most).astype(np.float64)
    s = np.repeat(scales, 256)[:700].astype(np.float64)
    t = np.sqrt(np.abs(x) / s) * most
    # the code is one of the two around t, the largest is kept, signs and zeros stay
    assert np.all(np.abs(np.abs(codes.astype(int)) - t) < 1 + 1e-5)
    assert np.all(back[np.abs(x) == s] == x[np.abs(x) == s].astype(np.float64)) or np.allclose(back[np.abs(x) == s], x[np.abs(x) == s], rtol=3e-7)
    assert np.all(np.sign(back) * np.sign(x) >= 0) and not back[300:310].any()
    if most == 255:
        assert np.all(back[x > 0] > 0)


def test_codes_are_right_on_average():
    """Over many seeds the mean code is t: no state is stuck, however small its steps."""
    x = np.array([1.0] + [0.3] * 255, np.float32)
    t = math.sqrt(0.3) * 127
    mean = np.mean([tr.encode(x, tr.random_pair(seed, 0, 256)[0], 127)[0][1:].astype(float).mean() for seed in range(400)])
    # 102000 draws of a variance of at most 1/4
    assert abs(mean - t) < 5 * math.sqrt(0.25 / (400 * 255))


def test_hash_is_even():
    for seed, tensor in ((0, 0), (1, 0), (0, 1), (123456789, 251)):
        a, b = tr.random_pair(seed, tensor, 1 << 16)
        for u in (a, b):
            assert u.min() >= 0 and u.max() < 1
            n = np.bincount((u * 64).astype(int), minlength=64)
            assert np.all(np.abs(n - 1024) < 6 * 32)           # six deviations of a bin of 1024
        assert abs(np.corrcoef(a, b)[0, 1]) < 5 / 256 and abs(np.corrcoef(a[1:], a[:-1])[0, 1]) < 5 / 256
    one, two = tr.random_pair(7, 3, 4096)[0], tr.random_pair(8, 3, 4096)[0]
    assert abs(np.corrcoef(one, two)[0, 1]) < 5 / 64


def test_not_finite_blocks():
    x = np.ones(512, np.float32)
    x[300] = np.inf
    codes, scales = tr.encode(x, np.zeros(512, np.float32), 127)
    assert scales[0] == 1 and np.isnan(scales[1]) and not codes[256:].any()
    assert np.isnan(tr.decode(codes, scales, 127)[256:]).all()
