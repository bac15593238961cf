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


# ---------------------------------------------------------------------------
# 8-bit moments over many steps. A code's rounding is right on average, a value's is not:
# the value goes as the code's square (of a root) or its square with a sign, so its average
# lies above by the variance of the code.
# ---------------------------------------------------------------------------
STEPS, WIDE = 200, 4096


def decaying_roots(step_fn, n=WIDE):
    """One step with gradients of all sizes, then STEPS without, but for the largest of each block, which keeps its size and
    so the block's scale. step_fn(gradient, step) -> codes of the roots. (Codes after the first step, codes at the end,
    elements that decay)."""
    g = np.random.default_rng(21)
    first = np.exp2(g.uniform(-6, -0.1, n)).astype(np.float32)
    first[::256] = 1
    rest = np.zeros(n, np.float32)
    rest[::256] = np.sqrt(np.float32(1 - 0.999))
    start = step_fn(first, 1).astype(np.float64)
    for step in range(2, STEPS + 2):
        last = step_fn(rest, step)
    at = np.arange(n) % 256 != 0
    return start[at], last.astype(np.float64)[at], at


def check_decaying_roots(start, last):
    """With beta2 = 0.999 a root's code is 255 sqrt(root / s) and falls by 0.999^(1/4) a step, on average exactly that from one
    code to the next. What is cut off or added in a step has the variance f (1 - f) <= 1/4 with f the code's fall, at most
    2.6e-4 of it: over all steps at most STEPS * 2.6e-4 times the code. Six deviations of the mean over the elements."""
    kept = 0.999 ** (STEPS / 4)
    deviation = np.sqrt((STEPS * 2.6e-4 * start).sum()) / len(start)
    off = (last - kept * start).mean()
    assert start.min() > 25 and abs(off) <= 6 * deviation, (off, deviation)


def _steps(encode_u=None):
    """step_fn of the oracle; encode_u: in the place of the random numbers (a planted mistake)."""
    state = {"r": (np.zeros(WIDE, np.uint8), np.zeros(WIDE // 256, np.float32)), "m": (np.zeros(WIDE, np.int8), np.zeros(WIDE // 256, np.float32))}
    kept = tr.random_pair

    def step(g, t):
        p = np.zeros(WIDE, np.float32)
        if encode_u is not None:
            tr.random_pair = lambda seed, tensor, n: (np.full(n, encode_u, np.float32),) * 2
        try:
            _, mc, ms, vc, vs = tr.adamw8(p, g, *state["m"], *state["r"], t, 1e-3, 0.9, 0.999, 1e-8, 0.0, t, 0)
        finally:
            tr.random_pair = kept
        state["m"], state["r"] = (mc, ms), (vc, vs)
        return vc

    step.state = state
    return step


def test_roots_decay_on_average():
    check_decaying_roots(*decaying_roots(_steps())[:2])


def test_roots_rounded_to_the_nearest_would_stick():
    start, last, _ = decaying_roots(_steps(0.5))
    assert np.array_equal(start, last)
    with pytest.raises(AssertionError):
        check_decaying_roots(start, last)


def turning_gradients(n=WIDE):
    """A gradient, and three quarters of it but for the largest of each block, which keeps the block's scale."""
    g = np.random.default_rng(22)
    first = np.exp2(g.uniform(-6, 0, n)) * np.where(g.integers(0, 2, n), 1, -1)
    first[::256] = 1
    at = np.arange(n) % 256 != 0
    return first.astype(np.float32), np.where(at, 0.75 * first, first).astype(np.float32), at


def check_first_moment(values, first, then, at, steps):
    """After `steps` of either gradient m = then (1 - 0.9^steps) + first (1 - 0.9^steps) 0.9^steps. With s <= 1 the largest of a
    block: a step's rounding moves the code by what it cuts or adds, variance at most 1/4, so the value by 2 c / 127^2 of that,
    and by at most 1 / (4 127^2) on average, always away from zero; what came before counts 0.9, so the mean adds up to 10 times
    that and the variance to 1 / (1 - 0.81). Six deviations of the mean over the elements, signs taken out."""
    fade = 0.9 ** steps
    want = (1 - fade) * (np.abs(then) + fade * np.abs(first))
    code = 127 * np.sqrt(np.abs(first))
    deviation = np.sqrt(((2 * code + 1) ** 2 / 4 / (1 - 0.81))[at].sum()) / 127 ** 2 / at.sum()
    off = (values * np.sign(first) - want)[at].mean()
    assert -6 * deviation <= off <= 10 / (4 * 127 ** 2) + 6 * deviation, (off, deviation)


@pytest.mark.parametrize("u", [None, 0.5])
def test_first_moment_follows_on_average(u):
    first, then, at = turning_gradients()
    step = _steps(u)
    for t in range(1, 121):
        step(first if t <= 60 else then, t)
    m = tr.decode(*step.state["m"], 127).astype(np.float64)
    if u is None:
        check_first_moment(m, first, then, at, 60)
    else:                                                # the nearest code: it stops on its way
        with pytest.raises(AssertionError):
            check_first_moment(m, first, then, at, 60)
