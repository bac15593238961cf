"""Layer norm with its gradients, and the AdamW step with float32 or 8-bit moments.

Sources:
  [P1] intro: the adaLN modulation layers of the block, whose outputs scale and
       shift the normalised rows of each sequence.
  The optimizer's update is that of "Decoupled Weight Decay Regularization"
  (Loshchilov, Hutter), Algorithm 2, with its schedule multiplier 1.

Definitions:
  xh = (x - mean) rstd, y = xh (w[s] + plus) + b[s], s the row's sequence
  g = dy (w[s] + plus); dx = base + rstd (g - mean(g) - xh mean(g xh))
  dw[s] = sum dy xh, db[s] = sum dy over the sequence's rows
  m' = b1 m + (1 - b1) g, v' = b2 v + (1 - b2) g^2
  p' = p (1 - lr wd) - lr m' / (1 - b1^t) / (sqrt(v' / (1 - b2^t)) + eps)
  8-bit moments, per 256 elements with s the largest magnitude of the values:
    m = s (c / 127) |c / 127|, sqrt(v) = s (c / 255)^2;
    code = floor(most sqrt(|value| / s) + u), at most `most`; for sqrt(v) > 0 at least 1
Layer norm and the update in float64; the codes in float32, each operation
rounded once, as their definition says.
"""
from __future__ import annotations

import math

import numpy as np

BLOCK = 256


def sequences(offsets, M: int) -> np.ndarray:
    """Sequence of every row, -1 for none; an offset below an earlier one counts as that one."""
    off = np.maximum.accumulate(np.asarray(offsets, np.int64))
    rows = np.full(M, -1, np.int64)
    for s in range(len(off) - 1):
        rows[max(off[s], 0):max(off[s + 1], 0)] = s
    return rows


def _affine(w, plus, rows, C):
    if w is None:
        return np.ones((len(rows), C))
    return np.asarray(w, np.float64).reshape(-1, C)[rows] + plus


def norm_forward(x, w=None, b=None, rows=None, plus=0.0, eps=1e-6):
    """(y, mean, rstd) in float64; rows: sequence of each row (default: all 0)."""
    x = np.asarray(x, np.float64)
    M, C = x.shape
    rows = np.zeros(M, np.int64) if rows is None else rows
    mean = x.sum(1) / C
    d = x - mean[:, None]
    rstd = 1 / np.sqrt((d * d).sum(1) / C + eps)
    y = d * rstd[:, None] * _affine(w, plus, rows, C)
    if b is not None:
        y = y + np.asarray(b, np.float64).reshape(-1, C)[rows]
    return y, mean, rstd


def norm_backward(dy, x, mean, rstd, w=None, rows=None, plus=0.0, S=1, base=None):
    """(dx, dw [S, C], db [S, C]) in float64; rows of no sequence (-1) add nothing to dw, db."""
    dy, x = np.asarray(dy, np.float64), np.asarray(x, np.float64)
    M, C = x.shape
    rows = np.zeros(M, np.int64) if rows is None else rows
    mean, rstd = np.asarray(mean, np.float64)[:, None], np.asarray(rstd, np.float64)[:, None]
    xh = (x - mean) * rstd
    g = dy * _affine(w, plus, rows, C)
    dx = rstd * (g - g.sum(1, keepdims=True) / C - xh * (g * xh).sum(1, keepdims=True) / C)
    if base is not None:
        dx = dx + np.asarray(base, np.float64)
    dw, db = np.zeros((S, C)), np.zeros((S, C))
    at = rows >= 0
    np.add.at(dw, rows[at], (dy * xh)[at])
    np.add.at(db, rows[at], dy[at])
    return dx, dw, db


def adamw(p, g, m, v, step, lr, b1, b2, eps, wd, grad_scale=1.0):
    """(p', m', v') in float64."""
    p, g, m, v = (np.asarray(t, np.float64) for t in (p, g, m, v))
    g = g * grad_scale
    m = b1 * m + (1 - b1) * g
    v = b2 * v + (1 - b2) * g * g
    step_m, step_v = m / (1 - b1 ** step), v / (1 - b2 ** step)
    return p - lr * wd * p - lr * step_m / (np.sqrt(step_v) + eps), m, v


def _mix(x: np.ndarray) -> np.ndarray:
    x = np.asarray(x, np.uint32)
    with np.errstate(over="ignore"):
        x = x ^ (x >> np.uint32(16))
        x = x * np.uint32(0x6A09E667)
        x = x ^ (x >> np.uint32(15))
        x = x * np.uint32(0xBB67AE85)
        return x ^ (x >> np.uint32(16))


def random_pair(seed: int, tensor: int, n: int):
    """u for m and for sqrt(v) of every element, float32 multiples of 2^-16 in [0, 1)."""
    key = _mix(np.array((seed + 0x9E3779B9 * (tensor + 1)) & 0xFFFFFFFF, np.uint32))
    h = _mix(_mix(np.arange(n, dtype=np.uint32)) ^ key)
    return (h & np.uint32(0xFFFF)).astype(np.float32) / np.float32(65536), (h >> np.uint32(16)).astype(np.float32) / np.float32(65536)


def encode(x: np.ndarray, u: np.ndarray, most: int):
    """(codes, scales float32) of float32 values; most 127 signed, 255 not negative."""
    x, u = np.asarray(x, np.float32), np.asarray(u, np.float32)
    codes = np.zeros(len(x), np.int64)
    scales = np.zeros(math.ceil(len(x) / BLOCK), np.float32)
    for k in range(len(scales)):
        at = slice(k * BLOCK, (k + 1) * BLOCK)
        v = x[at]
        if not np.isfinite(v).all():
            scales[k] = np.nan
            continue
        top = np.abs(v).max()
        scales[k] = top
        if top == 0:
            continue
        t = np.sqrt(np.abs(v) / top) * np.float32(most)
        c = np.minimum(np.floor(t + u[at]), most).astype(np.int64)
        if most == 255:
            c = np.where((v > 0) & (c < 1), 1, c)
        codes[at] = np.where(v < 0, -c, c)
    return codes.astype(np.int8 if most == 127 else np.uint8), scales


def decode(codes: np.ndarray, scales: np.ndarray, most: int) -> np.ndarray:
    """float32 values of codes: the integer c |c| times fl(s / most^2)."""
    c = codes.astype(np.float32)
    step = scales / np.float32(most * most)
    return c * np.abs(c) * np.repeat(step, BLOCK)[:len(c)]


def adamw8(p, g, mc, ms, vc, vs, step, lr, b1, b2, eps, wd, seed, tensor, grad_scale=None):
    """One step on 8-bit moments: (p' float64, m codes, m scales, v codes, v scales), moments in float32 as defined."""
    f = np.float32
    g32 = np.asarray(g, f) * f(grad_scale) if grad_scale is not None else np.asarray(g, f)
    m = decode(mc, ms, 127)
    r = decode(vc, vs, 255)
    v = r * r
    p1, _, _ = adamw(p, g32, m, v, step, lr, b1, b2, eps, wd)
    with np.errstate(invalid="ignore", over="ignore"):
        m = m * f(b1) + g32 * f(1 - b1)
        v = v * f(b2) + (g32 * g32) * f(1 - b2)
    um, uv = random_pair(seed, tensor, len(m))
    return (p1, *encode(m, um, 127), *encode(np.sqrt(v), uv, 255))
