"""Microscaled 4-bit floating point of rotated rows, and its product.

Sources:
  [P1] intro: the rotation offline on the weights and online on the
       activations, dynamic quantization (here in another number format).
  OCP Microscaling Formats (MX) v1.0: E2M1 elements, a power of two (E8M0) per
       32 of them, the power of the block's largest magnitude.

Definitions, per 32 consecutive columns of the orthonormally rotated values v:
  A = max |v|;  b = max(floor(log2 A) - 2 + 127, 0), 0 for A = 0
  code = sign and the nearest of 0, .5, 1, 1.5, 2, 3, 4, 6 to |v| 2^(127 - b),
         halfway between two the one whose code is even, 6 for all beyond
  value = 2^(b - 127) times that number
  A block with an infinity or NaN: b = 255, codes 0, value NaN.
The rotation's sums round to float32 one by one (hadamard.rotate); the factor
1 / sqrt(n) is exact.
Layout: tiles of 128 columns, codes [tiles][rows][64] (even column in the low
nibble), bytes [tiles][rows][4]; columns behind K are zeros with b = 0.
"""
from __future__ import annotations

import math

import numpy as np

from . import hadamard

GRID = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0)


def nearest_code(a: float) -> int:
    """Code of a magnitude in units of the block's power of two."""
    best, at = math.inf, 0
    for c, g in enumerate(GRID):
        d = abs(a - g)
        if d < best or (d == best and c % 2 == 0):
            best, at = d, c
    return at


_EDGES = [(GRID[c] + GRID[c + 1]) / 2 for c in range(7)]


def quantize(x: np.ndarray, rot_group: int = 0):
    """x float32 [rows, K] -> (codes uint8 [rows, K], bytes uint8 [rows, K/32])."""
    v = np.asarray(x, np.float32)
    rows, K = v.shape
    if rot_group:
        with np.errstate(invalid="ignore", over="ignore"):
            v = hadamard.rotate(v, rot_group)
    v = v.astype(np.float64) / math.sqrt(rot_group or 1)
    v = v.reshape(rows, K // 32, 32)
    bad = ~np.isfinite(v).all(-1)
    v = np.where(bad[..., None], 0.0, v)
    top = np.abs(v).max(-1)
    power = np.frexp(top)[1] - 1
    byte = np.where(top > 0, np.maximum(power - 2 + 127, 0), 0)
    a = np.abs(v) * np.exp2(127.0 - byte)[..., None]
    code = np.zeros(a.shape, np.int64)
    for c, edge in enumerate(_EDGES):
        code += (a >= edge) if (c + 1) % 2 == 0 else (a > edge)
    code = np.where((v < 0) & (code > 0), code + 8, code)
    byte = np.where(bad, 255, byte)
    code = np.where(bad[..., None], 0, code)
    return code.reshape(rows, K).astype(np.uint8), byte.astype(np.uint8)


def values(codes: np.ndarray, byte: np.ndarray) -> np.ndarray:
    """float64 [rows, K] of codes [rows, K] and bytes [rows, K/32]."""
    grid = np.array(GRID + tuple(-g for g in GRID))
    unit = np.where(byte == 255, np.nan, np.exp2(byte.astype(np.float64) - 127))
    return grid[codes] * np.repeat(unit, 32, axis=1)


def dequantize(codes: np.ndarray, byte: np.ndarray, rot_group: int = 0) -> np.ndarray:
    """The values, rotated back in float64."""
    v = values(codes, byte)
    if rot_group:
        rows, K = v.shape
        h = hadamard.regular_hadamard(rot_group).astype(np.float64)
        v = (v.reshape(-1, rot_group) @ h.T).reshape(rows, K) / math.sqrt(rot_group)
    return v


def pack(codes: np.ndarray, byte: np.ndarray):
    """The tiled layout of codes [rows, K] and bytes [rows, K/32]."""
    rows, K = codes.shape
    tiles = -(-K // 128)
    c = np.zeros((rows, tiles * 128), np.uint8)
    c[:, :K] = codes
    b = np.zeros((rows, tiles * 4), np.uint8)
    b[:, :K // 32] = byte
    two = c[:, 0::2] | (c[:, 1::2] << 4)
    return (np.ascontiguousarray(two.reshape(rows, tiles, 64).transpose(1, 0, 2)),
            np.ascontiguousarray(b.reshape(rows, tiles, 4).transpose(1, 0, 2)))


def unpack(codes: np.ndarray, byte: np.ndarray, K: int):
    """Inverse of pack."""
    tiles, rows, _ = codes.shape
    two = codes.transpose(1, 0, 2).reshape(rows, tiles * 64)
    c = np.stack([two & 15, two >> 4], -1).reshape(rows, tiles * 128)
    return c[:, :K], byte.transpose(1, 0, 2).reshape(rows, tiles * 4)[:, :K // 32]


def gemm(a: np.ndarray, w: np.ndarray, bias=None):
    """(a w^T + bias in float64, sum_k |a w|) of values [M, K] and [N, K]."""
    y, mag = a @ w.T, np.abs(a) @ np.abs(w).T
    if bias is not None:
        y, mag = y + bias, mag + np.abs(bias)
    return y, mag
