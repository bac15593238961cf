"""Batched low-rank adapters and 8-bit activation checkpoints, in float64.

Sources:
  [P2] passage on LoRA merge versus bypass: a delta kept as a separate branch
       beside the quantized weight; here each segment of rows names its own
       adapter, and the branch has gradients.
  [P3] Kernel Engineering: the quantized MLP around its GELU.

Definitions:
  la[m]  = x[m] down[a]^T;  out[m] = base[m] + c[a] la[m] up[a]^T
  dla[m] = c[a] dy[m] up[a];  dx[m] = dx_base[m] + dla[m] down[a]
  d_up[a] = c[a] sum_m dy[m]^T la[m];  d_down[a] = sum_m dla[m]^T x[m]
  a is the adapter of the segment that holds row m; rows outside every
  segment, and of segments whose number is not 0..A-1, have none.
  y = act(z); dz = dy act'(s q) with (q, s) the symmetric 8-bit codes of z per
  row and 64 columns (quant.quantize_sym).
"""
from __future__ import annotations

import math

import numpy as np
from scipy.special import erfc, expit

from . import hadamard, quant


def row_adapters(offsets, ids, M: int, A: int) -> np.ndarray:
    """Adapter of every row, -1 for none."""
    rows = np.full(M, -1, dtype=np.int64)
    for s, a in enumerate(ids):
        lo, hi = int(offsets[s]), int(offsets[s + 1])
        if 0 <= a < A:
            rows[lo:hi] = a
    return rows


def _scales(scale, A):
    return np.ones(A) if scale is None else np.asarray(scale, np.float64)


def lora_forward(x, down, up, offsets, ids, scale=None, base=None):
    """Returns (out [M, N], lora_act [M, R]) in float64."""
    x, down, up = (np.asarray(v, np.float64) for v in (x, down, up))
    M, (A, N, R) = x.shape[0], up.shape
    c = _scales(scale, A)
    rows = row_adapters(offsets, ids, M, A)
    la = np.zeros((M, R))
    out = np.zeros((M, N)) if base is None else np.array(base, np.float64)
    for a in range(A):
        at = rows == a
        la[at] = x[at] @ down[a].T
        out[at] += c[a] * (la[at] @ up[a].T)
    return out, la


def lora_backward(dy, la, x, down, up, offsets, ids, scale=None, dx_base=None):
    """Returns (dx [M, K], d_down [A, R, K], d_up [A, N, R], dla [M, R]) in float64."""
    dy, la, x, down, up = (np.asarray(v, np.float64) for v in (dy, la, x, down, up))
    M, (A, R, K) = dy.shape[0], down.shape
    c = _scales(scale, A)
    rows = row_adapters(offsets, ids, M, A)
    dla = np.zeros((M, R))
    dx = np.zeros((M, K)) if dx_base is None else np.array(dx_base, np.float64)
    d_down, d_up = np.zeros(down.shape), np.zeros(up.shape)
    for a in range(A):
        at = rows == a
        dla[at] = c[a] * (dy[at] @ up[a])
        dx[at] += dla[at] @ down[a]
        d_up[a] = c[a] * (dy[at].T @ la[at])
        d_down[a] = dla[at].T @ x[at]
    return dx, d_down, d_up, dla


def restore_input(codes, scales, rot_group: int) -> np.ndarray:
    """The input that rotated INT8 codes stand for: (s q) H / sqrt(n) per group
    of n columns (H / sqrt(n) is symmetric and its own inverse)."""
    codes = np.asarray(codes, np.float64)
    M, K = codes.shape
    s = np.asarray(scales, np.float64).reshape(-1, 1)
    H = hadamard.regular_hadamard(rot_group).astype(np.float64) / math.sqrt(rot_group)
    return ((codes * s).reshape(-1, rot_group) @ H).reshape(M, K)


def act_value(z, act: str):
    z = np.asarray(z, np.float64)
    if act == "gelu":
        return z * erfc(-z / math.sqrt(2)) / 2
    if act == "gelu_tanh":
        return z * expit(2 * math.sqrt(2 / math.pi) * (z + 0.044715 * z ** 3))
    C = z.shape[1] // 2
    return z[:, :C] * expit(z[:, :C]) * z[:, C:]


def act_backward(dy, z, act: str):
    dy, z = np.asarray(dy, np.float64), np.asarray(z, np.float64)
    if act == "gelu":
        return dy * (erfc(-z / math.sqrt(2)) / 2 + z * np.exp(-z * z / 2) / math.sqrt(2 * math.pi))
    if act == "gelu_tanh":
        a, b = 2 * math.sqrt(2 / math.pi), 0.044715
        p, q = expit(a * (z + b * z ** 3)), expit(-a * (z + b * z ** 3))
        return dy * (p + z * p * q * a * (1 + 3 * b * z * z))
    C = z.shape[1] // 2
    g, u = z[:, :C], z[:, C:]
    p = expit(g)
    return np.concatenate([dy * u * p * (1 + g * expit(-g)), dy * g * p], axis=1)


def checkpoint(z_f32):
    """(codes int8 [rows, W], scales float32 [rows, W / 64]) of float32 values
    that are bf16 numbers."""
    return quant.quantize_sym(np.asarray(z_f32, np.float32), quant.QMAX_INT8, "row_group", 64)


def restore_checkpoint(codes, scales) -> np.ndarray:
    return quant.dequant_sym(codes, scales, "row_group", 64)
