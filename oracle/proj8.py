"""8-bit projections of a layer: float64 oracle.

TEST INFRASTRUCTURE ONLY (tests and the smoke check).

Storage rule: a block of values shares the scale max(amax / 448, 2^-126), a
value's code is value / scale rounded to the nearest e4m3 number (ties to
even). Activations have a scale per row and 128 channels, weights one per
128 x 128 block; the last block of a row or column may be cut.
"""
from __future__ import annotations

import numpy as np

from . import dequantize, f64, quantize_e4m3

BLOCK = 128


def blocks(n: int) -> int:
    return -(-n // BLOCK)


def quantize_rows(v):
    """Codes (uint8 [rows, d]) and scales (float32 [rows, ceil(d / 128)])."""
    v = np.asarray(v, dtype=np.float64)
    rows, d = v.shape
    p = np.zeros((rows, blocks(d) * BLOCK))
    p[:, :d] = v
    codes, scales = quantize_e4m3(p, BLOCK)
    return np.ascontiguousarray(codes[:, :d]), scales


def quantize_weight(W):
    """Codes (uint8 [N, K]) and scales (float32 [ceil(N / 128), ceil(K / 128)])."""
    W = f64(W)
    N, K = W.shape
    nb, kb = blocks(N), blocks(K)
    p = np.zeros((nb * BLOCK, kb * BLOCK))
    p[:N, :K] = W
    # one row per 128 x 128 block
    t = p.reshape(nb, BLOCK, kb, BLOCK).transpose(0, 2, 1, 3).reshape(nb * kb, BLOCK * BLOCK)
    codes, scales = quantize_e4m3(t, BLOCK * BLOCK)
    codes = codes.reshape(nb, kb, BLOCK, BLOCK).transpose(0, 2, 1, 3).reshape(p.shape)
    return np.ascontiguousarray(codes[:N, :K]), scales.reshape(nb, kb)


def row_values(codes, scales):
    """Float64 values of stored activations."""
    c = np.asarray(codes)
    rows, d = c.shape
    p = np.zeros((rows, blocks(d) * BLOCK), dtype=np.uint8)
    p[:, :d] = c
    return dequantize(p, scales, BLOCK)[:, :d]


def weight_values(codes, scales):
    """Float64 values of a stored weight."""
    c = np.asarray(codes)
    N = c.shape[0]
    per_row = np.repeat(np.asarray(scales, dtype=np.float32), BLOCK, axis=0)[:N]
    return row_values(c, per_row)


def add_norm(x, residual=None, gamma=None, normalise: bool = True, eps: float = 1e-6):
    """(total, v) in float64: the sum, and its RMSNorm (or the sum itself)."""
    s = f64(x)
    if residual is not None:
        s = s + f64(residual)
    v = s
    if normalise:
        v = s / np.sqrt((s * s).mean(axis=-1, keepdims=True) + eps)
        if gamma is not None:
            v = v * f64(gamma)
    return s, v


def fp8_proj(A, A_scale, W, W_scale, groups: int = 1):
    """r [M, groups N] in float64 of stored operands, group by group."""
    a, w = row_values(A, A_scale), weight_values(W, W_scale)
    N, K = w.shape[0] // groups, w.shape[1]
    return np.concatenate([a[:, g * K:(g + 1) * K] @ w[g * N:(g + 1) * N].T
                           for g in range(groups)], axis=1)
