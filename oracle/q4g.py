"""4-bit weights with group scales (CPU oracle).

Test infrastructure only (see the package docstring). Codes, scales and zero
points are decided in fp32, step by step as the definition says (NumPy's fp32
operations are correctly rounded); products are fp64.
"""

import numpy as np

from .nf4 import bf16_bits_to_f32, f32_to_bf16_bits

F = np.float32


def _round_scale(s, bf16):
    return bf16_bits_to_f32(f32_to_bf16_bits(s)).astype(F) if bf16 else s


def quantize(W, group, symmetric, bf16_scale=True):
    """(codes [N, K], scale [N, groups] fp32 values, zero [N, groups]) of a
    fp32 W. Group by group, the last of a row may be shorter."""
    W = np.asarray(W, dtype=F)
    N, K = W.shape
    n = -(-K // group)
    codes = np.zeros((N, K), np.int64)
    scale, zero = np.zeros((N, n), F), np.full((N, n), 8, np.int64)
    for j in range(n):
        w = W[:, j * group:(j + 1) * group]
        hi, lo = np.maximum(w.max(axis=1), F(0)), np.minimum(w.min(axis=1), F(0))
        s = np.maximum(hi, -lo) / F(7) if symmetric else (hi - lo) / F(15)
        s = _round_scale(s.astype(F), bf16_scale)
        live = s >= F(2.0 ** -126)
        d = np.where(live, s, F(1)).astype(F)
        z = np.full(N, 8.0, F) if symmetric else np.minimum(np.rint(-lo / d), F(15))
        q = np.clip(np.rint(w / d[:, None]) + z[:, None], 0, 15)
        codes[:, j * group:(j + 1) * group] = np.where(live[:, None], q, 8)
        scale[:, j] = np.where(live, s, F(0))
        zero[:, j] = np.where(live, z, 8)
    return codes, scale, zero


def pack(codes):
    """uint8 [N, 16 ceil(K/32)]: element e in byte e/2, even e in the high nibble."""
    N, K = codes.shape
    full = np.zeros((N, -(-K // 32) * 32), np.uint8)
    full[:, :K] = codes
    return (full[:, 0::2] << 4 | full[:, 1::2]).astype(np.uint8)


def dequantize(codes, scale, zero, group):
    """w' = fl32(s (q - z)) as fp32 values."""
    at = np.arange(codes.shape[1]) // group
    return (scale[:, at] * (codes - zero[:, at]).astype(F)).astype(F)


def linear(X, codes, scale, zero, group):
    """X W'^T in fp64, W' unrounded, and the sum of the magnitudes s (q + z) |x|
    that a computation on separate sums of q x and z x goes through."""
    X = np.asarray(X, np.float64)
    at = np.arange(codes.shape[1]) // group
    s = scale.astype(np.float64)[:, at]
    return X @ (s * (codes - zero[:, at])).T, np.abs(X) @ (np.abs(s) * (codes + zero[:, at])).T
