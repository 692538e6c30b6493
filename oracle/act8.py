"""8-bit activation checkpoints and the gated activation (CPU oracle).

Test infrastructure only (see the package docstring). Blocks of 32 values of
a row share one scale 2^k, k the least integer with a 2^-k <= 448 (a the
largest finite magnitude) and at least -124; the values are the nearest
E4M3FN codes, ties to an even mantissa; NaN and infinities are stored as NaN.
Everything is computed in fp64 from the real-number definition.
"""

import numpy as np

BLOCK = 32
LOWEST = -124  # the restored values' last place is then at least 2^-133


def block_exponent(a):
    """Least integer k with a 2^-k <= 448, at least -124, for finite a >= 0."""
    a = np.asarray(a, dtype=np.float64)
    m, e = np.frexp(a)  # a = m 2^e, m in [1/2, 1); 448 = 0.875 2^9
    k = np.where(m > 0.875, e - 8, e - 9)
    return np.where(a > 0, np.maximum(k, LOWEST), LOWEST).astype(np.int64)


def e4m3_nearest(y):
    """The E4M3FN value nearest to y (|y| <= 448), ties to an even mantissa."""
    y = np.asarray(y, dtype=np.float64)
    step = np.ldexp(1.0, np.maximum(np.frexp(y)[1] - 1, -6) - 3)
    return np.rint(y / step) * step


def act8_exponents(X):
    """k per block of 32 along the last axis of X."""
    X = np.asarray(X, dtype=np.float64)
    v = X.reshape(X.shape[0], -1, BLOCK)
    return block_exponent(np.where(np.isfinite(v), np.abs(v), 0.0).max(axis=2))


def act8_restore(X):
    """The values an 8-bit checkpoint of X stands for (fp64, NaN for non-finite)."""
    X = np.asarray(X, dtype=np.float64)
    v = X.reshape(X.shape[0], -1, BLOCK)
    k = act8_exponents(X)[:, :, None]
    fin = np.isfinite(v)
    y = np.ldexp(e4m3_nearest(np.ldexp(np.where(fin, v, 0.0), -k)), k)
    # magnitudes from 1.9375 2^127 on round up to 2^128, infinite in bf16 and fp32
    y = np.where(np.abs(y) >= 2.0 ** 128, np.copysign(np.inf, y), y)
    return np.where(fin, y, np.nan).reshape(X.shape)


def swiglu(gate, up):
    """g sigmoid(g) u in fp64."""
    g, u = np.asarray(gate, np.float64), np.asarray(up, np.float64)
    with np.errstate(over="ignore"):
        return g / (1.0 + np.exp(-g)) * u


def swiglu_backward(gate, up, dH):
    """(dgate, dup) of swiglu in fp64."""
    g, u, d = (np.asarray(t, np.float64) for t in (gate, up, dH))
    with np.errstate(over="ignore"):
        p = 1.0 / (1.0 + np.exp(-g))
    return d * u * p * (1.0 + g * (1.0 - p)), d * g * p
