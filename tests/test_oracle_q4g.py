"""The 4-bit group quantization of the oracle: worked examples, invariants
and brute force over the sixteen values."""

import numpy as np
import pytest

from oracle import q4g


def test_worked_group():
    w = np.zeros((1, 32), np.float32)
    w[0, :5] = [-3.0, 12.0, 0.5, 1.5, -0.4]
    q, s, z = q4g.quantize(w, 32, False)
    assert s[0, 0] == 1.0 and z[0, 0] == 3
    # 0.5 and 1.5 are ties: to the even integers 0 and 2
    assert list(q[0, :6]) == [0, 15, 3, 5, 3, 3]
    q, s, z = q4g.quantize(w[:, [0, 4] + [8] * 30], 32, True)
    assert z[0, 0] == 8 and s[0, 0] == np.float32(219 / 512)  # 3 / 7 = 219.43 / 512, bf16 steps of 1 / 512 there
    assert q[0, 0] == 1 and q[0, 1] == 7 and q[0, 2] == 8


def test_packing():
    q = np.arange(40).reshape(1, 40) % 16
    p = q4g.pack(q)
    assert p.shape == (1, 32) and p[0, 0] == 0x01 and p[0, 7] == 0xEF and not p[0, 20:].any()


@pytest.mark.parametrize("sym", [False, True])
@pytest.mark.parametrize("bf16", [False, True])
@pytest.mark.parametrize("group", [32, 64, 128])
def test_nearest_of_the_sixteen_values(sym, bf16, group):
    rng = np.random.default_rng(group)
    W = rng.normal(0, 0.02, (7, 200)).astype(np.float32)
    q, s, z = q4g.quantize(W, group, sym, bf16)
    at = np.arange(200) // group
    grid = s[:, at, None].astype(np.float64) * (np.arange(16)[None, None, :] - z[:, at, None])
    d = np.abs(grid - W[:, :, None])
    got = np.take_along_axis(d, q[:, :, None], axis=2)[:, :, 0]
    assert np.all(got <= d.min(axis=2) * (1 + 1e-5))
    # inside the grid a value is at most half a step away; the scale's rounding
    # (2^-8 of 15 steps) may leave the ends outside by a little
    assert np.all(got <= s[:, at] * (0.5 + 15 * 2.0 ** -8))


def test_zero_is_a_grid_value_and_zero_groups():
    W = np.zeros((3, 64), np.float32)
    W[1, :32] = np.linspace(2, 3, 32)  # all of one sign: the range takes 0 in
    q, s, z = q4g.quantize(W, 32, False)
    assert s[0, 0] == 0 and z[0, 0] == 8 and np.all(q[0] == 8)
    assert z[1, 0] == 0 and s[1, 0] > 0
    assert np.all(q4g.dequantize(q, s, z, 32)[[0, 2]] == 0)
    tiny = np.full((1, 32), 2.0 ** -130, np.float32)
    assert q4g.quantize(tiny, 32, True)[1][0, 0] == 0


def test_linear_is_the_dequantized_product():
    rng = np.random.default_rng(5)
    q, s, z = q4g.quantize(rng.normal(size=(9, 72)).astype(np.float32), 32, False, False)
    X = rng.normal(size=(4, 72))
    y, mag = q4g.linear(X, q, s, z, 32)
    w = q4g.dequantize(q, s, z, 32).astype(np.float64)
    assert np.allclose(y, X @ w.T, rtol=1e-6, atol=1e-6) and np.all(mag >= np.abs(y) * (1 - 1e-12))
