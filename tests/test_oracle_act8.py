"""The 8-bit activation checkpoint of the oracle, pinned by torch's own
E4M3FN cast, by brute force over the code values and by worked examples."""

import numpy as np
import torch

import oracle
from oracle import act8


def test_nearest_value_matches_torch_cast():
    rng = np.random.default_rng(1)
    y = np.concatenate([rng.normal(0, 100, 20000).clip(-448, 448), rng.normal(0, 0.01, 20000),
                        np.ldexp(rng.integers(-2 ** 9, 2 ** 9, 4000), -12)]).astype(np.float32)
    want = torch.from_numpy(y).to(torch.float8_e4m3fn).float().numpy()
    assert np.array_equal(act8.e4m3_nearest(y), want)


def test_nearest_value_is_the_closest_code():
    table = oracle.e4m3fn_value_table()
    table = np.unique(table[np.isfinite(table)])
    rng = np.random.default_rng(2)
    y = rng.uniform(-448, 448, 3000)
    best = np.abs(table[None, :] - y[:, None]).min(axis=1)
    got = act8.e4m3_nearest(y)
    assert np.all(np.isin(got, table)) and np.array_equal(np.abs(got - y), best)


def test_exponent_is_the_least_that_fits():
    rng = np.random.default_rng(3)
    a = np.abs(rng.normal(0, 1, 2000)) * 2.0 ** rng.integers(-100, 100, 2000)
    a = np.concatenate([a, 448 * 2.0 ** np.arange(-20, 20), 448.0001 * 2.0 ** np.arange(-20, 20)])
    k = act8.block_exponent(a)
    assert np.all(a * 2.0 ** -k <= 448)
    assert np.all((a * 2.0 ** (1.0 - k) > 448) | (k == act8.LOWEST))
    assert act8.block_exponent(0.0) == -124 and act8.block_exponent(2.0 ** -133) == -124


def test_worked_block():
    x = np.zeros((1, 32))
    x[0, 0], x[0, 1], x[0, 2], x[0, 3] = 448.0, 449.0, 17.0, -0.001
    # 449 > 448: k = 1, values halved: 224.5 -> 224 -> 448; 8.5 -> 8 (tie to even) -> 16
    assert act8.act8_exponents(x)[0, 0] == 1
    got = act8.act8_restore(x)[0]
    assert got[0] == 448.0 and got[1] == 448.0 and got[2] == 16.0
    assert got[3] == 0.0  # 0.0005 is under half the smallest step 2^-9


def test_non_finite_values_become_nan_and_leave_the_scale():
    x = np.ones((1, 64))
    x[0, 3], x[0, 40], x[0, 41] = np.inf, np.nan, -np.inf
    got = act8.act8_restore(x)[0]
    bad = np.zeros(64, bool)
    bad[[3, 40, 41]] = True
    assert np.array_equal(np.isnan(got), bad) and np.all(got[~bad] == 1.0)


def test_restored_values_are_exact_in_bf16():
    rng = np.random.default_rng(4)
    x = torch.from_numpy(rng.normal(0, 1, (64, 64)) * 2.0 ** rng.integers(-133, 100, (64, 1))).to(torch.bfloat16)
    got = act8.act8_restore(x.double().numpy())
    assert np.array_equal(torch.from_numpy(got).to(torch.bfloat16).double().numpy(), got)


def test_swiglu_backward_against_autograd_and_differences():
    g = torch.randn(5, 32, dtype=torch.float64, requires_grad=True)
    u = torch.randn(5, 32, dtype=torch.float64, requires_grad=True)
    d = torch.randn(5, 32, dtype=torch.float64)
    h = g * torch.sigmoid(g) * u
    dg, du = torch.autograd.grad(h, (g, u), d)
    gn, un, dn = g.detach().numpy(), u.detach().numpy(), d.numpy()
    assert np.allclose(act8.swiglu(gn, un), h.detach().numpy(), rtol=1e-14)
    og, ou = act8.swiglu_backward(gn, un, dn)
    assert np.allclose(og, dg.numpy(), rtol=1e-12, atol=1e-14) and np.allclose(ou, du.numpy(), rtol=1e-12)
    e = 1e-6
    num = (act8.swiglu(gn + e, un) - act8.swiglu(gn - e, un)) / (2 * e) * dn
    assert np.allclose(og, num, rtol=1e-7, atol=1e-8)
