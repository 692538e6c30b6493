"""Codes of groups whose scale is small, down to fp32's smallest normal number:
the nearest of fl32(w / s) as everywhere, at values on and beside the ties."""

import numpy as np
import pytest
import torch

from oracle import q4g as og

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def qn():
    import bit_nf4_quantized_16_amd as qn

    assert torch.cuda.is_available()
    return qn


def _near_ties(rows, group, exponent, sym, seed):
    """fp32 rows of one group: values within three places of (k + 1/2) s, the
    ends set so that the range is about 15 s (7 s to each side, symmetric)."""
    rng = np.random.default_rng(seed)

    def beside(v):
        bits = v.astype(np.float32).view(np.int32)
        return np.where(bits & 0x7FFFFFFF, bits + rng.integers(-3, 4, bits.shape).astype(np.int32), bits).view(np.float32)

    s = np.ldexp(rng.uniform(1, 2, (rows, 1)), exponent)
    k = rng.integers(-6, 7, (rows, group)) + 0.5
    w = beside(k * s)
    w[:, :1] = (7 * s if sym else 8 * s).astype(np.float32)
    w[:, 1:2] = -7 * s
    # the range found is rounded: the ties of the scale that is kept
    kept = og.quantize(w, group, sym, False)[1].astype(np.float64)
    w[:, 2:] = beside(k * kept)[:, 2:]
    return w


@pytest.mark.parametrize("sym", [False, True])
@pytest.mark.parametrize("group", [32, 64, 128])
@pytest.mark.parametrize("exponent", [-127, -126, -125, -123, -120, -116, -110, -103, -80, -65, -64, -63, -20, 20, 100, 123])
def test_codes_beside_the_ties(qn, sym, group, exponent):
    W = _near_ties(512, group, exponent, sym, 200 + exponent + group)
    for sd in (torch.float32, torch.bfloat16):
        for bf in (False, True):
            X = torch.from_numpy(W)
            X = X.bfloat16() if bf else X
            w = qn.q4g_quantize(X.cuda(), group=group, symmetric=sym, scale_dtype=sd)
            q, s, z = og.quantize(X.float().numpy(), group, sym, sd == torch.bfloat16)
            assert np.array_equal(w.scale.float().cpu().numpy(), s)
            assert sym or np.array_equal(w.zero.cpu().numpy(), z)
            assert np.array_equal(w.packed.cpu().numpy(), og.pack(q))
