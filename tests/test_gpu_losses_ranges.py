"""Losses on logits over the whole range of their types: rows with a common
offset, rows too long for registers, values next to each other at the top of a
row, and a pair whose difference is infinite. Formulas and bounds are
test_gpu_losses'."""

import pytest
import torch

from test_gpu_losses import BF16, F32, _distill_case, _distill_check

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def qn():
    import bit_nf4_quantized_16_amd as qn

    assert torch.cuda.is_available()
    return qn


@pytest.mark.parametrize("dt,V", [(F32, 65540), (F32, 131080), (F32, 128001), (BF16, 140001)])
@pytest.mark.parametrize("offset", [1e4, 1e5, -1e6, 1e7])
def test_distill_long_rows_far_from_zero(qn, dt, V, offset):
    """Rows that are read in turns, with a running sum of each thread: its
    maximum rises many times, by the order of the values, and the offset's
    rounding with it."""
    z, _, index, top, labels, weight = _distill_case(3, V, 9, dt, seed=V)
    z.add_(offset)
    z[1] = z[1].sort().values  # a new maximum at nearly every turn
    for tau, alpha in ((1.0, 0.0), (0.7, 0.3), (2.0, 0.0), (1.0, 0.4)):
        _distill_check(qn, z, index, top, labels, tau, alpha, weight)
