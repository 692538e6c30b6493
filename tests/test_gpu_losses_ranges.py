"""Losses on logits over the whole range of their types: rows with a common
offset, rows too long for registers, values next to each other at the top of a
row, and a pair whose difference is infinite. Formulas and bounds are
test_gpu_losses'."""

import pytest
import torch

from test_gpu_losses import (BF16, F32, INF, NINF, _close, _distill_case, _distill_check, _e, _pref_case, _pref_check,
                             _pref_exact)

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


@pytest.mark.parametrize("V", [9, 40, 1500, 9000, 70001])
@pytest.mark.parametrize("sign", [1, -1])
def test_distill_neighbours_of_a_far_maximum(qn, V, sign):
    """Values one to three steps under the maximum where a step is 16 of the
    exponent: 2^-16 of the sum, and the whole of their own gradients."""
    tau = float(torch.tensor(2.7e-6, dtype=F32))
    g = torch.Generator(device="cuda").manual_seed(V)
    # under 512 (or over -512) steps of 2^-15, / tau = 11.3; m log2 e / tau = 2^28.03
    top_value = 512 - 2.0 ** -15 if sign > 0 else -512 + 2.0 ** -15 * 8
    z = top_value - 2.0 ** -15 * torch.randint(0, 4, (6, V), generator=g, device="cuda").double()
    z[:, 3] = top_value
    z = z.float()
    index = torch.randint(0, V, (6, 3), generator=g, device="cuda")
    labels = torch.randint(0, V, (6,), generator=g, device="cuda")
    top = tau * torch.randn(6, 3, generator=g, device="cuda")
    weight = torch.rand(6, generator=g, device="cuda") + 0.1
    _distill_check(qn, z, index, top, None, tau, 0.0, weight)
    z[:, :3] = top_value
    _distill_check(qn, z, index, top, labels, tau, 0.0, None)


@pytest.mark.parametrize("dt,V", [(F32, 20001), (F32, 65540), (F32, 131080), (F32, 128001), (BF16, 140001)])
def test_distill_offset_whose_steps_are_far_apart(qn, dt, V):
    """fp32 logits 16 apart: a neighbour of the maximum is 2^-33 of the sum, and
    has that gradient."""
    z, _, index, top, labels, weight = _distill_case(3, V, 9, dt, seed=V)
    z.add_(1.5e8)
    z[1] = z[1].sort().values
    for tau, alpha in ((1.0, 0.0), (0.7, 0.3), (2.0, 0.0), (1.0, 0.4)):
        _distill_check(qn, z, index, top, labels, tau, alpha, weight)


@pytest.mark.parametrize("top_value", [2.5e8, -2.5e8])
def test_preference_neighbours_of_a_far_maximum(qn, top_value):
    """512 values a step of 16 under the maximum: 5.8e-5 of the sum."""
    z = torch.full((8, 513), top_value - 16, device="cuda")
    at = torch.arange(8, device="cuda")
    z[at, 60 * at] = top_value
    assert bool((z.amin(1) == top_value - 16).all())
    labels = 60 * at
    want = torch.log_softmax(z.double(), 1).gather(1, labels[:, None])[:, 0]
    _close("logp", qn.token_logp(z, labels), want, _e(z) + 2.0 ** -22 * (want.abs() + 40))
    start = torch.tensor([0, 3, 4, 6, 8], device="cuda")
    _pref_check(qn, z, labels, start, torch.randn(4, device="cuda"), torch.rand(2, device="cuda") + 0.5)


def test_preference_smoothing_of_one_at_infinity(qn):
    """A preferred token that is ruled out (x = -inf): with smoothing 1 the loss
    is -log sigmoid(-x) alone, zero there and infinite at x = inf; with 0 the
    other way round. Between them it is infinite."""
    z, _, labels, _, ref, dloss = _pref_case(8, 65, F32, 2, seed=1, masked=0.0)
    start = torch.tensor([0, 2, 4, 6, 8], device="cuda")
    y = z.clone()
    y[0, labels[0]] = NINF  # pair 0: x = -inf
    y[7, labels[7]] = NINF  # pair 1: x = inf
    for smooth, want in ((1.0, (0.0, INF)), (0.0, (INF, 0.0)), (0.5, (INF, INF))):
        loss, L, st = qn.preference_loss_fwd(y, labels, start, ref, 0.3, smooth)
        assert loss.tolist() == list(want)
        dz = qn.preference_loss_bwd(y, labels, st, dloss)
        assert bool(dz.isfinite().all())
        for i in range(2):  # its slope is beta or nothing
            assert bool(dz[4 * i:4 * i + 4].any()) == (want[i] == INF)
    _pref_check(qn, z, labels, start, ref, dloss, 0.3, 1.0)


@pytest.mark.parametrize("V", [300, 1500, 4097, 9000, 20001, 60001, 70001])
@pytest.mark.parametrize("offset", [1e3, -1e5])
def test_a_common_offset(qn, V, offset):
    """The same offset on every logit, each way a row is dealt out: nothing but
    the offset's own rounding of the inputs changes."""
    z, _, index, top, labels, weight = _distill_case(4, V, 9, F32, seed=V)
    z.add_(offset)
    for tau, alpha in ((1.0, 0.0), (1.0, 0.3), (0.7, 0.3)):
        _distill_check(qn, z, index, top, labels, tau, alpha, weight)
    z, _, labels, start, ref, dloss = _pref_case(6, V, F32, 1, seed=V, masked=0.2)
    z.add_(offset)
    on = labels >= 0
    want = torch.where(on, torch.log_softmax(z.double(), 1).gather(1, labels.clamp(min=0)[:, None])[:, 0], 0.0)
    _close("logp", qn.token_logp(z, labels), want, _e(z) + 2.0 ** -22 * (want.abs() + 40))
    _pref_check(qn, z, labels, start, ref, dloss)


def test_preference_of_more_than_2_to_the_31_logits(qn):
    """Offsets past 32 bits in the sums and in the gradient, which is written in
    the logits' place from the last row to the first: rows on both sides of
    2^31."""
    T, V = 17000, 128002
    z = torch.empty(T, V, dtype=BF16, device="cuda")
    g = torch.Generator(device="cuda").manual_seed(0)
    for part in z.split(1000):
        part.copy_(2 * torch.randn(part.shape, generator=g, device="cuda"))
    labels = torch.randint(0, V, (T,), generator=g, device="cuda")
    labels[100:16700] = -100
    # pair 0: the first rows, pair 1: those around 2^31, and both in pair 2's second sequence
    start = torch.tensor([0, 40, 100, 16770, 16777, 16800, 17000], device="cuda")
    rows = torch.cat([torch.arange(100, device="cuda"), torch.arange(16700, T, device="cuda")])
    ends = torch.tensor([0, 40, 100, 170, 177, 200, 400], device="cuda")
    ref = -12.0 * (ends[1:] - ends[:-1]).float() + torch.randn(6, generator=g, device="cuda")
    dloss = torch.rand(3, generator=g, device="cuda") + 0.2
    zr, lr = z[rows], labels[rows]
    want, tol = _pref_exact(zr, lr, ends, ref, 0.01, 0.1, "sigmoid", False, dloss)
    loss, L, st = qn.preference_loss_fwd(z, labels, start, ref, 0.01, 0.1)
    _close("L", L, want["L"], tol["L"])
    _close("loss", loss, want["loss"], tol["loss"])
    dz = qn.preference_loss_bwd(z, labels, st, dloss, dlogits=z)
    assert dz is z
    _close("dz", z[rows], want["dz"], tol["dz"])
    assert not any(bool(part.any()) for part in z[100:16700].split(1000))
