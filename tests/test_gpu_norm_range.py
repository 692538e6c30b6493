"""Norms of rows whose squares leave fp32's range, and without eps: the formula
where it is finite. Formulas and bounds are test_gpu_norm's."""

import pytest
import torch

from test_gpu_norm import BF16, E, F32, _close, _exact, _inputs

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def qn():
    import bit_nf4_quantized_16_amd as qn

    assert torch.cuda.is_available()
    return qn


# one wave a row, several, two and four pieces a lane
@pytest.mark.parametrize("xt,C", [(F32, 8), (F32, 264), (BF16, 520), (F32, 4096), (BF16, 8192), (F32, 16384), (BF16, 16384)])
@pytest.mark.parametrize("rms", [False, True])
@pytest.mark.parametrize("eps", [0.0, 1e-5, 1e-40])
def test_rows_of_any_size(qn, xt, C, rms, eps):
    """Rows of 1e-37 to 1e37, ordinary ones between them. In fp32 a row under
    1e-19 has squares that are rounded to nothing, one over 1e19 infinite ones."""
    eps = float(torch.tensor(eps, dtype=F32))
    sizes = [1.0, 1e-37, 1e-30, 1e-23, 1e-20, 1e-16, 1.0, 1e12, 1e18, 1e20, 1e28, 1e37, 1.0]
    X, w, b, dY = _inputs(len(sizes), C, xt, F32, seed=C)
    X = (X.double() * torch.tensor(sizes, device="cuda").double()[:, None]).to(xt)
    want, tol = _exact(X, w, b, dY, eps, rms)
    Y, mean, rstd = qn.norm_fwd(X, w, b, eps, rms)
    _close("Y", Y, want["y"], tol["y"])
    _close("rstd", rstd, want["r"], E * want["r"])
    if not rms:
        _close("mean", mean, want["mu"], E * X.double().abs().mean(1))
    dX = qn.norm_bwd(X, w, dY, mean, rstd, need_dw=False, need_db=False)[0]
    _close("dX", dX, want["dx"], tol["dx"] + 2.0 ** -126)
    # a row's neighbours are what they are without it
    ones = torch.tensor([0, 6, 12], device="cuda")
    alone = qn.norm_fwd(X[ones], w, b, eps, rms)
    assert torch.equal(alone[0], Y[ones]) and torch.equal(alone[2], rstd[ones])


@pytest.mark.parametrize("C", [264, 4096])
def test_rows_that_have_no_norm(qn, C):
    """Without eps a row of zeros (or of one value) is 0 / 0; NaN and infinite
    values stay what they were."""
    X, w, b, _ = _inputs(6, C, F32, F32, seed=1)
    X[1] = 0.0
    X[2, 5], X[3, 5], X[4, 5] = float("nan"), float("inf"), float("-inf")
    for rms in (True, False):
        Y, _, rstd = qn.norm_fwd(X, w, b, 0.0, rms)
        assert bool(Y[1].isnan().all()) and bool(Y[2].isnan().all())
        assert bool(Y[3:5, 5].isnan().all()) and bool(Y[[0, 5]].isfinite().all())
        if rms:  # finite values over an infinite root
            keep = torch.arange(C, device="cuda") != 5
            assert torch.equal(Y[3:5, keep], b[keep].expand(2, -1))
        Y1, _, _ = qn.norm_fwd(X, w, b, 1e-5, rms)
        assert torch.equal(Y1[1], b) and bool(Y1[2].isnan().all())
