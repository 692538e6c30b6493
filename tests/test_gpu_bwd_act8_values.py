"""Infinite and NaN operands of the adapter gradients from a checkpoint: dB and
dA hold what the sums over the tokens hold, not NaN from the split of U and G
into terms, some of which are zero."""

import pytest
import torch

import workloads

pytestmark = pytest.mark.gpu

INF = float("inf")


@pytest.fixture(scope="module")
def qn():
    import bit_nf4_quantized_16_amd as qn

    assert torch.cuda.is_available()
    return qn


# ranks: terms split in the kernel (to 16), prepared (over 16), two steps over
# the rank tiles (over 64; 80 leaves the second one short); over 2048 tokens
# the sums come in parts
RANKS = [3, 8, 16, 24, 64, 80, 128]


def _layer(qn, T, N, K, r, seed=0):
    w = qn.quantize_weight(workloads.normal_weight(N, K, 0.02, seed).cuda())
    X = workloads.bf16_normal((T, K), 1.0, seed + 1).cuda()
    dY = workloads.bf16_normal((T, N), 1.0, seed + 2).cuda()
    A = workloads.bf16_normal((r, K), 0.05, seed + 3).cuda()
    B = workloads.bf16_normal((N, r), 0.05, seed + 4).cuda()
    return w, X, dY, A, B


@pytest.mark.parametrize("r", RANKS)
@pytest.mark.parametrize("T", [9, 300, 2100])
def test_infinite_dy(qn, T, r):
    w, X, dY, A, B = _layer(qn, T, 72, 64, r)
    U = torch.ones(T, r, device="cuda")
    U[:, 1] = -0.75
    U[:, 2] = 1.0 + 2.0 ** -10  # two terms and a zero one
    db = lambda d, u=U: qn.qlora_linear_bwd_act8(w, None, d, A, B, 2.0, U=u, need_dx=False, need_da=False)[2]
    plain = db(dY)
    d = dY.clone()
    d[T // 2, 5], d[T - 1, 6] = INF, -INF
    d[0, 7], d[T - 1, 7] = INF, -INF  # two that cancel
    d[T // 3, 9] = float("nan")
    got = db(d)
    assert torch.isposinf(got[5, [0, 2]]).all() and torch.isneginf(got[5, 1])
    assert torch.isneginf(got[6, [0, 2]]).all() and torch.isposinf(got[6, 1])
    assert torch.isposinf(got[5, 3:]).all() and torch.isneginf(got[6, 3:]).all()
    assert torch.isnan(got[7]).all() and torch.isnan(got[9]).all()
    other = [n for n in range(72) if n not in (5, 6, 7, 9)]
    assert torch.equal(got[other], plain[other])
    # as the ordinary backward, whose U is one bf16 term
    want = qn.qlora_linear_bwd(w, X, d, A, B, 2.0, U=U, need_dx=False, need_da=False)[2]
    for f in (torch.isposinf, torch.isneginf, torch.isnan):
        assert torch.equal(f(got), f(want))
    u = U.clone()
    u[T // 2, 0] = 0.0  # zero times infinity
    assert torch.isnan(db(d, u)[5, 0]) and torch.isneginf(db(d, u)[5, 1])


@pytest.mark.parametrize("r", RANKS)
@pytest.mark.parametrize("T", [9, 2100])
def test_values_that_a_checkpoint_restores_as_infinity(qn, T, r):
    """Magnitudes from 1.9375 2^127 on come back as 2^128, infinity."""
    w, X, dY, A, B = _layer(qn, T, 8, 128, r)
    X[T // 2, 70] = 3.38e38
    x8 = qn.act8_quantize(X)
    assert torch.isposinf(qn.act8_dequantize(x8)[T // 2, 70])
    # G = 8 of every token and rank: one term
    dA = qn.qlora_linear_bwd_act8(w, x8, torch.ones_like(dY), A, torch.ones_like(B), need_dx=False, need_db=False)[1]
    assert torch.isposinf(dA[:, 70]).all() and torch.isfinite(dA[:, :64]).all() and torch.isfinite(dA[:, 96:]).all()


def test_infinite_dy_in_a_group(qn):
    T, r = 40, 24
    w, X, dY, A, B = _layer(qn, T, 72, 64, r)
    U = torch.ones(T, r, device="cuda")
    d = dY.clone()
    d[3, 5] = INF
    _, _, dBs = qn.qlora_linear_bwd_group_act8([w, w], None, [dY, d], [A, A], [B, B], 1.0, Us=[U, U], need_dx=False,
                                               need_da=False)
    assert torch.isfinite(dBs[0]).all() and torch.isposinf(dBs[1][5]).all() and torch.isfinite(dBs[1][:5]).all()


def test_infinite_dy_captured(qn):
    T, r = 300, 16
    w, X, dY, A, B = _layer(qn, T, 72, 64, r)
    U = torch.ones(T, r, device="cuda")
    step = lambda: qn.qlora_linear_bwd_act8(w, None, dY, A, B, U=U, need_dx=False, need_da=False)[2]
    step()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = step()
    for v in (1.0, INF, 2.0):
        dY[7, 11] = v
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, step()) and bool(torch.isposinf(out[11]).all()) == (v == INF)
