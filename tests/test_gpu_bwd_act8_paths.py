"""Paths of the backward from a checkpoint that depend on the sizes: G formed
inside the dX launch (unsplit 256-wide plans, ranks 8 and 16), the gradient
kernel's 64-column tiles for ranks to 64, ranks between 65 and 96."""

import pytest
import torch

import workloads
from test_gpu_bwd_act8 import Case, _check

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def qn():
    import bit_nf4_quantized_16_amd as qn

    assert torch.cuda.is_available()
    return qn


# (T, N, K, r) whose dX runs unsplit 256 tiles where that tile is forced
IN_LAUNCH = [(300, 512, 1024, 16), (33, 256, 4160, 8), (257, 1024, 2048, 16), (1, 64, 64, 8)]


def _plain(qn, c, **kw):
    return qn.qlora_linear_bwd(c.w, c.Xc, c.dYc, c.Ac, c.Bc, c.scale, U=c.U, **kw)


@pytest.mark.parametrize("T,N,K,r", IN_LAUNCH)
def test_g_inside_the_dx_launch(qn, monkeypatch, T, N, K, r):
    """Against the exact sums, the launch before, the ordinary backward (dX)
    and the group call (dA, dB)."""
    monkeypatch.setenv("QLORA_NF4_GEMM_TILE", "256")
    monkeypatch.setenv("QLORA_NF4_GEMM_SPLITS", "1")
    assert qn.lib.qlora_linear_bwd_g_in_launch(N, K, T, r) == 1
    c = Case(qn, T, N, K, r, seed=T + r)
    got = c.run(qn)
    _check(c, got[1], got[2])
    assert torch.equal(got[0], _plain(qn, c)[0])
    gX, gA, gB = qn.qlora_linear_bwd_group_act8([c.w], c.X8, [c.dYc], [c.Ac], [c.Bc], c.scale, Us=[c.U])
    assert torch.equal(gA[0], got[1]) and torch.equal(gB[0], got[2]) and torch.equal(gX, got[0])
    for need in ((True, True, False), (True, False, True), (True, False, False), (False, True, True)):
        sub = c.run(qn, need_dx=need[0], need_da=need[1], need_db=need[2])
        for s, f, n in zip(sub, got, need):
            assert (s is not None) == n and (s is None or torch.equal(s, f))
    monkeypatch.setenv("QLORA_NF4_FWD_U", "prepass")
    assert qn.lib.qlora_linear_bwd_g_in_launch(N, K, T, r) == 0
    for a, b in zip(c.run(qn), got):
        assert torch.equal(a, b)


def test_a_layer_whose_plan_puts_g_inside(qn, monkeypatch):
    """The down projection at T = 1024, rank 16, by its own plan."""
    T, N, K, r = 1024, 4096, 11008, 16
    assert qn.lib.qlora_linear_bwd_g_in_launch(N, K, T, r) == 1
    c = Case(qn, T, N, K, r, seed=5)
    got = c.run(qn)
    _check(c, got[1], got[2])
    assert torch.equal(got[0], _plain(qn, c)[0])
    monkeypatch.setenv("QLORA_NF4_FWD_U", "prepass")
    for a, b in zip(c.run(qn), got):
        assert torch.equal(a, b)


@pytest.mark.parametrize("spin", [None, "-1"])
def test_g_inside_captured(qn, monkeypatch, spin):
    """Replays with new dY, also where the tiles form G themselves (forced);
    dA takes the projection's G either way."""
    monkeypatch.setenv("QLORA_NF4_GEMM_TILE", "256")
    if spin:
        monkeypatch.setenv("QLORA_NF4_GEMM_SPIN", spin)
    T, N, K, r = IN_LAUNCH[0]
    assert qn.lib.qlora_linear_bwd_g_in_launch(N, K, T, r) == 1
    c = Case(qn, T, N, K, r, seed=6)
    step = lambda: qn.qlora_linear_bwd_act8(c.w, c.X8, c.dYc, c.Ac, c.Bc, c.scale, U=c.U)
    step()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = step()
    for i in range(4):
        c.dY = workloads.bf16_normal((T, N), 1.0, 70 + i)
        c.dYc.copy_(c.dY.cuda())
        graph.replay()
        torch.cuda.synchronize()
        for a, b in zip(out, step()):
            assert torch.equal(a, b)
        _check(c, out[1], out[2])


def test_g_inside_on_two_streams(qn, monkeypatch):
    monkeypatch.setenv("QLORA_NF4_GEMM_TILE", "256")
    T, N, K, r = IN_LAUNCH[2]
    cs = [Case(qn, T, N, K, r, seed=s) for s in (40, 41)]
    want = [c.run(qn) for c in cs]
    got = []
    for c in cs:
        st = torch.cuda.Stream()
        st.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(st):
            got.append(qn.qlora_linear_bwd_act8(c.w, c.X8, c.dYc, c.Ac, c.Bc, c.scale, U=c.U))
    torch.cuda.synchronize()
    for g, w in zip(got, want):
        for a, b in zip(g, w):
            assert torch.equal(a, b)


# over 128 column tiles of 64: the wide form for ranks to 64, in one sum of
# the tokens and in two; the last columns and rows end inside a tile
@pytest.mark.parametrize("r", [5, 16, 20, 32, 40, 48, 61, 64])
@pytest.mark.parametrize("T", [33, 2100])
def test_many_columns(qn, T, r):
    p = 0.3 if r % 8 == 0 and T == 33 else 0.0
    c = Case(qn, T, 264, 8256, r, seed=T + r, p=p)
    _, dA, dB = c.run(qn, need_dx=False)
    _check(c, dA, dB)


@pytest.mark.parametrize("r", [65, 72, 80, 81, 96, 97, 112])
@pytest.mark.parametrize("T", [1, 33, 2500])
def test_ranks_over_64(qn, T, r):
    c = Case(qn, T, 72, 192, r, seed=T + r, p=0.3 if r % 2 else 0.0)
    dX, dA, dB = c.run(qn)
    _check(c, dA, dB)
    assert torch.equal(dX, _plain(qn, c, keep=c.bits, p=c.p)[0])
    a1 = torch.ones_like(dA)
    assert torch.equal(c.run(qn, need_dx=False, dA=a1, accumulate=True)[1], 1 + dA)
