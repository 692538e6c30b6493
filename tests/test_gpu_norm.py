"""Norms against the 64-bit formulas, element by element. Bounds: the output's
half step, and fp32 sums whose terms pass through at most 64 roundings each
(16 in a lane, 6 across it, 16 waves, the mean, the square root and the
products after it): 2^-18 of the terms' absolute values."""

import pytest
import torch

pytestmark = pytest.mark.gpu

BF16, F32 = torch.bfloat16, torch.float32
HALF = {t: torch.finfo(t).eps / 2 for t in (BF16, F32)}
E = 2.0 ** -18


@pytest.fixture(scope="module")
def qn():
    import bit_nf4_quantized_16_amd as qn

    assert torch.cuda.is_available()
    return qn


def _inputs(T, C, xt, wt, seed=0, shift=0.3):
    g = torch.Generator(device="cuda").manual_seed(seed)
    r = lambda *s: torch.randn(*s, generator=g, device="cuda")
    return (2 * r(T, C) + shift).to(xt), (1 + 0.2 * r(C)).to(wt), (0.3 * r(C)).to(wt), r(T, C).to(xt)


def _exact(X, w, b, dY, eps, rms):
    x, w, d = X.double(), w.double(), dY.double()
    mu = torch.zeros_like(x[:, :1]) if rms else x.mean(1, keepdim=True)
    r = 1 / torch.sqrt(((x - mu) ** 2).mean(1, keepdim=True) + eps)
    h = (x - mu) * r
    g = d * w
    dx = r * (g - h * (g * h).mean(1, keepdim=True) - (0 if rms else g.mean(1, keepdim=True)))
    q = r * x.abs().mean(1, keepdim=True)  # what the mean's rounding is of h
    hb = h.abs() + (0 if rms else q)
    tol = dict(y=E * hb * w.abs() + 2.0 ** -23 * (0 if b is None else b.double().abs()),
               dx=E * r * (2 * g.abs() + 2 * g.abs().mean(1, keepdim=True) + 3 * hb * (g.abs() * hb).mean(1, keepdim=True)),
               dw=(E + 2.0 ** -24 * x.shape[0]) * (d.abs() * hb).sum(0), db=(E + 2.0 ** -24 * x.shape[0]) * d.abs().sum(0))
    return dict(y=h * w + (0 if b is None else b.double()), dx=dx, dw=(d * h).sum(0), db=d.sum(0), mu=mu[:, 0], r=r[:, 0]), tol


def _close(name, got, want, tol):
    bad = (got.double() - want).abs() - (HALF[got.dtype] * want.abs() + tol)
    assert got.shape == want.shape and float(bad.max()) <= 0, (name, float(bad.max()))


@pytest.mark.parametrize("xt,wt", [(BF16, BF16), (BF16, F32), (F32, F32), (F32, BF16)])
@pytest.mark.parametrize("T,C", [(1, 8), (1, 4096), (3, 16), (5, 520), (77, 264), (7, 1032), (600, 72), (33, 2056),
                                 (65, 4104), (2, 8192), (17, 8200), (3, 16384), (1030, 16)])
@pytest.mark.parametrize("rms", [False, True])
def test_forward_and_backward(qn, T, C, xt, wt, rms):
    X, w, b, dY = _inputs(T, C, xt, wt, seed=T + C)
    b = None if rms and C % 16 else b
    eps = 1e-5
    want, tol = _exact(X, w, b, dY, eps, rms)
    Y, mean, rstd = qn.norm_fwd(X, w, b, eps, rms)
    assert (mean is None) == rms
    _close("Y", Y, want["y"], tol["y"])
    _close("rstd", rstd, want["r"], E * want["r"])
    if not rms:
        _close("mean", mean, want["mu"], E * X.double().abs().mean(1))
    dX, dW, dB = qn.norm_bwd(X, w, dY, mean, rstd)
    _close("dX", dX, want["dx"], tol["dx"])
    _close("dW", dW, want["dw"], tol["dw"])
    _close("dB", dB, want["db"], tol["db"])
    # each output alone, and added to what is there
    assert torch.equal(qn.norm_bwd(X, w, dY, mean, rstd, need_dw=False, need_db=False)[0], dX)
    assert torch.equal(qn.norm_bwd(X, w, dY, mean, rstd, need_dx=False, need_db=False)[1], dW)
    assert torch.equal(qn.norm_bwd(X, w, dY, mean, rstd, need_dx=False, need_dw=False)[2], dB)
    ones = torch.ones_like(dW)
    _, aW, aB = qn.norm_bwd(X, w, dY, mean, rstd, need_dx=False, dW=ones.clone(), dB=ones.clone(), accumulate=True)
    assert torch.equal(aW, 1 + dW) and torch.equal(aB, 1 + dB)
    assert torch.equal(qn.norm_fwd(X, w, b, eps, rms, stats=False)[0], Y)


@pytest.mark.parametrize("rms", [False, True])
def test_a_large_mean_and_tiny_rows(qn, rms):
    """The variance comes from x - mu: a mean a thousand times the spread costs
    the mean's rounding only; constant and zero rows end at eps."""
    X, w, b, dY = _inputs(9, 1024, F32, F32, seed=4)
    X[0] += 2000.0
    X[1] = 0.0
    X[2] = 3.0
    X[3] *= 1e-12
    want, tol = _exact(X, w, b, dY, 1e-5, rms)
    Y, mean, rstd = qn.norm_fwd(X, w, b, 1e-5, rms)
    _close("Y", Y, want["y"], tol["y"])
    _close("dX", qn.norm_bwd(X, w, dY, mean, rstd)[0], want["dx"], tol["dx"])


def test_rows_are_independent_of_nan_and_infinity(qn):
    X, w, b, dY = _inputs(8, 520, BF16, BF16, seed=5)
    Y, mean, rstd = qn.norm_fwd(X, w, b)
    X2 = X.clone()
    X2[2, 7], X2[5, 0], X2[6, 519] = float("nan"), float("inf"), float("-inf")
    Y2, _, _ = qn.norm_fwd(X2, w, b)
    on = torch.tensor([0, 1, 3, 4, 7], device="cuda")
    assert torch.equal(Y2[on], Y[on]) and bool(Y2[2].isnan().all())
    assert bool(Y2[5, 0].isnan()) and bool(Y2[6, 519].isnan())


def test_nothing_behind_the_arrays_is_written_and_repeats_are_equal(qn):
    X, w, b, dY = _inputs(37, 4104, BF16, F32, seed=6)
    Y, mean, rstd = qn.norm_fwd(X, w, b)
    dX, dW, dB = qn.norm_bwd(X, w, dY, mean, rstd)
    L = qn.lib
    guard = torch.full((X.numel() + 64,), 7.0, dtype=BF16, device="cuda")
    st = torch.full((37 + 16,), 7.0, device="cuda")
    s = torch.cuda.current_stream().cuda_stream
    assert L.qlora_norm_fwd(X.data_ptr(), 1, 37, 4104, w.data_ptr(), b.data_ptr(), 0, 1e-5, 0, guard.data_ptr(),
                            st.data_ptr(), rstd.data_ptr(), s) == 0
    assert torch.equal(guard[:X.numel()].view_as(Y), Y) and bool((guard[X.numel():] == 7).all())
    assert torch.equal(st[:37], mean) and bool((st[37:] == 7).all())
    gw = torch.full((4104 + 64,), 7.0, device="cuda")
    qn.norm_bwd(X, w, dY, mean, rstd, dW=gw[:4104], need_dx=False, need_db=False)
    assert torch.equal(gw[:4104], dW) and bool((gw[4104:] == 7).all())
    for _ in range(3):
        a = qn.norm_bwd(X, w, dY, mean, rstd)
        assert all(torch.equal(p, q) for p, q in zip(a, (dX, dW, dB)))


def test_in_place_and_no_rows(qn):
    X, w, b, dY = _inputs(20, 264, BF16, BF16, seed=7)
    Y, mean, rstd = qn.norm_fwd(X, w, b)
    dX, _, _ = qn.norm_bwd(X, w, dY, mean, rstd)
    Xc, dc = X.clone(), dY.clone()
    s = torch.cuda.current_stream().cuda_stream
    assert qn.lib.qlora_norm_bwd(X.data_ptr(), 1, 20, 264, w.data_ptr(), 1, dc.data_ptr(), mean.data_ptr(),
                                 rstd.data_ptr(), dc.data_ptr(), None, None, 0, None, 0, s) == 0
    assert torch.equal(dc, dX)
    assert qn.lib.qlora_norm_fwd(Xc.data_ptr(), 1, 20, 264, w.data_ptr(), b.data_ptr(), 1, 1e-5, 0, Xc.data_ptr(), None,
                                 None, s) == 0
    assert torch.equal(Xc, Y)
    Y0, m0, r0 = qn.norm_fwd(X[:0], w, b)
    assert Y0.shape == (0, 264)
    dX0, dW0, dB0 = qn.norm_bwd(X[:0], w, dY[:0], m0, r0)
    assert dX0.shape == (0, 264) and not bool(dW0.any()) and not bool(dB0.any())
    acc = torch.full((264,), 2.0, device="cuda")
    assert bool((qn.norm_bwd(X[:0], w, dY[:0], m0, r0, dW=acc, accumulate=True)[1] == 2).all())


def test_autograd(qn):
    """Views, a broadcast gradient, gradients against differences of the
    64-bit formula, and what is refused."""
    X, w, b, _ = _inputs(24, 64, F32, F32, seed=8)
    leaf = torch.cat([X, X], 1)[:, 32:96].contiguous().t().contiguous().t().requires_grad_()  # column-major
    assert not leaf.is_contiguous()
    wl, bl = w.clone().requires_grad_(), b.clone().requires_grad_()
    d = torch.randn(24, 64, device="cuda")
    for rms in (False, True):
        Y = qn.NormFunction.apply(leaf, wl, bl, 1e-5, rms)
        got = torch.autograd.grad(Y, (leaf, wl, bl), d)
        ref = [t.detach().double().requires_grad_() for t in (leaf, wl, bl)]

        def f(x, w_, b_):
            c = x if rms else x - x.mean(1, keepdim=True)
            return (c / torch.sqrt((c * c).mean(1, keepdim=True) + 1e-5) * w_ + b_)

        for g, e in zip(got, torch.autograd.grad(f(*ref), ref, d.double())):
            assert float((g - e).abs().max()) <= 1e-5 * float(e.abs().max())
        # a difference in one direction
        u = torch.randn_like(leaf).double()
        t = 1e-4
        num = ((f(ref[0] + t * u, ref[1], ref[2]) - f(ref[0] - t * u, ref[1], ref[2])) * d).sum() / (2 * t)
        assert abs(float(num - (got[0] * u).sum())) <= 1e-4 * float((got[0] * u).abs().sum())
    Y = qn.NormFunction.apply(leaf, wl, bl)
    Y.sum().backward()
    assert torch.allclose(bl.grad, torch.full((64,), 24.0, device="cuda"))
    only = qn.NormFunction.apply(X, wl)
    assert torch.autograd.grad(only.sum(), wl)[0].shape == (64,)
    g, = torch.autograd.grad(qn.NormFunction.apply(leaf, wl, bl).sum(), leaf, create_graph=True)
    with pytest.raises(RuntimeError, match="cannot be differentiated again"):
        torch.autograd.grad(g.sum(), leaf)


def test_graph_replays_and_a_second_stream(qn):
    X, w, b, dY = _inputs(300, 1032, BF16, BF16, seed=9)

    def step():
        Y, mean, rstd = qn.norm_fwd(X, w, b)
        return (Y, *qn.norm_bwd(X, w, dY, mean, rstd))

    step()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = step()
    for seed in (1, 2, 3):
        new = _inputs(300, 1032, BF16, BF16, seed=20 + seed)
        X.copy_(new[0]), dY.copy_(new[3])
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(p, q) for p, q in zip(out, step()))
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        a = step()
    b2 = step()
    side.synchronize()
    torch.cuda.synchronize()
    assert all(torch.equal(p, q) for p, q in zip(a, b2))


@pytest.mark.parametrize("xt,wt,T,C", [(BF16, BF16, 4100, 4096), (BF16, F32, 4099, 8192), (F32, F32, 4100, 1024), (F32, BF16, 5000, 4096),
                                       (BF16, F32, 9000, 2048), (BF16, BF16, 2050, 16384), (F32, F32, 300, 16384)])
@pytest.mark.parametrize("rms", [False, True])
def test_many_rows(qn, T, C, xt, wt, rms):
    """Several rows a workgroup at a time, many turns."""
    X, w, b, dY = _inputs(T, C, xt, wt, seed=C)
    want, tol = _exact(X, w, b, dY, 1e-5, rms)
    Y, mean, rstd = qn.norm_fwd(X, w, b, 1e-5, rms)
    _close("Y", Y, want["y"], tol["y"])
    dX, dW, dB = qn.norm_bwd(X, w, dY, mean, rstd)
    _close("dX", dX, want["dx"], tol["dx"])
    _close("dW", dW, want["dw"], tol["dw"])
    _close("dB", dB, want["db"], tol["db"])
    assert torch.equal(qn.norm_bwd(X, w, dY, mean, rstd, need_dx=False, need_db=False)[1], dW)
    assert torch.equal(qn.norm_bwd(X, w, dY, mean, rstd, need_dx=False, need_dw=False)[2], dB)


@pytest.mark.parametrize("T,C", [(9001, 512), (4099, 4096), (700, 8192)])
@pytest.mark.parametrize("rms", [False, True])
def test_gradient_in_place_over_many_turns(qn, T, C, rms):
    """dX in dY's place while later rows are loaded ahead, sums beside it: the
    bits of a call with arrays of its own."""
    X, w, b, dY = _inputs(T, C, BF16, F32, seed=T)
    Y, mean, rstd = qn.norm_fwd(X, w, b, 1e-5, rms)
    dX, dW, dB = qn.norm_bwd(X, w, dY, mean, rstd)
    d, sw, sb = dY.clone(), torch.zeros(C, device="cuda"), torch.zeros(C, device="cuda")
    n = qn.lib.qlora_norm_bwd_workspace(T, C)
    ws = torch.empty(n, dtype=torch.uint8, device="cuda")
    assert qn.lib.qlora_norm_bwd(X.data_ptr(), 1, T, C, w.data_ptr(), 0, d.data_ptr(),
                                 mean.data_ptr() if mean is not None else None, rstd.data_ptr(), d.data_ptr(),
                                 sw.data_ptr(), sb.data_ptr(), 1, ws.data_ptr(), n,
                                 torch.cuda.current_stream().cuda_stream) == 0
    assert torch.equal(d, dX) and torch.equal(sw, dW) and torch.equal(sb, dB)
