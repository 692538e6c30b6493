"""The preference loss and distillation against the 64-bit formulas, element by
element. With n = V / 256 + 64 roundings at most between an exponential and the
row's sum, and D the row's range (an exponential's argument is rounded twice):
e(V, D) = (n + 2 D) 2^-23 is the relative error of a softmax value, and the
absolute one of a log probability besides 2^-22 of it."""

import pytest
import torch

pytestmark = pytest.mark.gpu

BF16, F32 = torch.bfloat16, torch.float32
HALF = {t: torch.finfo(t).eps / 2 for t in (BF16, F32)}
NINF, INF, NAN = float("-inf"), float("inf"), float("nan")


@pytest.fixture(scope="module")
def qn():
    import bit_nf4_quantized_16_amd as qn

    assert torch.cuda.is_available()
    return qn


def _e(z):
    """e(V, D) of each row, finite values alone."""
    f = torch.where(torch.isfinite(z), z, z.new_full((), NAN))
    d = torch.nan_to_num(f, NAN, NAN, NAN)
    hi = torch.where(d.isnan(), d.new_full((), NINF), d).amax(1)
    lo = torch.where(d.isnan(), d.new_full((), INF), d).amin(1)
    return (z.shape[1] / 256 + 64 + 2 * (hi - lo)).double() * 2.0 ** -23


def _logits(T, V, dt, seed, ld=None, off=0):
    """[T, V] logits, rows ld values apart, the first `off` values past a
    16-byte boundary; and the memory they lie in."""
    g = torch.Generator(device="cuda").manual_seed(seed)
    ld = V if ld is None else ld
    flat = torch.full((off + T * ld + 32,), 9.0, dtype=dt, device="cuda")
    z = flat.as_strided((T, V), (ld, 1), off)
    z.copy_(2.5 * torch.randn(T, V, generator=g, device="cuda"))
    return z, flat


def _close(name, got, want, tol):
    diff = (got.double() - want).abs()
    bad = torch.where(got.double() == want, torch.zeros_like(diff), diff - (HALF[got.dtype] * want.abs() + tol))
    assert got.shape == want.shape and not bool(bad.isnan().any()) and float(bad.max() if bad.numel() else 0) <= 0, \
        (name, float(bad.max()))


# ---------------------------------------------------------------------------
# preference
# ---------------------------------------------------------------------------
def _pref_exact(z, labels, start, ref, beta, smooth, kind, average, dloss):
    z = z.double()
    T, V = z.shape
    on = (labels >= 0) & (labels < V)
    at = torch.where(on, labels, 0)
    logq = torch.log_softmax(z, 1) if T else z
    lp = torch.where(on, logq.gather(1, at[:, None])[:, 0], 0.0)
    e = _e(z)
    etok = torch.where(on, e + 2.0 ** -22 * (lp.abs() + 40), 0.0)
    L, eL, per = [], [], []
    ends = start.clamp(0, T).tolist()
    for a, b in zip(ends[:-1], ends[1:]):
        n = max(int(on[a:b].sum()), 1) if average else 1
        L.append(lp[a:b].sum() / n), eL.append(etok[a:b].sum() / n), per.append(1.0 / n)
    L, eL = (torch.stack(x) if x else z.new_zeros(0) for x in (L, eL))
    d = ((L - ref.double()).view(-1, 2) * torch.tensor([1.0, -1.0], device=z.device)).sum(1).requires_grad_()
    ed = eL.view(-1, 2).sum(1)
    x = beta * d
    if kind == "sigmoid":
        loss = -(1 - smooth) * torch.nn.functional.logsigmoid(x) - smooth * torch.nn.functional.logsigmoid(-x)
        eslope = beta * beta / 4 * ed
    elif kind == "hinge":
        loss, eslope = torch.relu(1 - x), 0 * ed
    else:
        loss, eslope = (d - 0.5 / beta) ** 2, 2 * ed
    slope, = torch.autograd.grad(loss.sum(), d) if d.numel() else (d.detach(),)
    f, ef = torch.zeros(T, device=z.device).double(), torch.zeros(T, device=z.device).double()
    for i, (a, b) in enumerate(zip(ends[:-1], ends[1:])):
        f[a:b] = slope[i // 2] * (1 if i % 2 == 0 else -1) * per[i] * dloss[i // 2].double()
        ef[a:b] = eslope[i // 2] * per[i] * dloss[i // 2].double().abs()
    f, ef = torch.where(on, f, 0.0), torch.where(on, ef, 0.0)
    q = torch.softmax(z, 1) if T else z
    hot = torch.zeros_like(q)
    hot[on, at[on]] = 1
    dz = torch.where(on[:, None], f[:, None] * (hot - q), 0.0)
    edz = ef[:, None] * (hot - q).abs() + (f.abs() * e)[:, None] * q + 2.0 ** -22 * f.abs()[:, None] * (hot + q)
    loss = loss.detach()
    eloss = (slope.abs() + eslope) * ed + 2.0 ** -23 * loss.abs() + 2.0 ** -23 * (beta * d.detach()).abs()
    return dict(loss=loss, L=L, dz=dz), dict(loss=eloss, L=eL, dz=torch.where(on[:, None], edz, 0.0))


def _pref_case(T, V, dt, pairs, seed, masked=0.3, ld=None, off=0):
    z, flat = _logits(T, V, dt, seed, ld, off)
    g = torch.Generator(device="cuda").manual_seed(seed + 1)
    labels = torch.randint(0, V, (T,), generator=g, device="cuda")
    labels = torch.where(torch.rand(T, generator=g, device="cuda") < masked, -100, labels)
    cuts = torch.randint(0, T + 1, (2 * pairs - 1,), generator=g, device="cuda").sort().values
    start = torch.cat([cuts.new_tensor([0]), cuts, cuts.new_tensor([T])])
    on = labels >= 0
    lp = torch.where(on, torch.log_softmax(z.double(), 1).gather(1, labels.clamp(min=0)[:, None])[:, 0], 0.0)
    c = torch.cat([lp.new_zeros(1), lp.cumsum(0)])
    ref = (c[start[1:]] - c[start[:-1]] + 3 * torch.randn(2 * pairs, generator=g, device="cuda")).float()
    dloss = torch.rand(pairs, generator=g, device="cuda") + 0.2
    return z, flat, labels, start, ref, dloss


def _pref_check(qn, z, labels, start, ref, dloss, beta=0.1, smooth=0.0, kind="sigmoid", average=False):
    want, tol = _pref_exact(z, labels, start, ref, beta, smooth, kind, average, dloss)
    loss, L, st = qn.preference_loss_fwd(z, labels, start, ref, beta, smooth, kind, average)
    _close("L", L, want["L"], tol["L"])
    _close("loss", loss, want["loss"], tol["loss"])
    dz = qn.preference_loss_bwd(z, labels, st, dloss)
    assert dz.stride() == z.stride() or z.shape[0] <= 1
    _close("dz", dz, want["dz"], tol["dz"])
    return loss, L, st, dz


@pytest.mark.parametrize("dt", [BF16, F32])
@pytest.mark.parametrize("T,V,pairs", [(2, 1, 1), (2, 2, 1), (5, 7, 1), (9, 8, 2), (33, 9, 3), (40, 300, 2), (6, 4097, 1),
                                       (20, 32000, 2), (3, 50257, 1), (700, 1001, 5), (4, 131073, 2), (1100, 64, 1)])
def test_preference(qn, T, V, pairs, dt):
    z, _, labels, start, ref, dloss = _pref_case(T, V, dt, pairs, seed=T + V)
    for kind, smooth, average in (("sigmoid", 0.0, False), ("sigmoid", 0.2, True), ("hinge", 0.0, False),
                                  ("squared", 0.0, True)):
        r = ref / 7 if average else ref
        _pref_check(qn, z, labels, start, r, dloss, 0.3, smooth, kind, average)


@pytest.mark.parametrize("dt,V,ld,off", [(BF16, 257, 264, 0), (BF16, 257, 259, 3), (BF16, 64, 71, 1), (F32, 257, 301, 1),
                                         (F32, 30, 33, 3), (BF16, 5, 9, 7), (F32, 2, 3, 1), (BF16, 40000, 40003, 5)])
def test_preference_strides_and_offsets(qn, dt, V, ld, off):
    """Rows at every offset; nothing between and behind the rows is touched;
    the gradient in place of the logits."""
    z, flat, labels, start, ref, dloss = _pref_case(11, V, dt, 2, seed=V, ld=ld, off=off)
    _, _, st, dz = _pref_check(qn, z, labels, start, ref, dloss)
    assert (dz.data_ptr() - z.data_ptr()) % 16 == 0
    keep = torch.ones_like(flat, dtype=torch.bool)
    keep.as_strided(z.shape, z.stride(), off).fill_(False)
    out = qn.preference_loss_bwd(z, labels, st, dloss, dlogits=z)
    assert out is z and torch.equal(z, dz) and bool((flat[keep] == 9).all())


def test_preference_edges(qn):
    z, _, labels, start, ref, dloss = _pref_case(30, 777, BF16, 2, seed=3)
    # empty sequences, rows before the first and behind the last, a masked sequence
    start = torch.tensor([4, 4, 11, 20, 26], device="cuda")
    labels[11:20] = -1
    loss, L, st, dz = _pref_check(qn, z, labels, start, ref, dloss)
    assert float(L[0]) == 0 and float(L[2]) == 0 and not bool(dz[:4].any()) and not bool(dz[26:].any())
    _pref_check(qn, z, labels, start, ref, dloss, average=True)
    # starts outside [0, T]
    _pref_check(qn, z, labels, torch.tensor([-5, 4, 11, 20, 1000], device="cuda"), ref, dloss)
    # labels outside the vocabulary
    labels[:4] = torch.tensor([777, 1 << 40, -(1 << 40), 776], device="cuda")
    _pref_check(qn, z, labels, torch.tensor([0, 4, 11, 20, 26], device="cuda"), ref, dloss)
    # no rows, no pairs
    none = torch.zeros(5, dtype=torch.int64, device="cuda")
    loss, L, st = qn.preference_loss_fwd(z[:0], labels[:0], none, ref)
    assert not bool(L.any()) and qn.preference_loss_bwd(z[:0], labels[:0], st, dloss).shape == (0, 777)
    loss, L, st = qn.preference_loss_fwd(z, labels, none[:1], ref[:0])
    assert loss.numel() == 0 and not bool(qn.preference_loss_bwd(z, labels, st, dloss[:0]).any())
    assert qn.token_logp(z[:0], labels[:0]).shape == (0,)


def test_preference_values(qn):
    """Masked vocabulary entries, the type's extremes, infinities and NaN; a
    loss far from its bend."""
    z, _, labels, start, ref, dloss = _pref_case(24, 513, F32, 2, seed=5, masked=0.0)
    z[:, 400:] = NINF
    labels %= 400
    z[3, 5:] = torch.finfo(F32).min
    labels[3] = 2
    z[4] = torch.finfo(F32).min  # all alike at the lowest value
    z[5] = torch.finfo(F32).max
    z[6, 1:] = NINF  # one entry left
    labels[6] = 0
    want = torch.log_softmax(z.double(), 1).gather(1, labels[:, None])[:, 0]
    _close("logp", qn.token_logp(z, labels), want, _e(z).clamp(max=1e-3) + 2.0 ** -22 * (want.abs() + 40))
    for shift in (-4000.0, 4000.0):
        r = ref.clone()
        r[0] += shift
        zs = 0.1 * torch.randn(24, 513, device="cuda")
        for kind in ("sigmoid", "hinge", "squared"):
            _pref_check(qn, zs, labels, start, r, dloss, 0.5, 0.0, kind)
    # rows with NaN, +inf and without any finite value spoil their own pair alone
    z = torch.randn(24, 513, device="cuda")
    start = torch.tensor([0, 6, 12, 18, 24], device="cuda")
    base = _pref_check(qn, z, labels, start, ref, dloss)
    for bad in (NAN, INF, NINF):
        y = z.clone()
        y[2, 100] = bad
        if bad == NINF:
            y[2] = NINF
        loss, L, st = qn.preference_loss_fwd(y, labels, start, ref)
        dz = qn.preference_loss_bwd(y, labels, st, dloss)
        assert bool(loss[0].isnan()) and torch.equal(loss[1:], base[0][1:]) and torch.equal(L[1:], base[1][1:])
        assert bool(dz[2].isnan().any()) and torch.equal(dz[12:], base[3][12:])


def test_token_logp_is_the_reference_side(qn):
    """The reference model's log probabilities by the same kernel: a model
    against itself is at the loss's middle."""
    z, _, labels, start, ref, dloss = _pref_case(50, 1000, BF16, 3, seed=6)
    lp = qn.token_logp(z, labels).double()
    c = torch.cat([lp.new_zeros(1), lp.cumsum(0)])
    own = (c[start[1:]] - c[start[:-1]]).float()
    loss, L, _ = qn.preference_loss_fwd(z, labels, start, own)
    assert float((loss - 0.6931472).abs().max()) < 1e-4 and torch.allclose(L, own, rtol=2 ** -22, atol=0)


def test_preference_autograd(qn):
    z, _, labels, start, ref, _ = _pref_case(26, 130, F32, 3, seed=7)
    zl = z.clone().requires_grad_()
    loss, L = qn.PreferenceLossFunction.apply(zl, labels, start, ref, 0.2)
    assert not L.requires_grad
    loss.mean().backward()  # a broadcast gradient
    want, tol = _pref_exact(z, labels, start, ref, 0.2, 0.0, "sigmoid", False, torch.full((3,), 1 / 3, device="cuda"))
    _close("dz", zl.grad, want["dz"], tol["dz"])
    # against a difference of the 64-bit loss
    u = torch.randn_like(z).double()
    t = 1e-4
    f = lambda s: _pref_exact(z.double() + s * u, labels, start, ref, 0.2, 0.0, "sigmoid", False, torch.ones(3, device="cuda"))[0]["loss"].mean()
    assert abs(float((f(t) - f(-t)) / (2 * t) - (zl.grad * u).sum())) <= 1e-4 * float((zl.grad * u).abs().sum())
    # a transposed leaf, logits written before the backward, second order, a reference with a gradient
    zt = z.t().contiguous().t().requires_grad_()
    loss, _ = qn.PreferenceLossFunction.apply(zt, labels, start, ref, 0.2)
    assert torch.equal(torch.autograd.grad(loss.mean(), zt)[0], zl.grad)
    y = z.clone().requires_grad_()
    w = y * 1
    loss, _ = qn.PreferenceLossFunction.apply(w, labels, start, ref)
    w.mul_(2)
    with pytest.raises(RuntimeError, match="modified by an inplace operation"):
        loss.sum().backward()
    loss, _ = qn.PreferenceLossFunction.apply(y, labels, start, ref)
    g, = torch.autograd.grad(loss.sum(), y, create_graph=True)
    with pytest.raises(RuntimeError, match="cannot be differentiated again"):
        torch.autograd.grad(g.sum(), y)
    with pytest.raises(qn.QLoraError, match="ref_logp"):
        qn.PreferenceLossFunction.apply(y, labels, start, ref.clone().requires_grad_())


# ---------------------------------------------------------------------------
# distillation
# ---------------------------------------------------------------------------
def _distill_exact(z, index, top, labels, tau, alpha, weight):
    z = z.double()
    T, V = z.shape
    there = (index >= 0) & (index < V)
    at = torch.where(there, index, 0)
    t = torch.where(there, top.double() / tau, NINF)
    some = (t > NINF).any(1)
    logp = torch.where(some[:, None], torch.log_softmax(torch.where(some[:, None], t, 0.0), 1), NINF)
    p = logp.exp()
    logq = torch.log_softmax(z / tau, 1)
    lq = logq.gather(1, at)
    kl = torch.where(p > 0, p * (logp - lq), 0.0).sum(1)
    on = torch.ones(T, dtype=torch.bool, device=z.device) if labels is None else (labels >= 0) & (labels < V)
    e = _e(z / tau) + _e(torch.where(torch.isfinite(t), t, 0.0))
    loss = (1 - alpha) * tau ** 2 * kl
    # a term's error: that of p, and of both logarithms
    eloss = (1 - alpha) * tau ** 2 * torch.where(p > 0, p * (2 * e[:, None] * ((logp - lq).abs() + 1) + 2.0 ** -22 * (lq.abs() + logp.abs() + 40)), 0.0).sum(1)
    dz = (1 - alpha) * tau * logq.exp() * some[:, None]
    edz = 2 * e[:, None] * dz
    sub = torch.zeros_like(dz).scatter_add_(1, at, torch.where(there, p, 0.0))
    dz = dz - (1 - alpha) * tau * sub
    edz = edz + (1 - alpha) * tau * sub * (2 * e[:, None] + 2.0 ** -16)  # 257 entries added
    if alpha > 0:
        lab = torch.where(on, labels, 0)
        ls = torch.log_softmax(z, 1)
        e1 = _e(z)
        l1 = ls.gather(1, lab[:, None])[:, 0]
        loss = loss - alpha * l1
        eloss = eloss + alpha * (e1 + 2.0 ** -22 * (l1.abs() + 40))
        hot = torch.zeros_like(dz).scatter_(1, lab[:, None], 1.0)
        dz = dz + alpha * (ls.exp() - hot)
        edz = edz + alpha * (2 * e1[:, None] * ls.exp() + 2.0 ** -16 * hot)
    w = (torch.ones(T, device=z.device) if weight is None else weight).double()[:, None]
    o = on[:, None]
    return (dict(loss=torch.where(on, loss, 0.0), dz=torch.where(o, w * dz, 0.0)),
            dict(loss=torch.where(on, eloss + 2.0 ** -18 * eloss.abs(), 0.0),
                 dz=torch.where(o, w.abs() * (edz + 2.0 ** -22 * dz.abs()), 0.0)))


def _distill_case(T, V, K, dt, seed, ld=None, off=0):
    z, flat = _logits(T, V, dt, seed, ld, off)
    g = torch.Generator(device="cuda").manual_seed(seed + 1)
    index = torch.randint(0, V, (T, K), generator=g, device="cuda")  # the same index twice among them
    top = 2 * torch.randn(T, K, generator=g, device="cuda")
    labels = torch.randint(0, V, (T,), generator=g, device="cuda")
    labels = torch.where(torch.rand(T, generator=g, device="cuda") < 0.2, -100, labels)
    return z, flat, index, top, labels, torch.rand(T, generator=g, device="cuda") + 0.1


def _distill_check(qn, z, index, top, labels, tau, alpha, weight):
    want, tol = _distill_exact(z, index, top, labels, tau, alpha, weight)
    loss, none = qn.distill_loss(z, index, top, labels, tau, alpha, weight)
    assert none is None
    _close("loss", loss, want["loss"], tol["loss"])
    loss2, dz = qn.distill_loss(z, index, top, labels, tau, alpha, weight, need_grad=True)
    assert torch.equal(loss, loss2)
    _close("dz", dz, want["dz"], tol["dz"])
    assert torch.equal(qn.distill_loss(z, index, top, labels, tau, alpha, weight, need_loss=False, need_grad=True)[1], dz)
    return loss, dz


@pytest.mark.parametrize("dt,tt", [(BF16, F32), (F32, BF16), (BF16, BF16)])
@pytest.mark.parametrize("T,V,K", [(1, 1, 1), (2, 3, 2), (3, 7, 9), (4, 8, 1), (9, 300, 8), (5, 4097, 64), (3, 9000, 33),
                                   (2, 20001, 256), (3, 32000, 8), (2, 50257, 17), (2, 66000, 5), (1, 131080, 4),
                                   (700, 65, 3)])
def test_distill(qn, T, V, K, dt, tt):
    z, _, index, top, labels, weight = _distill_case(T, V, K, dt, seed=T + V + K)
    top = top.to(tt)
    for tau, alpha, lab, w in ((1.0, 0.0, None, None), (2.0, 0.0, labels, weight), (1.0, 0.4, labels, weight),
                               (0.7, 0.3, labels, None), (1.5, 1.0, labels, weight)):
        _distill_check(qn, z, index, top, lab, tau, alpha, w)


@pytest.mark.parametrize("dt,V,ld,off", [(BF16, 257, 264, 0), (BF16, 257, 259, 3), (BF16, 64, 71, 1), (F32, 257, 301, 1),
                                         (F32, 30, 33, 3), (BF16, 5, 9, 7), (F32, 2, 3, 1), (BF16, 140001, 140003, 5),
                                         (F32, 70001, 70002, 1)])
def test_distill_strides_and_offsets(qn, dt, V, ld, off):
    z, flat, index, top, labels, weight = _distill_case(11, V, 12, dt, seed=V, ld=ld, off=off)
    loss, dz = _distill_check(qn, z, index, top, labels, 1.0, 0.5, weight)
    keep = torch.ones_like(flat, dtype=torch.bool)
    keep.as_strided(z.shape, z.stride(), off).fill_(False)
    l2, out = qn.distill_loss(z, index, top, labels, 1.0, 0.5, weight, dlogits=z)
    assert out is z and torch.equal(z, dz) and torch.equal(loss, l2) and bool((flat[keep] == 9).all())


def test_distill_edges(qn):
    z, _, index, top, labels, weight = _distill_case(12, 513, 16, F32, seed=4)
    labels = labels.clamp(min=0)
    index[0] = -1  # a row without entries
    index[1, 3:] = 513  # outside
    index[2] = 77  # all the same
    index[3, :4] = labels[3]
    top[4] = NINF  # entries of probability zero
    top[5, 2:] = NINF
    z[6, 200:] = NINF  # masked vocabulary, the teacher's entries elsewhere
    index[6] %= 200
    labels[6] %= 200
    z[7] = torch.finfo(F32).min
    z[8, index[8, 3]] = NINF  # an entry that has no weight
    top[8, 3] = NINF
    top[8][index[8] == index[8, 3]] = NINF
    if int(labels[8]) == int(index[8, 3]):
        labels[8] = (labels[8] + 1) % 513
    for tau, alpha in ((1.0, 0.0), (2.0, 0.3), (1.0, 0.5)):
        loss, dz = _distill_check(qn, z, index, top, labels, tau, alpha, weight)
        if alpha == 0:
            assert float(loss[0]) == 0 and not bool(dz[0].any()) and float(loss[4]) == 0
    base = _distill_check(qn, z, index, top, None, 1.0, 0.0, weight)
    y, t2 = z.clone(), top.clone()
    y[9, 10], y[10, 0], t2[11, 0] = NAN, INF, NAN
    loss, dz = qn.distill_loss(y, index, t2, weight=weight, need_grad=True)
    assert torch.equal(loss[:9], base[0][:9]) and torch.equal(dz[:9], base[1][:9])
    assert bool(loss[9:].isnan().all()) and bool(dz[9].isnan().any())
    # a student that rules a wanted token out
    y = z.clone()
    y[10, index[10, 0]] = NINF
    assert float(qn.distill_loss(y, index, top)[0][10]) == INF
    l0, d0 = qn.distill_loss(z[:0], index[:0], top[:0], need_grad=True)
    assert l0.shape == (0,) and d0.shape == (0, 513)


def test_distill_autograd(qn):
    z, _, index, top, labels, _ = _distill_case(10, 190, 7, F32, seed=5)
    zl = z.clone().requires_grad_()
    loss = qn.DistillLossFunction.apply(zl, index, top, labels, 2.0, 0.25)
    loss.sum().backward()
    want, tol = _distill_exact(z, index, top, labels, 2.0, 0.25, None)
    _close("dz", zl.grad, want["dz"], tol["dz"])
    u, t = torch.randn_like(z).double(), 1e-4
    f = lambda s: _distill_exact(z.double() + s * u, index, top, labels, 2.0, 0.25, None)[0]["loss"].sum()
    assert abs(float((f(t) - f(-t)) / (2 * t) - (zl.grad * u).sum())) <= 1e-4 * float((zl.grad * u).abs().sum())
    g, = torch.autograd.grad(qn.DistillLossFunction.apply(zl, index, top).sum(), zl, create_graph=True)
    with pytest.raises(RuntimeError, match="cannot be differentiated again"):
        torch.autograd.grad(g.sum(), zl)
    with pytest.raises(qn.QLoraError, match="top_logits"):
        qn.DistillLossFunction.apply(zl, index, top.clone().requires_grad_())


def test_losses_in_a_graph_and_on_two_streams(qn):
    z, _, labels, start, ref, dloss = _pref_case(60, 3001, BF16, 2, seed=8)
    index = torch.randint(0, 3001, (60, 9), device="cuda")
    top = torch.randn(60, 9, device="cuda")

    def step():
        loss, L, st = qn.preference_loss_fwd(z, labels, start, ref)
        return (loss, L, qn.preference_loss_bwd(z, labels, st, dloss),
                *qn.distill_loss(z, index, top, labels, 2.0, 0.5, need_grad=True))

    step()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = step()
    for seed in (1, 2, 3):
        z.copy_(torch.randn(60, 3001, device="cuda") * seed)
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(p, q) for p, q in zip(out, step()))
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        a = step()
    b = step()
    side.synchronize()
    torch.cuda.synchronize()
    assert all(torch.equal(p, q) for p, q in zip(a, b))


def test_more_than_2_to_the_31_logits(qn):
    """Offsets past 32 bits: 17000 rows of 128002 values, checked at rows on
    both sides of 2^31."""
    T, V = 17000, 128002
    z = torch.empty(T, V, dtype=BF16, device="cuda")
    g = torch.Generator(device="cuda").manual_seed(0)
    for part in z.split(1000):
        part.copy_(2 * torch.randn(part.shape, generator=g, device="cuda"))
    labels = torch.randint(0, V, (T,), device="cuda")
    rows = torch.tensor([0, 1, 8191, 16776, 16777, 16778, 16999], device="cuda")
    want = torch.log_softmax(z[rows].double(), 1).gather(1, labels[rows, None])[:, 0]
    _close("logp", qn.token_logp(z, labels)[rows], want, _e(z[rows]) + 2.0 ** -22 * (want.abs() + 40))
    index = torch.randint(0, V, (T, 4), device="cuda")
    top = torch.randn(T, 4, device="cuda")
    wantd, told = _distill_exact(z[rows], index[rows], top[rows], None, 1.0, 0.0, None)
    loss, dz = qn.distill_loss(z, index, top, dlogits=z)  # in place
    _close("loss", loss[rows], wantd["loss"], told["loss"])
    _close("dz", dz[rows], wantd["dz"], told["dz"])


def test_a_spoiled_loss_gradient_stays_in_its_pair(qn):
    """NaN and infinities in dloss: rows in no sequence and of other pairs keep
    their gradients."""
    z, _, labels, _, ref, dloss = _pref_case(30, 257, F32, 2, seed=11, masked=0.2)
    start = torch.tensor([3, 8, 15, 20, 26], device="cuda")
    _, _, st = qn.preference_loss_fwd(z, labels, start, ref)
    base = qn.preference_loss_bwd(z, labels, st, dloss)
    for bad in (NAN, INF):
        d = dloss.clone()
        d[0] = bad
        dz = qn.preference_loss_bwd(z, labels, st, d)
        assert torch.equal(dz[15:26], base[15:26]) and not bool(dz[:3].any()) and not bool(dz[26:].any())
        counted = (labels[3:15] >= 0).nonzero()[:, 0] + 3
        assert not bool(dz[counted].isfinite().all(1).any())


def test_timers_count_the_launches(qn):
    z, _, labels, start, ref, dloss = _pref_case(12, 300, BF16, 1, seed=12)
    from bit_nf4_quantized_16_amd import _lib

    index, top = torch.randint(0, 300, (12, 3), device="cuda"), torch.randn(12, 3, device="cuda")
    X, w = torch.randn(4, 64, device="cuda"), torch.ones(64, device="cuda")

    def step():
        _, _, st = qn.preference_loss_fwd(z, labels, start, ref)
        qn.preference_loss_bwd(z, labels, st, dloss)
        qn.distill_loss(z, index, top)
        _, mean, rstd = qn.norm_fwd(X, w)
        qn.norm_bwd(X, w, X, mean, rstd)
        qn.epilogue_bwd(X.to(BF16), X, "silu")

    for kid, n in ((_lib.QL_KERNEL_LOGP, 1), (_lib.QL_KERNEL_PREFERENCE, 1), (_lib.QL_KERNEL_LOGP_GRAD, 1),
                   (_lib.QL_KERNEL_DISTILL, 1), (_lib.QL_KERNEL_NORM, 2), (_lib.QL_KERNEL_EPILOGUE, 1)):
        timer = qn.KernelTimer(kid)
        timer.arm()
        step()
        count, ms = timer.read()
        timer.disarm()
        assert count == n and ms > 0
