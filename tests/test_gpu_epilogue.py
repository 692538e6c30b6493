"""The linear forwards with bias, activation and residual, and the epilogue's
backward, against the 64-bit formulas element by element. Bounds: a product's
sum passes through at most K / 8 + 64 roundings of its terms' absolute values;
on the NF4 weight past 16 tokens s U enters as two bf16 terms (2^-16 of the
adapter term's absolute values); activations have slopes of
at most 1.13, are formed to 2^-16 of the value (the normal distribution
function to 1.1e-5) and the sum is rounded to bf16 once."""

import math

import pytest
import torch

import workloads

pytestmark = pytest.mark.gpu

BF16 = torch.bfloat16
HALF = torch.finfo(BF16).eps / 2
ACTS = ("none", "silu", "gelu", "gelu_tanh")


@pytest.fixture(scope="module")
def qn():
    import bit_nf4_quantized_16_amd as qn

    assert torch.cuda.is_available()
    return qn


def _act(z, act):
    """Value and slope in 64 bits."""
    if act == "none":
        return z, torch.ones_like(z)
    if act == "gelu":
        c = torch.special.ndtr(z)
        return z * c, c + z * torch.exp(-z * z / 2) / math.sqrt(2 * math.pi)
    k = 2 * math.sqrt(2 / math.pi)
    u, du = (z, torch.ones_like(z)) if act == "silu" else (k * (z + 0.044715 * z ** 3), k * (1 + 0.134145 * z * z))
    return z * torch.sigmoid(u), torch.sigmoid(u) * (1 + z * du * torch.sigmoid(-u))


def _close(name, got, want, tol):
    bad = (got.double() - want).abs() - ((HALF if got.dtype == BF16 else 2.0 ** -24) * want.abs() + tol)
    assert got.shape == want.shape and float(bad.max()) <= 0, (name, float(bad.max()))


def _rnd(g, *s, std=1.0):
    return (std * torch.randn(*s, generator=g, device="cuda")).to(BF16)


def _nf4_case(qn, T, N, K, r, seed, dq=True):
    g = torch.Generator(device="cuda").manual_seed(seed)
    w = qn.quantize_weight((0.02 * torch.randn(N, K, generator=g, device="cuda")), double_quant=dq)
    A = _rnd(g, r, K, std=0.02) if r else None
    B = _rnd(g, N, r, std=0.1) if r else None
    return w, _rnd(g, T, K), A, B, _rnd(g, N, std=0.7), _rnd(g, T, N)


def _z(qn, w, X, A, B, s, bias, rows=slice(None), keep=None, c=1.0):
    """z and its bound in 64 bits."""
    W = qn.nf4_dequantize(w).double()[rows]
    x, K = X.double(), X.shape[1]
    e = (K / 8 + 64) * 2.0 ** -24
    z = torch.mm(x, W.t().contiguous())
    tol = e * torch.mm(x.abs(), W.t().abs().contiguous())
    if A is not None:
        xa = x if keep is None else x * keep
        u, b = c * torch.mm(xa, A.double().t().contiguous()), B.double()[rows].t().contiguous()
        au = c * torch.mm(xa.abs(), A.double().t().abs().contiguous())
        z = z + s * torch.mm(u, b)
        tol = tol + abs(s) * (2.0 ** -16 * torch.mm(u.abs(), b.abs()) + 2 * e * torch.mm(au, b.abs()))
    if bias is not None:
        z = z + bias.double()[rows]
        tol = tol + 2.0 ** -23 * bias.double()[rows].abs()
    return z, tol + 2.0 ** -23 * z.abs()


def _check_nf4(qn, case, s, act, use_bias, use_res, rows=slice(None), keep=None, p=0.0, bits=None):
    w, X, A, B, bias, res = case
    bias, res = bias if use_bias else None, res if use_res else None
    Y, U, Z = qn.qlora_linear_fwd_epilogue(w, X, A, B, s, bias, act, res, save_z=True, keep=keep, p=p)
    Y2, _, Z2 = qn.qlora_linear_fwd_epilogue(w, X, A, B, s, bias, act, res, save_u=False, save_z=BF16, keep=keep, p=p)
    assert Z.dtype == torch.float32 and torch.equal(Z.to(BF16), Z2) and torch.equal(Y, Y2)
    z, tz = _z(qn, w, X, A, B, s, bias, rows, bits, 1 / (1 - p))
    _close("Z", Z[:, rows], z, tz)
    v, _ = _act(z, act)
    want = v if res is None else v + res.double()[:, rows]
    _close("Y", Y[:, rows], want, 1.13 * tz + 2.0 ** -16 * v.abs() + 2.0 ** -23 * want.abs())
    return Y, U, Z


# T, N, K, r: decode in every width and ring; 17 to 1000 tokens in every tile and
# split, ranks on and off the padded paths, U inside the GEMM's launch
SHAPES = [(1, 8, 64, 0), (1, 264, 192, 8), (2, 4096, 4096, 16), (3, 520, 1088, 3), (5, 72, 11008, 64), (16, 264, 4096, 33),
          (17, 8, 64, 3), (17, 264, 192, 0), (40, 520, 1088, 16), (33, 256, 8192, 64), (300, 1024, 512, 8),
          (300, 72, 320, 33), (130, 4096, 4096, 16), (1000, 264, 448, 128)]


@pytest.mark.parametrize("T,N,K,r", SHAPES)
def test_nf4(qn, T, N, K, r):
    case = _nf4_case(qn, T, N, K, r, seed=T + N + K + r, dq=(N // 8) % 2 == 1)
    w, X, A, B, bias, res = case
    for act in ACTS:
        for use_bias, use_res in ((True, True), (False, True), (True, False)):
            Y, U, Z = _check_nf4(qn, case, 0.7, act, use_bias, use_res)
    # nothing asked for: the plain forward's U (and Y, to 16 tokens); the residual in place
    Y0, U0 = qn.qlora_linear_fwd(w, X, A, B, 0.7)
    Y1, U1, none = qn.qlora_linear_fwd_epilogue(w, X, A, B, 0.7)
    assert none is None and (T > 16 or torch.equal(Y0, Y1)) and (U0 is None or torch.equal(U0, U1))
    assert U is None or torch.equal(U0, U)
    Y2, _, _ = qn.qlora_linear_fwd_epilogue(w, X, A, B, 0.7, bias, "gelu", res)
    r2 = res.clone()
    Y3, _, _ = qn.qlora_linear_fwd_epilogue(w, X, A, B, 0.7, bias, "gelu", r2, out=r2)
    assert Y3 is r2 and torch.equal(Y2, Y3)


@pytest.mark.parametrize("T,N,K,r", [(1024, 11008, 4096, 16), (1001, 11008, 4096, 64), (300, 4096, 11008, 16)])
def test_nf4_full_size(qn, T, N, K, r):
    """The 7B MLP shapes, every 61st output: U inside the launch and beside it,
    the reduction split."""
    case = _nf4_case(qn, T, N, K, r, seed=r)
    rows = torch.arange(0, N, 61, device="cuda")
    for act in ("gelu", "silu"):
        _check_nf4(qn, case, 0.5, act, True, True, rows=rows)


@pytest.mark.parametrize("tile,splits", [("128", None), ("256", "1"), ("256", "3")])
def test_nf4_every_plan(qn, monkeypatch, tile, splits):
    monkeypatch.setenv("QLORA_NF4_GEMM_TILE", tile)
    if splits:
        monkeypatch.setenv("QLORA_NF4_GEMM_SPLITS", splits)
    for T, N, K, r in ((77, 264, 1088, 16), (300, 520, 512, 5)):
        case = _nf4_case(qn, T, N, K, r, seed=T)
        for act in ACTS:
            _check_nf4(qn, case, 0.7, act, True, True)


def test_nf4_dropout(qn):
    for T in (1, 40):
        case = _nf4_case(qn, T, 264, 192, 8, seed=T)
        keep = workloads.keep_mask(T, 192, 0.25, seed=3)
        bits = workloads.pack_keep_bits(keep).cuda()
        _check_nf4(qn, case, 0.7, "silu", True, True, keep=bits, p=0.25, bits=keep.cuda().double())


def test_nothing_behind_the_outputs_is_written(qn):
    for T, N, K, r in ((3, 264, 192, 8), (40, 264, 192, 8), (300, 520, 512, 16)):
        w, X, A, B, bias, res = _nf4_case(qn, T, N, K, r, seed=T)
        buf = torch.full((T * N + 256,), 7.0, dtype=BF16, device="cuda")
        Y, _, Z = qn.qlora_linear_fwd_epilogue(w, X, A, B, 1.0, bias, "gelu", res, save_z=True)
        qn.qlora_linear_fwd_epilogue(w, X, A, B, 1.0, bias, "gelu", res, out=buf[:T * N].view(T, N))
        assert torch.equal(buf[:T * N].view(T, N), Y) and bool((buf[T * N:] == 7).all())


def _q4g_z(qn, w, X, bias):
    W = qn.q4g_dequantize(w, torch.float32).double().t().contiguous()
    # the codes' sums and the zero points' are apart: terms s q and s z with q, z up to 15
    big = w.scale.double().repeat_interleave(w.group, 1)[:, :w.cols].t().contiguous() * 15
    z = torch.mm(X.double(), W)
    tol = (X.shape[1] / 8 + 64) * 2.0 ** -24 * 2 * torch.mm(X.double().abs(), big)
    if bias is not None:
        z = z + bias.double()
    return z, tol + 2.0 ** -22 * z.abs()


@pytest.mark.parametrize("T,N,K,group,sym", [(1, 8, 32, 32, False), (1, 4096, 4096, 128, False), (4, 264, 200, 64, True),
                                             (8, 520, 1088, 32, False), (7, 16400, 128, 128, True), (16, 264, 4096, 128, False),
                                             (13, 72, 1000, 32, True), (24, 520, 512, 64, False), (64, 1032, 264, 128, False),
                                             (130, 264, 512, 32, True)])
def test_q4g(qn, T, N, K, group, sym):
    g = torch.Generator(device="cuda").manual_seed(T + N)
    w = qn.q4g_quantize(0.02 * torch.randn(N, K, generator=g, device="cuda"), group, sym)
    X, bias, res = _rnd(g, T, K), _rnd(g, N, std=0.7), _rnd(g, T, N)
    for act in ACTS:
        for b, r in ((bias, res), (None, res), (bias, None)):
            Y = qn.q4g_linear_fwd_epilogue(w, X, b, act, r)
            z, tz = _q4g_z(qn, w, X, b)
            v, _ = _act(z, act)
            want = v if r is None else v + r.double()
            _close("Y", Y, want, 1.13 * tz + 2.0 ** -16 * v.abs() + 2.0 ** -23 * want.abs())
    assert torch.equal(qn.q4g_linear_fwd_epilogue(w, X), qn.q4g_linear_fwd(w, X))
    want = qn.q4g_linear_fwd_epilogue(w, X, bias, "silu", res)
    assert qn.q4g_linear_fwd_epilogue(w, X, bias, "silu", res, out=res) is res and torch.equal(res, want)


def test_infinities_and_nan(qn):
    """A token's stay its own; act of infinities is the documented one."""
    w, X, A, B, bias, res = _nf4_case(qn, 20, 264, 192, 8, seed=1)
    q4 = qn.q4g_quantize(qn.nf4_dequantize(w), 32)
    X2, b2 = X.clone(), bias.clone()
    X2[3, 5] = float("nan")
    b2[7], b2[9] = float("inf"), float("-inf")
    for act in ("silu", "gelu", "gelu_tanh"):
        for T in (5, 20):
            for call in (lambda x, b: qn.qlora_linear_fwd_epilogue(w, x[:T], A, B, 1.0, b, act)[0],
                         lambda x, b: qn.q4g_linear_fwd_epilogue(q4, x[:T], b, act)):
                base, got, nan = call(X, bias), call(X, b2), call(X2, bias)
                keep = torch.ones(264, dtype=torch.bool, device="cuda")
                keep[[7, 9]] = False
                assert torch.equal(got[:, keep], base[:, keep])
                assert bool((got[:, 7] == float("inf")).all()) and bool(got[:, 9].isnan().all())
                rows = torch.arange(T, device="cuda") != 3
                assert torch.equal(nan[rows], base[rows]) and bool(nan[3].isnan().all())


@pytest.mark.parametrize("zt", [BF16, torch.float32])
@pytest.mark.parametrize("act", ACTS)
@pytest.mark.parametrize("T,N", [(1, 8), (3, 16), (17, 264), (64, 72), (300, 512), (1000, 1032), (5, 11008), (2500, 24)])
def test_backward(qn, T, N, act, zt):
    g = torch.Generator(device="cuda").manual_seed(T + N)
    dY, Z = _rnd(g, T, N), (2.5 * torch.randn(T, N, generator=g, device="cuda")).to(zt)
    dZ, db = qn.epilogue_bwd(dY, Z, act)
    _, slope = _act(Z.double(), act)
    z = Z.double().abs().clamp(max=8)
    e = dY.double().abs() * (2.0 ** -16 + 2.0 ** -21 * (1 + z + z ** 3)) * (act != "none")
    want = dY.double() * slope
    _close("dZ", dZ, want, e)
    _close("db", db, want.sum(0), e.sum(0) + (T / 8 + 300) * 2.0 ** -24 * want.abs().sum(0))
    if act == "none":
        assert dZ is dY
    assert torch.equal(qn.epilogue_bwd(dY, Z, act, need_dbias=False)[0], dZ)
    assert torch.equal(qn.epilogue_bwd(dY, Z, act, need_dz=False)[1], db)
    acc = torch.ones(N, device="cuda")
    assert torch.equal(qn.epilogue_bwd(dY, Z, act, dbias=acc, accumulate=True)[1], 1 + db)
    none, zero = qn.epilogue_bwd(dY[:0], Z[:0], act)
    assert none.shape == (0, N) and not bool(zero.any())


def test_slopes_everywhere(qn):
    """Every finite bf16 z: far out the slopes are 0 and 1."""
    bits = torch.arange(1 << 16, dtype=torch.int32, device="cuda").to(torch.int16).view(BF16)
    Z = torch.nn.functional.pad(bits[bits.isfinite()], (0, 0)).view(1, -1)
    Z = Z[:, :Z.shape[1] // 8 * 8].contiguous()
    dY = torch.ones_like(Z)
    for act in ACTS[1:]:
        dZ, _ = qn.epilogue_bwd(dY, Z, act, need_dbias=False)
        z = Z.double()
        _, slope = _act(z.clamp(-60, 60), act)
        c = z.abs().clamp(max=8)
        _close(act, dZ, slope, 2.0 ** -16 + 2.0 ** -21 * (1 + c + c ** 3))


def test_autograd(qn):
    g = torch.Generator(device="cuda").manual_seed(2)
    for T, act, res_on in ((24, "gelu", True), (5, "silu", False), (300, "gelu_tanh", True), (24, "none", True)):
        w, X, A, B, bias, res = _nf4_case(qn, T, 72, 128, 8, seed=T)
        leaves = [t.clone().requires_grad_() for t in (X, A, B, bias, res)]
        dY = _rnd(g, T, 72)
        Y = qn.QLoRALinearEpilogueFunction.apply(leaves[0], leaves[1], leaves[2], w, 0.5, leaves[3], act,
                                                 leaves[4] if res_on else None)
        got = torch.autograd.grad(Y, leaves if res_on else leaves[:4], dY)
        W = qn.nf4_dequantize(w).double()
        x, a, b, c, r = [t.double().requires_grad_() for t in (X, A, B, bias, res)]
        z = x @ W.t() + 0.5 * (x @ a.t()) @ b.t() + c
        want = torch.autograd.grad(_act(z, act)[0] + r, (x, a, b, c, r), dY.double())
        for n, p, q in zip("X A B bias res".split(), got, want):
            assert p.dtype == BF16 and p.shape == q.shape
            # dZ is a bf16 operand of the other gradients: 2^-9 of each term, 2e-2 normwise
            assert float((p.double() - q).abs().max()) <= 2e-2 * float(q.abs().max()), n
        assert not res_on or torch.equal(got[4], dY)
    # one leaf at a time, broadcast gradients and views
    for i in range(5):
        ts = [t.clone().requires_grad_(i == j) for j, t in enumerate((X, A, B, bias, res))]
        Y = qn.QLoRALinearEpilogueFunction.apply(*ts[:3], w, 0.5, ts[3], "gelu", ts[4])
        Y.float().sum().backward()
        assert [t.grad is not None for t in ts] == [i == j for j in range(5)]
    xt = X.t().contiguous().t().requires_grad_()
    y1 = qn.QLoRALinearEpilogueFunction.apply(xt, A, B, w, 0.5, bias, "gelu")
    x1 = X.clone().requires_grad_()
    y2 = qn.QLoRALinearEpilogueFunction.apply(x1, A, B, w, 0.5, bias, "gelu")
    y1.float().sum().backward(), y2.float().sum().backward()
    assert torch.equal(y1, y2) and torch.equal(xt.grad, x1.grad)
    # no adapters; second order is refused
    y = qn.QLoRALinearEpilogueFunction.apply(x1, None, None, w, 1.0, None, "silu")
    gx, = torch.autograd.grad(y.float().sum(), x1, create_graph=True)
    with pytest.raises(RuntimeError, match="cannot be differentiated again"):
        torch.autograd.grad(gx.float().sum(), x1)


@pytest.mark.parametrize("T", [1, 24, 300])
def test_graph_replays_and_two_streams(qn, T):
    w, X, A, B, bias, res = _nf4_case(qn, T, 1024, 512, 8, seed=T)
    q4 = qn.q4g_quantize(qn.nf4_dequantize(w), 64)
    dY = torch.ones_like(res)

    def step():
        Y, U, Z = qn.qlora_linear_fwd_epilogue(w, X, A, B, 0.5, bias, "gelu", res, save_z=True)
        return (Y, U, *qn.epilogue_bwd(dY, Z, "gelu"), qn.q4g_linear_fwd_epilogue(q4, X, bias, "silu", res))

    step()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = step()
    for seed in (1, 2, 3):
        g = torch.Generator(device="cuda").manual_seed(seed)
        X.copy_(_rnd(g, *X.shape)), res.copy_(_rnd(g, *res.shape))
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


@pytest.mark.parametrize("N,K,T,r", [(1024, 512, 300, 16), (520, 256, 33, 8)])
def test_u_inside_the_launch(qn, monkeypatch, N, K, T, r):
    """The same bits as with U beside the launch; and where a tile does not wait
    for the words and forms U itself, in two terms as well, the formula."""
    monkeypatch.setenv("QLORA_NF4_GEMM_TILE", "256")
    assert qn.lib.qlora_linear_fwd_u_in_launch(N, K, T, r) == 1
    case = _nf4_case(qn, T, N, K, r, seed=9)
    w, X, A, B, bias, res = case
    for act in ("none", "gelu"):
        call = lambda: qn.qlora_linear_fwd_epilogue(w, X, A, B, 0.7, bias, act, res, save_z=True)
        inside = call()
        with monkeypatch.context() as m:
            m.setenv("QLORA_NF4_FWD_U", "prepass")
            assert all(torch.equal(p, q) for p, q in zip(inside, call()))
        for spin in ("-1", "0"):
            with monkeypatch.context() as m:
                m.setenv("QLORA_NF4_GEMM_SPIN", spin)
                Y, U, Z = call()
            z, tz = _z(qn, w, X, A, B, 0.7, bias)
            # a tile's U is a chain of K products
            u = torch.mm(X.double().abs(), A.double().t().abs().contiguous())
            tz = tz + 0.7 * K * 2.0 ** -24 * torch.mm(u, B.double().t().abs().contiguous())
            _close("Z", Z, z, tz)
            v, _ = _act(z, act)
            want = v + res.double()
            _close("Y", Y, want, 1.13 * tz + 2.0 ** -16 * v.abs() + 2.0 ** -23 * want.abs())
