"""The layer's backward from an 8-bit checkpoint of its input: dX bitwise the
ordinary backward's, dA and dB against the exact sums in 64 bits."""

import numpy as np
import pytest
import torch

import oracle
import workloads
from oracle import act8 as oa

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def qn():
    import bit_nf4_quantized_16_amd as qn

    assert torch.cuda.is_available()
    return qn


def _f64(t):
    return t.detach().cpu().double().numpy()


class Case:
    def __init__(self, qn, T, N, K, r, seed=1, dq=True, p=0.0, scale=0.5, u=None):
        self.T, self.N, self.K, self.r, self.scale, self.p = T, N, K, r, scale, p
        self.w = qn.quantize_weight(workloads.normal_weight(N, K, 0.02, seed).cuda(), double_quant=dq)
        self.X = workloads.bf16_normal((T, K), 1.0, seed + 1)
        self.dY = workloads.bf16_normal((T, N), 1.0, seed + 2)
        self.A = workloads.bf16_normal((r, K), 0.05, seed + 3)
        self.B = workloads.bf16_normal((N, r), 0.05, seed + 4)
        self.keep = workloads.keep_mask(T, K, p, seed + 5) if p > 0 else None
        self.bits = workloads.pack_keep_bits(self.keep).cuda() if p > 0 else None
        self.Xc, self.dYc, self.Ac, self.Bc = (t.cuda() for t in (self.X, self.dY, self.A, self.B))
        self.X8 = qn.act8_quantize(self.Xc)
        _, self.U = qn.qlora_linear_fwd(self.w, self.Xc, self.Ac, self.Bc, scale, keep=self.bits, p=p)

    def run(self, qn, **kw):
        kw = dict(dict(U=self.U, keep=self.bits, p=self.p), **kw)
        out = qn.qlora_linear_bwd_act8(self.w, self.X8, self.dYc, self.Ac, self.Bc, self.scale, **kw)
        torch.cuda.synchronize()
        return out

    def exact(self):
        """(dA, dB) in fp64 and their bounds. fp32 sums: G over N products, dA
        over T and dB over T, each step off by at most 2^-23 (MFMA partial
        sums included) of the sum of magnitudes; the split of G and U leaves
        2^-24, scale and c two roundings more."""
        d, B = _f64(self.dY), _f64(self.B)
        U = _f64(self.U)
        c = 1.0 / (1.0 - self.p)
        x = oa.act8_restore(_f64(self.X)) * (self.keep.numpy() if self.keep is not None else 1.0)
        G, Ga = self.scale * (d @ B), self.scale * (np.abs(d) @ np.abs(B))
        dA, dB = c * (G.T @ x), self.scale * (d.T @ U)
        bA = c * (Ga.T @ np.abs(x)) * (self.N + self.T + 8) * 2.0 ** -23
        bB = self.scale * (np.abs(d).T @ np.abs(U)) * (self.T + 8) * 2.0 ** -23
        return dA, dB, bA, bB


def _check(c, dA, dB):
    wA, wB, bA, bB = c.exact()
    assert np.all(np.abs(_f64(dA) - wA) <= bA)
    assert np.all(np.abs(_f64(dB) - wB) <= bB)


def _plain_dx(qn, c):
    return qn.qlora_linear_bwd(c.w, c.Xc, c.dYc, c.Ac, c.Bc, c.scale, U=c.U, keep=c.bits, p=c.p)[0]


# tokens, rows, columns, rank: one token, odd token counts, ragged rows and
# columns, ranks that are no multiple of 4 or 16, one over a tile, the largest
CASES = [(1, 8, 64, 1), (1, 256, 256, 16), (3, 40, 64, 3), (17, 72, 192, 5), (31, 264, 320, 8), (32, 64, 64, 16),
         (33, 104, 128, 33), (255, 136, 64, 64), (257, 64, 448, 100), (300, 320, 192, 128), (2048, 64, 64, 16),
         (2049, 72, 64, 20), (2500, 136, 192, 128)]


@pytest.mark.parametrize("T,N,K,r", CASES)
@pytest.mark.parametrize("p", [0.0, 0.3])
def test_gradients(qn, T, N, K, r, p):
    c = Case(qn, T, N, K, r, seed=T + N + r, p=p, dq=r % 2 == 0)
    dX, dA, dB = c.run(qn)
    _check(c, dA, dB)
    assert torch.equal(dX, _plain_dx(qn, c))


@pytest.mark.parametrize("T,N,K,r,p", [(1024, 4096, 4096, 16, 0.0), (1000, 11008, 4096, 16, 0.05)])
def test_model_shapes(qn, T, N, K, r, p):
    """The G projection inside the dX launch where the plan has it there."""
    c = Case(qn, T, N, K, r, seed=3, p=p)
    dX, dA, dB = c.run(qn)
    _check(c, dA, dB)
    assert torch.equal(dX, _plain_dx(qn, c))
    # far inside the bf16 rounding of G and U (2^-9 on average): fp32 sums
    wA, wB, _, _ = c.exact()
    for got, want in ((dA, wA), (dB, wB)):
        assert np.linalg.norm(_f64(got) - want) <= 2.0 ** -18 * np.linalg.norm(want)


@pytest.mark.parametrize("dx", [False, True])
@pytest.mark.parametrize("da", [False, True])
@pytest.mark.parametrize("db", [False, True])
def test_each_output_alone(qn, dx, da, db):
    c = Case(qn, 2100, 136, 192, 16, seed=5)
    full = c.run(qn)
    got = c.run(qn, need_dx=dx, need_da=da, need_db=db)
    for g, f, want in zip(got, full, (dx, da, db)):
        assert (g is not None) == want
    # the token split may differ with the columns asked for: sums in another order
    if dx:
        assert torch.equal(got[0], full[0])
    wA, wB, bA, bB = c.exact()
    if da:
        assert np.all(np.abs(_f64(got[1]) - wA) <= bA)
    if db:
        assert np.all(np.abs(_f64(got[2]) - wB) <= bB)


@pytest.mark.parametrize("T", [40, 2100])
def test_accumulate(qn, T):
    c = Case(qn, T, 72, 128, 12, seed=6)
    _, dA, dB = c.run(qn)
    a0, b0 = torch.randn_like(dA), torch.randn_like(dB)
    a1, b1 = a0.clone(), b0.clone()
    _, ra, rb = c.run(qn, dA=a1, dB=b1, accumulate=True)
    assert ra is a1 and rb is b1
    assert torch.equal(a1, a0 + dA) and torch.equal(b1, b0 + dB)
    c.run(qn, dA=a1, dB=b1)
    assert torch.equal(a1, dA) and torch.equal(b1, dB)


def test_rank_zero_and_no_tokens(qn):
    c = Case(qn, 33, 72, 128, 8, seed=7)
    dX, dA, dB = qn.qlora_linear_bwd_act8(c.w, None, c.dYc)
    assert dA is None and dB is None
    assert torch.equal(dX, qn.qlora_linear_bwd(c.w, None, c.dYc)[0])
    e = torch.empty(0, 72, dtype=torch.bfloat16, device="cuda")
    x8 = qn.act8_quantize(torch.empty(0, 128, dtype=torch.bfloat16, device="cuda"))
    dX, dA, dB = qn.qlora_linear_bwd_act8(c.w, x8, e, c.Ac, c.Bc, U=torch.empty(0, 8, device="cuda"))
    assert dX.shape == (0, 128) and not dA.any() and not dB.any()


def test_non_finite_input_stays_in_its_column(qn):
    """A NaN of X reaches only its column of dA, nothing of dB (U is given)
    and dX; an infinite dY entry its column of dB."""
    c = Case(qn, 50, 72, 128, 8, seed=8)
    _, dA, dB = c.run(qn)
    X = c.Xc.clone()
    X[7, 70] = float("nan")
    c.X8 = qn.act8_quantize(X)
    _, eA, eB = c.run(qn)
    assert torch.isnan(eA[:, 70]).all() and torch.equal(eB, dB)
    ok = torch.ones(128, dtype=torch.bool)
    ok[64:96] = False  # its block may have taken a finer scale
    assert torch.equal(eA[:, ok], dA[:, ok]) and torch.isfinite(eA[:, 71:]).all()
    c.dYc = c.dYc.clone()
    c.dYc[3, 5] = float("inf")
    _, _, fB = c.run(qn)
    assert not torch.isfinite(fB[5]).any()
    assert torch.equal(fB[:5], dB[:5]) and torch.equal(fB[6:], dB[6:])


def test_infinite_u_stays_infinite(qn):
    """An infinite entry of U times finite positive values is +inf, not NaN
    from the split into terms."""
    c = Case(qn, 9, 8, 64, 4, seed=9)
    c.U = torch.ones(9, 4, device="cuda")
    c.U[2, 1] = float("inf")
    c.dYc = torch.ones_like(c.dYc)
    _, _, dB = c.run(qn)
    assert torch.isposinf(dB[:, 1]).all() and torch.isfinite(dB[:, [0, 2, 3]]).all()


def test_repeatable(qn):
    c = Case(qn, 2100, 264, 320, 33, seed=10)
    one = c.run(qn)
    for _ in range(3):
        for a, b in zip(c.run(qn), one):
            assert torch.equal(a, b)


def test_memory_behind_the_arrays_stays(qn):
    c = Case(qn, 37, 72, 128, 7, seed=11)
    big = torch.full((7 + 2, 128), 7.0, device="cuda")
    bigb = torch.full((72 + 3, 7), 7.0, device="cuda")
    c.run(qn, dA=big[:7], dB=bigb[:72])
    assert bool((big[7:] == 7).all()) and bool((bigb[72:] == 7).all())
    # rows behind the last token are not read: poison them
    codes = torch.full((64, 128), 0x7F, dtype=torch.uint8, device="cuda")
    xs = torch.full((64, 4), 0xFF, dtype=torch.uint8, device="cuda")
    U, dY = torch.full((64, 7), float("nan"), device="cuda"), torch.full((64, 72), float("nan"), device="cuda",
                                                                         dtype=torch.bfloat16)
    codes[:37], xs[:37], U[:37], dY[:37] = c.X8.codes, c.X8.scale, c.U, c.dYc
    want = c.run(qn)
    c.X8, c.U, c.dYc = qn.Act8(37, 128, codes[:37], xs[:37]), U[:37], dY[:37]
    for a, b in zip(c.run(qn), want):
        assert torch.equal(a, b)


@pytest.mark.parametrize("T,Ns,r", [(1, (64, 72), 8), (40, (64, 72, 8), 16), (300, (136, 136), 33), (2100, (72, 40), 16)])
def test_group(qn, T, Ns, r):
    """dX bitwise the grouped backward's, dA and dB bitwise the single call's."""
    cs = [Case(qn, T, n, 192, r, seed=20) for n in Ns]
    for i, c in enumerate(cs):  # one X for all, other dY and adapters
        c.X8, c.Xc = cs[0].X8, cs[0].Xc
        c.dYc = (c.dYc * (i + 1)).contiguous()
        c.U = qn.qlora_linear_fwd(c.w, c.Xc, c.Ac, c.Bc, c.scale)[1]
    ws, dYs = [c.w for c in cs], [c.dYc for c in cs]
    As, Bs, Us = [c.Ac for c in cs], [c.Bc for c in cs], [c.U for c in cs]
    dX, dAs, dBs = qn.qlora_linear_bwd_group_act8(ws, cs[0].X8, dYs, As, Bs, 0.5, Us=Us)
    want = qn.qlora_linear_bwd_group(ws, cs[0].Xc, dYs, As, Bs, 0.5, Us=Us)[0]
    assert torch.equal(dX, want)
    for i, c in enumerate(cs):
        _, a, b = c.run(qn, need_dx=False)
        assert torch.equal(dAs[i], a) and torch.equal(dBs[i], b)
    only = qn.qlora_linear_bwd_group_act8(ws, cs[0].X8, dYs, As, Bs, 0.5, Us=Us, need_dx=False, need_db=False)
    assert only[0] is None and only[2] is None
    assert torch.equal(qn.qlora_linear_bwd_group_act8(ws, None, dYs)[0], qn.qlora_linear_bwd_group(ws, None, dYs)[0])


def test_gradients_against_differences(qn):
    """The loss sum(dY * Y) with Y of the restored X is linear in A and in B:
    its difference along a direction is the inner product with the gradient."""
    c = Case(qn, 37, 72, 128, 6, seed=30)
    x = oa.act8_restore(_f64(c.X))
    # dB takes U as saved; here that of the restored X
    c.U = torch.from_numpy(x @ _f64(c.A).T).float().cuda()
    _, dA, dB = c.run(qn)
    Wd = _f64(qn.nf4_dequantize(c.w))
    A, B, d = _f64(c.A), _f64(c.B), _f64(c.dY)
    loss = lambda a, b: float((d * oracle.lora_forward(x, Wd, a, b, c.scale)[0]).sum())
    rng = np.random.default_rng(0)
    for _ in range(3):
        EA, EB = rng.normal(size=A.shape), rng.normal(size=B.shape)
        for got, num in ((float((_f64(dA) * EA).sum()), (loss(A + 1e-3 * EA, B) - loss(A - 1e-3 * EA, B)) / 2e-3),
                         (float((_f64(dB) * EB).sum()), (loss(A, B + 1e-3 * EB) - loss(A, B - 1e-3 * EB)) / 2e-3)):
            # the sums of dA and dB are off by (N + T + 8) 2^-23 of their magnitudes at most
            _, _, bA, bB = c.exact()
            assert abs(got - num) <= max((bA * np.abs(EA)).sum(), (bB * np.abs(EB)).sum()) + 1e-8 * abs(num)


def test_captured_backward_replays(qn):
    c = Case(qn, 300, 264, 320, 16, seed=31)
    step = lambda: qn.qlora_linear_bwd_act8(c.w, qn.act8_quantize(c.Xc), c.dYc, c.Ac, c.Bc, c.scale, U=c.U)
    step()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = step()
    for i in range(3):
        c.Xc.copy_(workloads.bf16_normal((300, 320), 1.0, 50 + i).cuda())
        c.dYc.copy_(workloads.bf16_normal((300, 264), 1.0, 60 + i).cuda())
        graph.replay()
        torch.cuda.synchronize()
        for a, b in zip(out, step()):
            assert torch.equal(a, b)


def test_two_streams(qn):
    cs = [Case(qn, 515, 264, 320, 16, seed=s) for s in (40, 41)]
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


@pytest.mark.parametrize("T,p", [(5, 0.0), (48, 0.0), (48, 0.1)])
def test_autograd(qn, T, p):
    c = Case(qn, T, 72, 128, 8, seed=32, p=p)
    X, A, B = (t.clone().requires_grad_() for t in (c.Xc, c.Ac, c.Bc))
    Y = qn.QLoRALinearFunction.apply(X, A, B, c.w, c.scale, c.bits, p, True)
    assert torch.equal(Y, qn.QLoRALinearFunction.apply(X, A, B, c.w, c.scale, c.bits, p))
    dX, dA, dB = torch.autograd.grad(Y, (X, A, B), c.dYc)
    want = c.run(qn)
    assert torch.equal(dX, want[0])
    assert torch.equal(dA, want[1].bfloat16()) and torch.equal(dB, want[2].bfloat16())
    Y = qn.QLoRALinearFunction.apply(X.detach(), A, c.Bc, c.w, c.scale, c.bits, p, c.X8)
    assert torch.equal(torch.autograd.grad(Y, A, c.dYc)[0], dA)


def test_autograd_group(qn):
    cs = [Case(qn, 48, n, 128, 8, seed=33) for n in (72, 64)]
    X = cs[0].Xc.clone().requires_grad_()
    leaves = [t.clone().requires_grad_() for c in cs for t in (c.Ac, c.Bc)]
    Ys = qn.QLoRAGroupAct8Function.apply(X, None, 0.5, [c.w for c in cs], *leaves)
    grads = torch.autograd.grad(Ys, [X, *leaves], [c.dYc for c in cs])
    outs = qn.qlora_linear_fwd_group([c.w for c in cs], cs[0].Xc, leaves[0::2], leaves[1::2], 0.5)
    dX, dAs, dBs = qn.qlora_linear_bwd_group_act8([c.w for c in cs], cs[0].X8, [c.dYc for c in cs], leaves[0::2],
                                                  leaves[1::2], 0.5, Us=[U for _, U in outs])
    assert torch.equal(grads[0], dX)
    for i in range(2):
        assert torch.equal(grads[1 + 2 * i], dAs[i].bfloat16()) and torch.equal(grads[2 + 2 * i], dBs[i].bfloat16())


def test_mlp_block_with_checkpoints(qn):
    """gate and up sharing one checkpoint of X, the gated activation with its
    own, down with the activation's h8: the gradients of the three calls put
    together by hand, through autograd, are the same."""
    T, D, F, r = 45, 128, 192, 8
    wg, wu = (qn.quantize_weight(workloads.normal_weight(F, D, 0.05, s).cuda()) for s in (1, 2))
    wd = qn.quantize_weight(workloads.normal_weight(D, F, 0.05, 3).cuda())
    ad = [workloads.bf16_normal(s, 0.05, i).cuda().requires_grad_()
          for i, s in enumerate([(r, D), (F, r), (r, D), (F, r), (r, F), (D, r)])]
    X = workloads.bf16_normal((T, D), 1.0, 7).cuda().requires_grad_()
    dY = workloads.bf16_normal((T, D), 1.0, 8).cuda()
    G, U = qn.QLoRAGroupAct8Function.apply(X, None, 2.0, [wg, wu], *ad[:4])
    Y = qn.QLoRALinearFunction.apply(qn.SwiGLUFunction.apply(G, U), ad[4], ad[5], wd, 2.0, None, 0.0, True)
    got = torch.autograd.grad(Y, [X, *ad], dY)
    # by hand
    x = X.detach()
    a = [t.detach() for t in ad]
    x8 = qn.act8_quantize(x)
    (g, ug), (u, uu) = qn.qlora_linear_fwd_group([wg, wu], x, [a[0], a[2]], [a[1], a[3]], 2.0)
    h, g8, u8, h8 = qn.swiglu_fwd(g, u, h8=True)
    y, ud = qn.qlora_linear_fwd(wd, h, a[4], a[5], 2.0)
    dh, dad, dbd = qn.qlora_linear_bwd_act8(wd, h8, dY, a[4], a[5], 2.0, U=ud)
    dg, du = qn.swiglu_bwd(g8, u8, dh)
    dx, das, dbs = qn.qlora_linear_bwd_group_act8([wg, wu], x8, [dg, du], [a[0], a[2]], [a[1], a[3]], 2.0, Us=[ug, uu])
    want = [dx, das[0], dbs[0], das[1], dbs[1], dad, dbd]
    assert torch.equal(Y, y)
    for q, (s, t) in enumerate(zip(got, want)):
        assert torch.equal(s, t.to(s.dtype)), q
    # and near the block that keeps everything in bf16: an 8-bit value is off
    # by at most 2^-4, so each gradient stays well inside that, normwise
    G, U = qn.QLoRAGroupFunction.apply(X, 2.0, [wg, wu], *ad[:4])
    H = (torch.nn.functional.silu(G.float()) * U.float()).bfloat16()
    ref = torch.autograd.grad(qn.QLoRALinearFunction.apply(H, ad[4], ad[5], wd, 2.0), [X, *ad], dY)
    for s, t in zip(got, ref):
        assert float((s.float() - t.float()).norm()) <= 2.0 ** -4 * float(t.float().norm())


def test_refusals(qn):
    c = Case(qn, 40, 72, 128, 8, seed=12)
    bad = [dict(U=None), dict(U=c.U[:39]), dict(U=c.U.double()), dict(dA=torch.empty(8, 64, device="cuda")),
           dict(dB=torch.empty(72, 8, device="cuda").bfloat16()), dict(p=0.5), dict(keep=c.X8.codes, p=0.5)]
    for kw in bad:
        with pytest.raises((qn.QLoraError, RuntimeError)):
            c.run(qn, **kw)
    for x8 in (None, qn.act8_quantize(c.Xc[:39].contiguous()), qn.act8_quantize(c.Xc[:, :64].contiguous())):
        with pytest.raises(qn.QLoraError):
            qn.qlora_linear_bwd_act8(c.w, x8, c.dYc, c.Ac, c.Bc, U=c.U)
    with pytest.raises(qn.QLoraError):
        qn.qlora_linear_bwd_act8(c.w, c.X8, c.dYc, c.Ac[:, :64].contiguous(), c.Bc, U=c.U)
    with pytest.raises(qn.QLoraError):
        qn.qlora_linear_bwd_act8(c.w, c.X8, c.dYc.float(), c.Ac, c.Bc, U=c.U)
    with pytest.raises(qn.QLoraError):
        qn.QLoRALinearFunction.apply(c.Xc, c.Ac, c.Bc, c.w, 1.0, None, 0.0, qn.act8_quantize(c.Xc[:39].contiguous()))
