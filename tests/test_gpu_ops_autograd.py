"""The checkpoint operators under autograd: tensors written through ``out=``
count as modified, gradients are first order only, and nothing is kept or
computed that no gradient needs."""

import pytest
import torch

import workloads

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def qn():
    import bit_nf4_quantized_16_amd as qn

    assert torch.cuda.is_available()
    return qn


def _layer(qn, T=33, N=72, K=128, r=8, seed=0):
    w = qn.quantize_weight(workloads.normal_weight(N, K, 0.02, seed).cuda())
    t = lambda shape, s, i: workloads.bf16_normal(shape, s, seed + i).cuda()
    return w, t((T, K), 1.0, 1), t((T, N), 1.0, 2), t((r, K), 0.05, 3), t((N, r), 0.05, 4)


def test_a_checkpoint_written_again_is_refused_in_the_backward(qn):
    w, X, dY, A, B = _layer(qn)
    A.requires_grad_()
    x8 = qn.act8_quantize(X)
    Y = qn.QLoRALinearFunction.apply(X, A, B, w, 1.0, None, 0.0, x8)
    want = torch.autograd.grad(Y, A, dY, retain_graph=True)[0]
    assert torch.equal(torch.autograd.grad(Y, A, dY, retain_graph=True)[0], want)
    assert qn.act8_quantize(2 * X, out=x8) is x8
    with pytest.raises(RuntimeError, match="modified by an inplace operation"):
        torch.autograd.grad(Y, A, dY)


def test_a_keep_mask_written_again_is_refused_in_the_backward(qn):
    """The next step's mask drawn into the same memory before the backward."""
    w, X, dY, A, B = _layer(qn)
    A.requires_grad_()
    keep = workloads.pack_keep_bits(workloads.keep_mask(33, 128, 0.5, 8)).cuda()
    Y = qn.QLoRALinearFunction.apply(X, A, B, w, 1.0, keep, 0.5, True)
    torch.autograd.grad(Y, A, dY, retain_graph=True)
    keep.copy_(workloads.pack_keep_bits(workloads.keep_mask(33, 128, 0.5, 9)).cuda())
    with pytest.raises(RuntimeError, match="modified by an inplace operation"):
        torch.autograd.grad(Y, A, dY)


def test_every_out_counts_as_modified(qn):
    w, X, dY, A, B = _layer(qn)
    x8 = qn.act8_quantize(X)
    w4 = qn.q4g_quantize(workloads.normal_weight(72, 128, 0.02, 5).cuda(), group=32)
    outs = {
        "act8_dequantize": (torch.empty_like(X), lambda o: qn.act8_dequantize(x8, out=o)),
        "q4g_dequantize": (torch.empty(72, 128, device="cuda").bfloat16(), lambda o: qn.q4g_dequantize(w4, out=o)),
        "q4g_linear_fwd": (torch.empty(33, 72, device="cuda").bfloat16(), lambda o: qn.q4g_linear_fwd(w4, X, out=o)),
    }
    for name, (o, call) in outs.items():
        v = o._version
        assert call(o) is o and o._version > v, name
    U = torch.ones(33, 8, device="cuda")
    dA, dB = torch.zeros(8, 128, device="cuda"), torch.zeros(72, 8, device="cuda")
    va, vb = dA._version, dB._version
    qn.qlora_linear_bwd_act8(w, x8, dY, A, B, U=U, dA=dA, dB=dB, accumulate=True)
    assert dA._version > va and dB._version > vb
    va, vb = dA._version, dB._version
    qn.qlora_linear_bwd_group_act8([w], x8, [dY], [A], [B], Us=[U], dAs=[dA], dBs=[dB], accumulate=True)
    assert dA._version > va and dB._version > vb
    with torch.inference_mode():  # such tensors have no version
        i8 = qn.act8_quantize(X)
        qn.act8_quantize(X, out=i8)
    qn.act8_quantize(X, out=i8)
    assert torch.equal(i8.codes, x8.codes)


def test_second_order_by_the_adapters_is_refused(qn):
    w, X, dY, A, B = _layer(qn)
    A, B, dY = (t.requires_grad_() for t in (A, B, dY))
    spread = torch.stack([B, B], dim=2)[:, :, 0]  # B's values, not contiguous
    assert not spread.is_contiguous()
    for call in (lambda: qn.QLoRALinearFunction.apply(X, A, B, w, 1.0, None, 0.0, True),
                 lambda: qn.QLoRALinearFunction.apply(X, A, spread, w, 1.0, None, 0.0, True),
                 lambda: qn.QLoRAGroupAct8Function.apply(X, None, 1.0, [w], A, B)[0],
                 lambda: qn.QLoRAGroupAct8Function.apply(X, None, 1.0, [w], A, spread)[0]):
        gA, = torch.autograd.grad(call(), A, dY, create_graph=True)
        for leaf in (B, dY):  # dA = (s dY B)^T X
            with pytest.raises(RuntimeError, match="cannot be differentiated again"):
                torch.autograd.grad(gA.float().sum(), leaf, retain_graph=True)


def test_a_checkpoint_does_not_hold_the_input(qn):
    """What the backward keeps of X is its checkpoint, not its memory."""
    w, _, dY, A, B = _layer(qn, T=2048, N=64, K=2048)
    A.requires_grad_()
    torch.cuda.synchronize()
    before = torch.cuda.memory_allocated()
    X = torch.randn(2048, 2048, device="cuda").bfloat16().requires_grad_()
    held = lambda t: torch.cuda.memory_allocated() - before
    Z = X * 1  # not a leaf: only autograd would hold it
    Y = qn.QLoRALinearFunction.apply(Z, A, B, w, 1.0, None, 0.0, True)
    H = qn.SwiGLUFunction.apply(Z, Z)
    del Z
    # X, Y, H, three checkpoints, U; not Z (8 MiB)
    mine = X.nbytes + Y.nbytes + H.nbytes + 3 * 2048 * 2048 * 33 // 32 + 2048 * 8 * 4
    assert held(X) <= mine + (1 << 20)
    (Y.float().sum() + H.float().sum()).backward()


def test_second_order_is_refused(qn):
    """Also where dY is a constant (a plain sum), which is no argument of the
    backward that could require a gradient."""
    w, X, dY, A, B = _layer(qn)
    X, A, B = (t.requires_grad_() for t in (X, A, B))
    calls = {
        "linear": lambda: qn.QLoRALinearFunction.apply(X, A, B, w, 1.0, None, 0.0, True),
        "group": lambda: sum(qn.QLoRAGroupAct8Function.apply(X, None, 1.0, [w, w], A, B, A, B)),
        "swiglu": lambda: qn.SwiGLUFunction.apply(X, X),
    }
    for name, call in calls.items():
        want = torch.autograd.grad(call().sum(), X)[0]
        got, = torch.autograd.grad(call().sum(), X, create_graph=True)
        assert torch.equal(got, want), name
        assert got.requires_grad, name
        refused = pytest.raises(RuntimeError, match="cannot be differentiated again")
        with refused:
            torch.autograd.grad(got.float().square().sum(), X, retain_graph=True)
        with refused:  # beside a path that can be
            torch.autograd.grad((got * X).float().sum(), X, retain_graph=True)
        with refused:
            got.float().square().sum().backward()
        # the first order through create_graph stays usable, beside other paths
        other, = torch.autograd.grad((call().float() * 0).sum() + X.float().square().sum(), X, create_graph=True)
        assert torch.equal(other, (2 * X.float()).to(other.dtype)), name


SUBSETS = [(x, a, b) for x in (False, True) for a in (False, True) for b in (False, True) if x or a or b]


@pytest.mark.parametrize("need", SUBSETS)
@pytest.mark.parametrize("own", [False, True])
def test_linear_keeps_and_computes_what_is_needed(qn, need, own):
    w, X, dY, A, B = _layer(qn)
    full = [t.clone().requires_grad_() for t in (X, A, B)]
    want = torch.autograd.grad(qn.QLoRALinearFunction.apply(*full, w, 1.0, None, 0.0, True), full, dY)
    ins = [t.clone().requires_grad_(n) for t, n in zip((X, A, B), need)]
    Y = qn.QLoRALinearFunction.apply(*ins, w, 1.0, None, 0.0, qn.act8_quantize(X) if own else True)
    codes, scale, _, _, U, _ = Y.grad_fn.saved_tensors
    assert (codes is not None) == need[1] and (scale is not None) == need[1] and (U is not None) == need[2]
    timer = qn.KernelTimer(qn._lib.QL_KERNEL_ACT8_GRAD)
    timer.arm()
    got = torch.autograd.grad(Y, [t for t, n in zip(ins, need) if n], dY)
    torch.cuda.synchronize()
    launches = timer.read()[0]
    timer.disarm()
    assert (launches > 0) == (need[1] or need[2])
    for g, t in zip(got, [t for t, n in zip(want, need) if n]):
        assert torch.equal(g, t)


@pytest.mark.parametrize("need", [(1, 0, 0, 0, 0), (0, 1, 0, 0, 0), (0, 0, 1, 0, 0), (0, 0, 0, 1, 1), (1, 1, 0, 0, 1),
                                  (1, 0, 1, 1, 0), (1, 1, 1, 1, 1)])
def test_group_keeps_and_computes_what_is_needed(qn, need):
    """need: X, then A and B of two layers."""
    w, X, dY, A, B = _layer(qn)
    w2, _, dY2, A2, B2 = _layer(qn, N=40, seed=9)
    leaves = (X, A, B, A2, B2)
    full = [t.clone().requires_grad_() for t in leaves]
    call = lambda ts: qn.QLoRAGroupAct8Function.apply(ts[0], None, 1.0, [w, w2], *ts[1:])
    want = torch.autograd.grad(call(full), full, (dY, dY2))
    ins = [t.clone().requires_grad_(bool(n)) for t, n in zip(leaves, need)]
    Ys = call(ins)
    saved = Ys[0].grad_fn.saved_tensors
    assert (saved[0] is not None) == bool(need[1] or need[3])
    assert [u is not None for u in saved[6:]] == [bool(need[2]), bool(need[4])]
    got = torch.autograd.grad(Ys, [t for t in ins if t.requires_grad], (dY, dY2))
    for g, t in zip(got, [t for t, n in zip(want, need) if n]):
        assert torch.equal(g, t)
    # one output alone: the other layer's dY is zero
    ins = [t.clone().requires_grad_() for t in leaves]
    dX, dA, dB, dA2, dB2 = torch.autograd.grad(call(ins)[1], ins, dY2)
    assert torch.equal(dA2, want[3]) and torch.equal(dB2, want[4]) and not dA.any() and not dB.any()


def test_group_lists_of_wishes(qn):
    w, X, dY, A, B = _layer(qn)
    x8, U = qn.act8_quantize(X), qn.qlora_linear_fwd(w, X, A, B)[1]
    call = lambda **kw: qn.qlora_linear_bwd_group_act8([w, w], x8, [dY, dY], [A, A], [B, B], Us=[U, U], **kw)
    _, dAs, dBs = call()
    dX, a, b = call(need_dx=False, need_da=[False, True], need_db=(True, False))
    assert dX is None and a[0] is None and b[1] is None and torch.equal(a[1], dAs[1]) and torch.equal(b[0], dBs[0])
    _, a, b = call(need_da=[False, False], need_db=1)
    assert a is None and torch.equal(b[1], dBs[1])
    with pytest.raises(qn.QLoraError):
        call(need_da=[True])


@pytest.mark.parametrize("need", [(False, False), (True, False), (False, True), (True, True)])
@pytest.mark.parametrize("h8", [False, True])
def test_swiglu_keeps_and_returns_what_is_needed(qn, need, h8):
    T, F = 512, 1024
    g0, u0, dH = (workloads.bf16_normal((T, F), 1.0, s).cuda() for s in (1, 2, 3))
    g, u = g0.clone().requires_grad_(need[0]), u0.clone().requires_grad_(need[1])
    torch.cuda.synchronize()
    before = torch.cuda.memory_allocated()
    out = qn.SwiGLUFunction.apply(g, u, True) if h8 else qn.SwiGLUFunction.apply(g, u)
    H, a8 = out if h8 else (out, None)
    one = T * F * 33 // 32  # a checkpoint
    mine = H.nbytes + (2 * one if any(need) else 0) + (one if h8 else 0)
    assert mine <= torch.cuda.memory_allocated() - before < mine + one
    assert H.requires_grad == any(need)
    want = qn.swiglu_fwd(g0, u0, h8=True)
    assert torch.equal(H, want[0])
    if h8:
        assert torch.equal(a8.codes, want[3].codes) and torch.equal(a8.scale, want[3].scale)
    if any(need):
        got = torch.autograd.grad(H, [t for t in (g, u) if t.requires_grad], dH)
        full = qn.swiglu_bwd(want[1], want[2], dH)
        for a, b in zip(got, [t for t, n in zip(full, need) if n]):
            assert torch.equal(a, b)


def test_block_with_the_activations_own_checkpoint(qn):
    """gate/up, the gated activation and down with h8 handed on: the same
    gradients as with down storing H again."""
    T, D, F, r = 45, 128, 192, 8
    wg, wu = (qn.quantize_weight(workloads.normal_weight(F, D, 0.05, s).cuda()) for s in (1, 2))
    wd = qn.quantize_weight(workloads.normal_weight(D, F, 0.05, 3).cuda())
    leaves = [workloads.bf16_normal(s, 0.05, i).cuda().requires_grad_()
              for i, s in enumerate([(r, D), (F, r), (r, D), (F, r), (r, F), (D, r)])]
    X = workloads.bf16_normal((T, D), 1.0, 7).cuda().requires_grad_()
    dY = workloads.bf16_normal((T, D), 1.0, 8).cuda()

    def block(handed):
        G, U = qn.QLoRAGroupAct8Function.apply(X, None, 2.0, [wg, wu], *leaves[:4])
        H, h8 = qn.SwiGLUFunction.apply(G, U, True) if handed else (qn.SwiGLUFunction.apply(G, U), True)
        return qn.QLoRALinearFunction.apply(H, leaves[4], leaves[5], wd, 2.0, None, 0.0, h8)

    one, two = block(True), block(False)
    assert torch.equal(one, two)
    for a, b in zip(torch.autograd.grad(one, [X, *leaves], dY), torch.autograd.grad(two, [X, *leaves], dY)):
        assert torch.equal(a, b)
