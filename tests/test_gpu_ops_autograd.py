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
    for call in (lambda: qn.QLoRALinearFunction.apply(X, A, B, w, 1.0, None, 0.0, True),
                 lambda: qn.QLoRAGroupAct8Function.apply(X, None, 1.0, [w], A, B)[0]):
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
