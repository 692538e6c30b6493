"""Calls on 8-bit checkpoints and 4-bit group weights that the other tests do
not make: large arrays, several threads, other streams, captured wide products,
and arguments that must be refused."""

import threading

import pytest
import torch

import workloads

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def qn():
    import bit_nf4_quantized_16_amd as qn

    assert torch.cuda.is_available()
    return qn


def _layer(qn, T, N, K, r, seed=3):
    w = qn.quantize_weight(workloads.normal_weight(N, K, 0.02, seed).cuda())
    X, dY, A, B = (workloads.bf16_normal(s, std, seed + i).cuda()
                   for i, (s, std) in enumerate((((T, K), 1.0), ((T, N), 1.0), ((r, K), 0.05), ((N, r), 0.05))))
    return w, X, dY, A, B


def test_activation_over_2_31_values(qn):
    """2.2e9 values: rows behind 2^31 as a call of their own gives them."""
    rows, cols, tail = 200000, 11008, 5
    X = torch.empty(rows, cols, dtype=torch.bfloat16, device="cuda").fill_(1.0)
    X[-tail:] = workloads.bf16_normal((tail, cols), 1.0, 1).cuda()
    up = torch.empty_like(X).fill_(-0.5)
    up[-tail:] = workloads.bf16_normal((tail, cols), 1.0, 2).cuda()
    H, g8, u8, h8 = qn.swiglu_fwd(X, up, h8=True)
    sH, sg8, su8, sh8 = qn.swiglu_fwd(X[-tail:].contiguous(), up[-tail:].contiguous(), h8=True)
    assert torch.equal(H[-tail:], sH)
    for big, small in ((g8, sg8), (u8, su8), (h8, sh8)):
        assert torch.equal(big.codes[-tail:], small.codes) and torch.equal(big.scale[-tail:], small.scale)
    a = qn.act8_quantize(X)
    assert torch.equal(a.codes[-tail:], g8.codes[-tail:]) and torch.equal(a.scale, g8.scale)
    del H, h8, a
    assert torch.equal(qn.act8_dequantize(g8)[-tail:], qn.act8_dequantize(sg8))
    dg, du = qn.swiglu_bwd(g8, u8, X)
    sdg, sdu = qn.swiglu_bwd(sg8, su8, X[-tail:].contiguous())
    assert torch.equal(dg[-tail:], sdg) and torch.equal(du[-tail:], sdu)


def test_checkpoint_gradients_over_2_31_values(qn):
    """T K over 2^31 and T N over 2^31: with small integers every sum is exact,
    and only the last tokens count."""
    T, N, K, r, tail = 300000, 8192, 8192, 4, 40
    w = qn.quantize_weight(torch.zeros(N, K, device="cuda"))
    gen = torch.Generator("cuda").manual_seed(5)
    ints = lambda *s: torch.randint(-2, 3, s, device="cuda", generator=gen)
    X = torch.zeros(T, K, dtype=torch.bfloat16, device="cuda")
    X[-tail:] = ints(tail, K).bfloat16()
    dY = torch.zeros(T, N, dtype=torch.bfloat16, device="cuda")
    dY[-tail:] = ints(tail, N).bfloat16()
    A, B, U = ints(r, K).bfloat16(), ints(N, r).bfloat16(), ints(T, r).float()
    X8 = qn.act8_quantize(X)
    _, dA, dB = qn.qlora_linear_bwd_act8(w, X8, dY, A, B, 1.0, U=U, need_dx=False)
    d = dY[-tail:].double()
    G = (d[:, :, None] * B.double()).sum(1)
    assert torch.equal(dA.double(), (G[:, :, None] * X[-tail:].double()[:, None, :]).sum(0))
    assert torch.equal(dB.double(), (d[:, :, None] * U[-tail:].double()[:, None, :]).sum(0))


def test_group_weight_over_2_31_values(qn):
    """2.2e9 values and, with 4100 tokens, outputs over 2^31."""
    N, K, tail, T = 540000, 4096, 19, 4100
    W = torch.empty(N, K, dtype=torch.bfloat16, device="cuda").fill_(0.01)
    W[-tail:] = workloads.bf16_normal((tail, K), 0.02, 3).cuda()
    w = qn.q4g_quantize(W, group=64)
    small = qn.q4g_quantize(W[-tail:].contiguous(), group=64)
    assert torch.equal(w.packed[-tail:], small.packed)
    assert torch.equal(w.scale[-tail:], small.scale) and torch.equal(w.zero[-tail:], small.zero)
    assert torch.equal(qn.q4g_dequantize(w)[-tail:], qn.q4g_dequantize(small))
    del W
    X = workloads.bf16_normal((T, K), 1.0, 4).cuda()
    wd = qn.q4g_dequantize(small, torch.float32).double()
    z = small.zero.double()[:, torch.arange(K, device="cuda") // 64]
    s = small.scale.double()[:, torch.arange(K, device="cuda") // 64]
    for t in (1, 7, 30, T):
        Y = qn.q4g_linear_fwd(w, X[:t])
        got = Y[-1:, -tail:].double()
        x = X[t - 1:t].double()
        y, mag = x @ wd.t().contiguous(), x.abs() @ (wd.abs() + 2 * s * z).t().contiguous()
        assert bool(((got - y).abs() <= y.abs() * 2.0 ** -8 + mag * (K + 8) * 2.0 ** -23).all())
        del Y


@pytest.mark.parametrize("T,N,K,group", [(24, 72, 520, 64), (40, 4128, 1032, 32), (64, 16500, 1288, 32), (130, 4090, 776, 128)])
def test_captured_wide_products_replay(qn, T, N, K, group):
    """Tokens for the wider kernels, whose LDS passes 64 KiB: each replay, with
    eager work between, gives the eager call's bits."""
    w = qn.q4g_quantize(workloads.normal_weight(N, K, 0.02, 1).cuda(), group=group)
    X = workloads.bf16_normal((T, K), 1.0, 2).cuda()
    out = torch.empty(T, N, dtype=torch.bfloat16, device="cuda")
    qn.q4g_linear_fwd(w, X, out=out)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        qn.q4g_linear_fwd(w, X, out=out)
    for i in range(4):
        X.copy_(workloads.bf16_normal((T, K), 1.0, 10 + i).cuda())
        want = qn.q4g_linear_fwd(w, X)
        out.zero_()
        g.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, want)


def test_two_graphs_of_the_backward(qn):
    """Two captured backwards replayed in turn and together, each with its own
    workspace, beside eager calls."""
    cases = [_layer(qn, T, 136, 192, r, seed) for T, r, seed in ((70, 8, 3), (33, 40, 9))]
    graphs, outs, wants = [], [], []
    for w, X, dY, A, B in cases:
        X8 = qn.act8_quantize(X)
        _, U = qn.qlora_linear_fwd(w, X, A, B, 0.5)
        run = lambda w=w, X8=X8, dY=dY, A=A, B=B, U=U: qn.qlora_linear_bwd_act8(w, X8, dY, A, B, 0.5, U=U)
        wants.append([t.clone() for t in run()])
        torch.cuda.synchronize()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            outs.append(run())
        graphs.append((g, run))
    side = torch.cuda.Stream()
    for _ in range(4):
        for o in outs:
            for t in o:
                t.zero_()
        side.wait_stream(torch.cuda.current_stream())
        graphs[0][0].replay()
        with torch.cuda.stream(side):
            graphs[1][0].replay()
        eager = graphs[0][1]()
        torch.cuda.synchronize()
        for o, want in zip(outs + [eager], wants + [wants[0]]):
            assert all(torch.equal(a, b) for a, b in zip(o, want))


def test_threads(qn):
    """Calls from four threads at once, each on a stream of its own, give the
    single thread's bits, and an error stays with its thread."""
    w, X, dY, A, B = _layer(qn, 50, 200, 256, 12)
    q = qn.q4g_quantize(workloads.normal_weight(200, 256, 0.02, 5).cuda(), group=32)

    def work():
        X8 = qn.act8_quantize(X)
        _, U = qn.qlora_linear_fwd(w, X, A, B, 0.5)
        H, g8, u8, _ = qn.swiglu_fwd(X, X)
        return [X8.codes, *qn.qlora_linear_bwd_act8(w, X8, dY, A, B, 0.5, U=U), H, *qn.swiglu_bwd(g8, u8, X),
                qn.q4g_linear_fwd(q, X), qn.q4g_linear_fwd(q, X[:3])]

    want = work()
    torch.cuda.synchronize()
    bad = []

    def thread(i):
        try:
            with torch.cuda.stream(torch.cuda.Stream()):
                for _ in range(10):
                    if i == 0:
                        with pytest.raises(qn.QLoraError):
                            qn.q4g_quantize(X[:, :12].contiguous())
                    got = work()
                    torch.cuda.current_stream().synchronize()
                    if not all(torch.equal(a, b) for a, b in zip(got, want)):
                        bad.append(i)
                torch.cuda.current_stream().synchronize()
        except BaseException as e:  # noqa: BLE001
            bad.append(e)

    threads = [threading.Thread(target=thread, args=(i,)) for i in range(4)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    torch.cuda.synchronize()
    assert not bad, bad


def test_one_tensor_in_several_places(qn):
    """The same weight twice in a group, gate and up from one tensor."""
    w, X, dY, A, B = _layer(qn, 40, 96, 128, 8)
    X8 = qn.act8_quantize(X)
    _, U = qn.qlora_linear_fwd(w, X, A, B, 1.0)
    one = qn.qlora_linear_bwd_act8(w, X8, dY, A, B, 1.0, U=U)
    dX, dAs, dBs = qn.qlora_linear_bwd_group_act8([w, w], X8, [dY, dY], [A, A], [B, B], 1.0, Us=[U, U])
    for i in range(2):
        assert torch.equal(dAs[i], one[1]) and torch.equal(dBs[i], one[2])
    # the sum of two equal terms, rounded once: one's terms are rounded once too
    assert bool(((dX.double() - 2 * one[0].double()).abs() <= 2 * one[0].double().abs() * 2.0 ** -7 + 1e-5).all())
    H = qn.swiglu_fwd(X, X, checkpoint=False)[0]
    assert torch.equal(H, qn.swiglu_fwd(X, X.clone(), checkpoint=False)[0])


def test_strided_and_broadcast_inputs_through_autograd(qn):
    w, X, dY, A, B = _layer(qn, 40, 96, 128, 8)
    wide = torch.zeros(40, 256, dtype=torch.bfloat16, device="cuda")
    wide[:, ::2] = X
    res = []
    for x, a, d in ((X.clone(), A, dY[:1].expand(40, 96)), (wide[:, ::2], A.t().contiguous().t(), dY[:1].expand(40, 96).contiguous())):
        x = x.detach().requires_grad_()
        a, b = a.detach().requires_grad_(), B.detach().clone().requires_grad_()
        qn.QLoRALinearFunction.apply(x, a, b, w, 0.5, None, 0.0, True).backward(d)
        res.append((x.grad, a.grad, b.grad))
    assert all(torch.equal(p, q) for p, q in zip(*res))
    gate = X[:1].expand(40, 128).detach().requires_grad_()
    up = X.clone().requires_grad_()
    qn.SwiGLUFunction.apply(gate, up).backward(torch.ones(1, 1, dtype=torch.bfloat16, device="cuda").expand(40, 128))
    g8, u8 = qn.act8_quantize(gate.detach().contiguous()), qn.act8_quantize(X)
    dg, du = qn.swiglu_bwd(g8, u8, torch.ones_like(X))
    assert torch.equal(gate.grad, dg) and torch.equal(up.grad, du)


def test_autograd_with_every_argument_given(qn):
    """act8 None or False in its place: the layer without a checkpoint."""
    w, X, dY, A, B = _layer(qn, 40, 96, 128, 8)
    res = []
    for more in ((), (None, 0.0, None), (None, 0.0, False)):
        x, a, b = (t.detach().clone().requires_grad_() for t in (X, A, B))
        qn.QLoRALinearFunction.apply(x, a, b, w, 0.5, *more).backward(dY)
        res.append((x.grad, a.grad, b.grad))
    for r in res[1:]:
        assert all(torch.equal(p, q) for p, q in zip(res[0], r))


def test_no_tokens_with_a_mask(qn):
    w, X, dY, A, B = _layer(qn, 40, 96, 128, 8)
    X8 = qn.act8_quantize(X[:0])
    keep = torch.empty(0, 16, dtype=torch.uint8, device="cuda")
    dX, dA, dB = qn.qlora_linear_bwd_act8(w, X8, dY[:0], A, B, U=torch.empty(0, 8, device="cuda"), keep=keep, p=0.5)
    assert dX.shape == (0, 128) and not bool(dA.any()) and not bool(dB.any())


def test_refused_arguments(qn):
    w, X, dY, A, B = _layer(qn, 40, 96, 128, 8)
    X8 = qn.act8_quantize(X)
    _, U = qn.qlora_linear_fwd(w, X, A, B, 1.0)
    keep = torch.zeros(40, 16, dtype=torch.uint8, device="cuda")
    for kw in (dict(keep=keep[:39], p=0.5), dict(keep=keep.bool(), p=0.5), dict(keep=keep.cpu(), p=0.5),
               dict(keep="mask", p=0.5), dict(keep=keep, p=1.0), dict(U=U.cpu())):
        with pytest.raises(qn.QLoraError):
            qn.qlora_linear_bwd_act8(w, X8, dY, A, B, **dict(dict(U=U), **kw))
    with pytest.raises(qn.QLoraError):
        qn.qlora_linear_bwd_act8(w, X8, dY.cpu(), A, B, U=U)
    with pytest.raises(qn.QLoraError):
        qn.qlora_linear_bwd_act8(w, X8, dY, A, None, U=U)
    group = lambda **kw: qn.qlora_linear_bwd_group_act8(
        **dict(dict(ws=[w, w], X8=X8, dYs=[dY, dY], As=[A, A], Bs=[B, B], Us=[U, U]), **kw))
    for kw in (dict(ws=[]), dict(dYs=[dY]), dict(As=[A]), dict(Bs=None), dict(Bs=[B]), dict(Us=None), dict(Us=[U]),
               dict(As=[A, A[:4]], Bs=[B, B[:, :4].contiguous()]), dict(As=[A, None]), dict(ws=[w] * 5, dYs=[dY] * 5, As=[A] * 5, Bs=[B] * 5, Us=[U] * 5),
               dict(dAs=[None, torch.empty(8, 128, device="cuda", dtype=torch.float64)]), dict(X8=None)):
        with pytest.raises(qn.QLoraError):
            group(**kw)
    q = qn.q4g_quantize(workloads.normal_weight(16, 64, 0.02, 5).cuda(), group=32)
    for bad in (qn.Q4GWeight(16, 64, 0, q.packed, q.scale, q.zero), qn.Q4GWeight(16, 64, 64, q.packed, q.scale, q.zero),
                qn.Q4GWeight(16, 64, 32, q.packed, q.scale.half(), q.zero), qn.Q4GWeight(16, 64, 32, q.packed, q.scale, q.zero.cpu()),
                qn.Q4GWeight(16, 96, 32, q.packed, q.scale, q.zero)):
        with pytest.raises(qn.QLoraError):
            qn.q4g_linear_fwd(bad, X[:, :64].contiguous())
        with pytest.raises(qn.QLoraError):
            qn.q4g_dequantize(bad)
