"""A training step through the operators together, as they are used: norm,
grouped gate and up from a checkpoint, gated activation, down projection with
bias onto the residual stream, a projection with activation, norm, a frozen
head, and a loss on the logits; gradients against autograd of the 64-bit
formulas on the same dequantized weights, then an optimizer step."""

import pytest
import torch

import workloads

pytestmark = pytest.mark.gpu

BF16 = torch.bfloat16
C, F, V, R = 128, 192, 401, 8


@pytest.fixture(scope="module")
def qn():
    import bit_nf4_quantized_16_amd as qn

    assert torch.cuda.is_available()
    return qn


def _model(qn, seed):
    t = lambda shape, s, i: workloads.bf16_normal(shape, s, seed + i).cuda()
    ws = {n: qn.quantize_weight(workloads.normal_weight(*s, 0.06, seed + 40 + i).cuda())
          for i, (n, s) in enumerate((("gate", (F, C)), ("up", (F, C)), ("down", (C, F)), ("proj", (C, C))))}
    p = {}
    for i, (n, w) in enumerate(ws.items()):
        p["A_" + n], p["B_" + n] = t((R, w.cols), 0.1, 2 * i), t((w.rows, R), 0.1, 2 * i + 1)
    p["n1"], p["n2"], p["b2"] = (1 + t((C,), 0.1, 20)).to(BF16), (1 + t((C,), 0.1, 21)).to(BF16), t((C,), 0.1, 22)
    p["b_down"], p["b_proj"] = t((C,), 0.2, 23), t((C,), 0.2, 24)
    return ws, p, t((V, C), 0.3, 30)


def _ours(qn, ws, p, X, scale):
    h = qn.NormFunction.apply(X, p["n1"], None, 1e-5, True)
    g, u = qn.QLoRAGroupAct8Function.apply(h, None, scale, [ws["gate"], ws["up"]], p["A_gate"], p["B_gate"], p["A_up"],
                                           p["B_up"])
    m = qn.SwiGLUFunction.apply(g, u)
    x = qn.QLoRALinearEpilogueFunction.apply(m, p["A_down"], p["B_down"], ws["down"], scale, p["b_down"], "none", X)
    y = qn.QLoRALinearEpilogueFunction.apply(x, p["A_proj"], p["B_proj"], ws["proj"], scale, p["b_proj"], "gelu", x)
    return qn.NormFunction.apply(y, p["n2"], p["b2"], 1e-5, False)


def _exact(qn, ws, p, X, scale):
    W = {n: qn.nf4_dequantize(w).double() for n, w in ws.items()}
    lin = lambda x, n: x @ W[n].t() + scale * (x @ p["A_" + n].t()) @ p["B_" + n].t()
    h = X / torch.sqrt((X * X).mean(1, keepdim=True) + 1e-5) * p["n1"]
    g = lin(h, "gate")
    x = X + lin(g * torch.sigmoid(g) * lin(h, "up"), "down") + p["b_down"]
    z = lin(x, "proj") + p["b_proj"]
    y = x + z * torch.special.ndtr(z)
    c = y - y.mean(1, keepdim=True)
    return c / torch.sqrt((c * c).mean(1, keepdim=True) + 1e-5) * p["n2"] + p["b2"]


def _losses(T, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    labels = torch.randint(0, V, (T,), generator=g, device="cuda")
    labels[::7] = -100
    cut = T // 2
    start = torch.tensor([0, cut // 2, cut, cut + 3, T], device="cuda")
    ref = -6.0 * (start[1:] - start[:-1]).float()
    index = torch.randint(0, V, (T, 5), generator=g, device="cuda")
    return labels, start, ref, index, torch.randn(T, 5, generator=g, device="cuda")


def _loss64(kind, z, labels, start, ref, index, top):
    on = labels >= 0
    ls = torch.log_softmax(z, 1)
    lp = torch.where(on, ls.gather(1, labels.clamp(min=0)[:, None])[:, 0], 0.0)
    if kind == "preference":
        L = torch.stack([lp[a:b].sum() for a, b in zip(start[:-1].tolist(), start[1:].tolist())]) - ref.double()
        return -torch.nn.functional.logsigmoid(0.1 * (L[0::2] - L[1::2])).mean()
    p = torch.log_softmax(top.double() / 2, 1)
    kl = (p.exp() * (p - torch.log_softmax(z / 2, 1).gather(1, index))).sum(1)
    return torch.where(on, 0.75 * 4 * kl - 0.25 * lp, 0.0).mean()


@pytest.mark.parametrize("T", [12, 60, 300])
@pytest.mark.parametrize("kind", ["preference", "distill"])
def test_step(qn, T, kind):
    ws, p, head = _model(qn, seed=T)
    X = workloads.bf16_normal((T, C), 1.0, 99).cuda()
    labels, start, ref, index, top = _losses(T, T)
    leaves = {n: t.clone().requires_grad_() for n, t in p.items()}
    x = X.clone().requires_grad_()
    z = _ours(qn, ws, leaves, x, 2.0) @ head.t()
    if kind == "preference":
        loss = qn.PreferenceLossFunction.apply(z, labels, start, ref, 0.1)[0].mean()
    else:
        loss = qn.DistillLossFunction.apply(z, index, top, labels, 2.0, 0.25).mean()
    loss.backward()

    l64 = {n: t.double().requires_grad_() for n, t in p.items()}
    x64 = X.double().requires_grad_()
    want = _loss64(kind, _exact(qn, ws, l64, x64, 2.0) @ head.double().t(), labels, start, ref, index, top)
    want.backward()
    # the activations between the operators are bf16, gate and up E4M3: their roundings (2^-4 and
    # 2^-9 a value) average out in the gradients' sums; a twentieth of the largest value holds a
    # wrong term or a missing factor apart from them
    assert abs(float(loss.detach()) - float(want)) <= 2e-2 * abs(float(want))
    for n, t in [("X", x)] + list(leaves.items()):
        e = (x64 if n == "X" else l64[n]).grad
        assert t.grad is not None and t.grad.dtype == BF16
        assert float((t.grad.double() - e).norm()) <= 5e-2 * float(e.norm()), (n, float((t.grad.double() - e).norm() / e.norm()))

    # the adapters' optimizer step
    flat = torch.cat([leaves[n].detach().float().flatten() for n in p if n[:2] in ("A_", "B_")])
    grad = torch.cat([leaves[n].grad.float().flatten() for n in p if n[:2] in ("A_", "B_")])
    m, v, before = torch.zeros_like(flat), torch.zeros_like(flat), flat.clone()
    qn.paged_adamw_step(flat, grad, m, v, 1, lr=1e-3)
    moved = grad.abs() > 1e-6
    assert torch.allclose((before - flat)[moved], 1e-3 * grad[moved].sign(), rtol=2e-2)


def test_the_step_in_a_graph(qn):
    """Forward, loss and backward by the plain calls, captured, replayed with
    new inputs."""
    T = 40
    ws, p, head = _model(qn, seed=5)
    X = workloads.bf16_normal((T, C), 1.0, 98).cuda()
    labels, start, ref, index, top = _losses(T, 5)
    dloss = torch.full((2,), 0.5, device="cuda")

    def step():
        h, _, r1 = qn.norm_fwd(X, p["n1"], None, 1e-5, True)
        Y, U, Z = qn.qlora_linear_fwd_epilogue(ws["proj"], h, p["A_proj"], p["B_proj"], 2.0, p["b_proj"], "gelu", X,
                                               save_z=True)
        n, mean, r2 = qn.norm_fwd(Y, p["n2"], p["b2"])
        z = n @ head.t()
        loss, _, st = qn.preference_loss_fwd(z, labels, start, ref)
        dz = qn.preference_loss_bwd(z, labels, st, dloss, dlogits=z)
        dY, dn2, db2 = qn.norm_bwd(Y, p["n2"], dz @ head, mean, r2)
        dZ, db = qn.epilogue_bwd(dY, Z, "gelu")
        dh, dA, dB = qn.qlora_linear_bwd(ws["proj"], h, dZ, p["A_proj"], p["B_proj"], 2.0, U=U)
        dX, dn1, _ = qn.norm_bwd(X, p["n1"], dh, None, r1, need_db=False)
        return loss, dX, dn1, dA, dB, db, dn2, db2

    step()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = step()
    for seed in (1, 2, 3):
        X.copy_(workloads.bf16_normal((T, C), 1.0, seed))
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(out, step()))
