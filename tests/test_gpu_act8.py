"""8-bit activation checkpoints and the gated activation on the GPU against
the oracle: codes and scales exactly, the activation within the roundings it
makes."""

import numpy as np
import pytest
import torch

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


def _check(qn, X):
    a = qn.act8_quantize(X.cuda())
    got16, got32 = qn.act8_dequantize(a), qn.act8_dequantize(a, torch.float32)
    torch.cuda.synchronize()
    want = oa.act8_restore(_f64(X))
    assert np.array_equal(a.scale.cpu().numpy().astype(np.int64) - 127, oa.act8_exponents(_f64(X)))
    codes = a.codes.cpu().view(torch.float8_e4m3fn).double().numpy().reshape(X.shape[0], -1, 32)
    stored = np.ldexp(codes, oa.act8_exponents(_f64(X))[:, :, None]).reshape(X.shape)
    stored = np.where(np.abs(stored) == 2.0 ** 128, np.copysign(np.inf, stored), stored)  # rounded up past fp32
    for got in (stored, _f64(got16), _f64(got32)):
        assert np.array_equal(got, want, equal_nan=True)
        assert np.array_equal(np.signbit(got)[np.isfinite(want)], np.signbit(_f64(X))[np.isfinite(want)])


@pytest.mark.parametrize("T,K", [(1, 32), (1, 4096), (3, 96), (17, 160), (77, 11008), (300, 4128), (1024, 64)])
def test_store_and_restore(qn, T, K):
    _check(qn, workloads.bf16_normal((T, K), 1.0, T + K))


def test_every_bf16_value(qn):
    """All 65536 bit patterns, each alone in a block with small values, and
    again in blocks of like magnitude."""
    bits = torch.arange(65536, dtype=torch.int32).to(torch.int16).view(torch.bfloat16)
    alone = torch.full((65536, 32), 2.0 ** -100, dtype=torch.bfloat16)
    alone[:, 7] = bits
    _check(qn, alone)
    _check(qn, bits.view(-1, 32).contiguous())


def test_block_maxima_around_the_scale_steps(qn):
    """Maxima at, below and above 1.75 2^e, over the whole exponent range."""
    rows = []
    for e in list(range(-133, -110)) + list(range(-20, 20)) + list(range(100, 128)):
        for m in (1.0, 1.7421875, 1.75, 1.7578125, 1.9921875):
            r = workloads.bf16_normal((32,), 1.0, e + 200).float().clamp(-0.9, 0.9).double() * 2.0 ** e
            r[11] = -m * 2.0 ** e
            rows.append(r.to(torch.bfloat16))
    _check(qn, torch.stack(rows))


def test_zero_and_non_finite_blocks(qn):
    X = workloads.bf16_normal((8, 96), 3.0, 5)
    X[0] = 0.0
    X[1, 32:64] = -0.0
    X[2, 5], X[2, 40] = float("inf"), float("nan")
    X[3, :32] = float("nan")
    X[4, 32:64] = float("-inf")
    X[5, 64] = 3.3895e38  # the largest finite value
    _check(qn, X)


def test_rows_behind_the_activation_stay(qn):
    X = workloads.bf16_normal((5, 64), 1.0, 9).cuda()
    codes = torch.full((8, 64), 0x5A, dtype=torch.uint8, device="cuda")
    scale = torch.full((8, 2), 0x5A, dtype=torch.uint8, device="cuda")
    qn.act8_quantize(X, out=qn.Act8(5, 64, codes[:5], scale[:5]))
    torch.cuda.synchronize()
    assert bool((codes[5:] == 0x5A).all()) and bool((scale[5:] == 0x5A).all())
    assert bool((codes[:5] != 0x5A).any())


def test_no_rows(qn):
    X = torch.empty(0, 64, dtype=torch.bfloat16, device="cuda")
    a = qn.act8_quantize(X)
    assert qn.act8_dequantize(a).shape == (0, 64)
    H, g8, u8, h8 = qn.swiglu_fwd(X, X, h8=True)
    dg, du = qn.swiglu_bwd(g8, u8, X)
    assert H.shape == dg.shape == du.shape == (0, 64) and h8.rows == 0


# ---- gated activation -------------------------------------------------------
# H: one bf16 rounding (2^-8 relative) and the fp32 arithmetic: the exponent
# -g log2(e) carries 2 roundings of relative 2^-24, worth 2 |g| 2^-24 in e^-g;
# v_exp_f32, the sum, v_rcp_f32 and the two products add at most 12 2^-24.
# Below g = -88 the sigmoid underflows to 0 where h is under 1e-36 |u|.
def _h_bound(g, u, h):
    return np.abs(h) * (2.0 ** -8 + (2 * np.abs(g) + 12) * 2.0 ** -24) + 1e-36 * (np.abs(u) + 1)


def _bwd_bounds(g, u, d, dg, du):
    """As above; dg's factor 1 + g (1 - p) may cancel, so its error counts
    against 1 + |g|, with the relative error of p and four more roundings."""
    p = 1.0 / (1.0 + np.exp(-np.clip(g, -700, 700)))
    fp = (2 * np.abs(g) + 16) * 2.0 ** -24
    tiny = 1e-36 * (np.abs(d) + 1) * (np.abs(u) + np.abs(g) + 1)
    return (np.abs(dg) * 2.0 ** -8 + 2 * np.abs(d * u * p) * (1 + np.abs(g)) * fp + tiny,
            np.abs(du) * (2.0 ** -8 + fp) + tiny)


def _swiglu_check(qn, g, u, d):
    H, g8, u8, h8 = qn.swiglu_fwd(g.cuda(), u.cuda(), h8=True)
    dg, du = qn.swiglu_bwd(g8, u8, d.cuda())
    torch.cuda.synchronize()
    gn, un, dn = _f64(g), _f64(u), _f64(d)
    h = oa.swiglu(gn, un)
    assert np.all(np.abs(_f64(H) - h) <= _h_bound(gn, un, h))
    # the checkpoints are those of the three tensors
    gr, ur = oa.act8_restore(gn), oa.act8_restore(un)
    assert np.array_equal(_f64(qn.act8_dequantize(g8)), gr)
    assert np.array_equal(_f64(qn.act8_dequantize(u8)), ur)
    assert np.array_equal(_f64(qn.act8_dequantize(h8)), oa.act8_restore(_f64(H)))
    wg, wu = oa.swiglu_backward(gr, ur, dn)
    bg, bu = _bwd_bounds(gr, ur, dn, wg, wu)
    assert np.all(np.abs(_f64(dg) - wg) <= bg)
    assert np.all(np.abs(_f64(du) - wu) <= bu)


@pytest.mark.parametrize("T,F,std", [(1, 32, 1.0), (1, 11008, 2.0), (3, 96, 20.0), (77, 4128, 2.0), (513, 64, 0.01)])
def test_swiglu(qn, T, F, std):
    _swiglu_check(qn, workloads.bf16_normal((T, F), std, T + F), workloads.bf16_normal((T, F), 1.0, T + F + 1),
                  workloads.bf16_normal((T, F), 1.0, T + F + 2))


def test_swiglu_over_the_gate_range(qn):
    g = torch.linspace(-120, 120, 64 * 320).view(-1, 320).to(torch.bfloat16)
    _swiglu_check(qn, g, workloads.bf16_normal(tuple(g.shape), 1.0, 3), workloads.bf16_normal(tuple(g.shape), 1.0, 4))


def test_swiglu_without_checkpoints(qn):
    g, u = (workloads.bf16_normal((9, 64), 1.0, s).cuda() for s in (1, 2))
    H, a, b, c = qn.swiglu_fwd(g, u, checkpoint=False)
    assert a is None and b is None and c is None
    assert torch.equal(H, qn.swiglu_fwd(g, u, h8=True)[0])


def test_swiglu_non_finite_values_stay_in_place(qn):
    g, u = workloads.bf16_normal((4, 64), 1.0, 1), workloads.bf16_normal((4, 64), 1.0, 2)
    clean = qn.swiglu_fwd(g.cuda(), u.cuda())
    dclean = qn.swiglu_bwd(clean[1], clean[2], u.cuda())
    g[1, 3], g[2, 40], u[3, 63] = float("nan"), float("inf"), float("inf")
    H, g8, u8, _ = qn.swiglu_fwd(g.cuda(), u.cuda())
    bad = torch.zeros(4, 64, dtype=torch.bool)
    bad[1, 3] = bad[2, 40] = bad[3, 63] = True
    assert not torch.isfinite(H.cpu()[bad]).any()
    assert torch.equal(H.cpu()[~bad], clean[0].cpu()[~bad])
    for got, want in zip(qn.swiglu_bwd(g8, u8, workloads.bf16_normal((4, 64), 1.0, 2).cuda()), dclean):
        same = (got.cpu() == want.cpu()) | bad
        # a block that lost its largest value may have a finer scale
        blocks = torch.zeros(4, 2, dtype=torch.bool)
        blocks[1, 0] = blocks[2, 1] = blocks[3, 1] = True
        assert bool((same | blocks.repeat_interleave(32, dim=1)).all())
        assert torch.isfinite(got.cpu()[~bad]).all()


def test_swiglu_autograd(qn):
    g, u, d = (workloads.bf16_normal((33, 96), 1.5, s).cuda() for s in (1, 2, 3))
    gl, ul = g.clone().requires_grad_(), u.clone().requires_grad_()
    H = qn.SwiGLUFunction.apply(gl, ul)
    dg, du = torch.autograd.grad(H, (gl, ul), d)
    ref = qn.swiglu_fwd(g, u)
    want = qn.swiglu_bwd(ref[1], ref[2], d)
    assert torch.equal(H, ref[0]) and torch.equal(dg, want[0]) and torch.equal(du, want[1])


def test_captured_calls_replay(qn):
    """Store, restore and both passes of the activation captured once and
    replayed with new inputs equal the eager calls, with eager work between."""
    g, u, d = (workloads.bf16_normal((40, 96), 1.0, s).cuda() for s in (1, 2, 3))

    def step():
        H, g8, u8, h8 = qn.swiglu_fwd(g, u, h8=True)
        return (H, qn.act8_dequantize(h8), *qn.swiglu_bwd(g8, u8, d))

    step()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = step()
    for i in range(3):
        for t, s in ((g, 10), (u, 20), (d, 30)):
            t.copy_(workloads.bf16_normal((40, 96), 1.0, s + i).cuda())
        graph.replay()
        torch.cuda.synchronize()
        for a, b in zip(out, step()):
            assert torch.equal(a, b)


def test_calls_on_two_streams(qn):
    X = [workloads.bf16_normal((257, 4096), 1.0, s).cuda() for s in (1, 2)]
    want = [qn.act8_quantize(x) for x in X]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in X]
    got = []
    for x, st in zip(X, streams):
        st.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(st):
            got.append(qn.act8_quantize(x))
    torch.cuda.synchronize()
    for a, b in zip(got, want):
        assert torch.equal(a.codes, b.codes) and torch.equal(a.scale, b.scale)


def test_refusals(qn):
    X = torch.zeros(4, 64, dtype=torch.bfloat16, device="cuda")
    a = qn.act8_quantize(X)
    for call in (lambda: qn.act8_quantize(X.float()), lambda: qn.act8_quantize(X.cpu()),
                 lambda: qn.act8_quantize(X.t()), lambda: qn.act8_quantize(X[:, :40].contiguous()),
                 lambda: qn.act8_quantize(X[0]), lambda: qn.act8_quantize(X[:3], out=a),
                 lambda: qn.act8_dequantize(a, torch.float16),
                 lambda: qn.act8_dequantize(qn.Act8(4, 64, a.codes, a.scale[:3])),
                 lambda: qn.act8_dequantize(a, out=X[:3]),
                 lambda: qn.swiglu_fwd(X, X[:3]), lambda: qn.swiglu_fwd(X, X.float()),
                 lambda: qn.swiglu_bwd(a, qn.act8_quantize(X[:3]), X), lambda: qn.swiglu_bwd(a, a, X[:3])):
        with pytest.raises(qn.QLoraError):
            call()
