"""4-bit weights with group scales on the GPU against the oracle: codes,
scales, zero points and expanded values exactly, products within the
roundings they make."""

import numpy as np
import pytest
import torch

import workloads
from oracle import q4g as og

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def qn():
    import bit_nf4_quantized_16_amd as qn

    assert torch.cuda.is_available()
    return qn


def _f64(t):
    return t.detach().cpu().double().numpy()


def _weight(N, K, seed, f32):
    W = workloads.student_t_weight(N, K, 5, 0.02, seed)
    return W if f32 else W.to(torch.bfloat16)


def _quantized(qn, W, group, sym, sd):
    w = qn.q4g_quantize(W.cuda(), group=group, symmetric=sym, scale_dtype=sd)
    q, s, z = og.quantize(W.float().numpy(), group, sym, sd == torch.bfloat16)
    return w, q, s, z


@pytest.mark.parametrize("N,K", [(1, 8), (1, 64), (3, 40), (5, 136), (17, 1000), (130, 4096), (7, 11008), (300, 200)])
@pytest.mark.parametrize("group", [32, 64, 128])
@pytest.mark.parametrize("sym,f32,sd", [(False, False, torch.bfloat16), (True, True, torch.bfloat16),
                                        (False, True, torch.float32), (True, False, torch.float32)])
def test_quantize_and_expand(qn, N, K, group, sym, f32, sd):
    w, q, s, z = _quantized(qn, _weight(N, K, N + K, f32), group, sym, sd)
    assert np.array_equal(w.packed.cpu().numpy(), og.pack(q))
    assert np.array_equal(w.scale.float().cpu().numpy(), s)
    assert (w.zero is None) == sym
    if not sym:
        assert np.array_equal(w.zero.cpu().numpy(), z)
    want = og.dequantize(q, s, z, group)
    assert np.array_equal(qn.q4g_dequantize(w, torch.float32).cpu().numpy(), want)
    assert torch.equal(qn.q4g_dequantize(w).cpu(), torch.from_numpy(want).to(torch.bfloat16))


@pytest.mark.parametrize("sym", [False, True])
def test_quantize_special_groups(qn, sym):
    W = torch.zeros(12, 96)
    W[1] = 1.0
    W[2] = -2.5
    W[3, :32] = torch.linspace(-1, 0, 32)
    W[4, 5] = 3e37
    W[5, :64] = torch.arange(64) * 2.0 ** -140  # scales under the smallest normal number
    W[6] = torch.arange(96) % 16 - 8.0  # on the grid and at ties
    W[7] = (torch.arange(96) % 31 - 15.0) / 2
    W[8] = 2.0 ** -125 * (torch.arange(96) % 7 - 3)
    W[9, 40] = -1e-30
    W[10] = workloads.normal_weight(1, 96, 1e30, 3)[0]
    for f32 in (False, True):
        X = W if f32 else W.to(torch.bfloat16)
        for sd in (torch.bfloat16, torch.float32):
            w, q, s, z = _quantized(qn, X, 32, sym, sd)
            assert np.array_equal(w.packed.cpu().numpy(), og.pack(q))
            assert np.array_equal(w.scale.float().cpu().numpy(), s)
            assert sym or np.array_equal(w.zero.cpu().numpy(), z)


# ---- products -----------------------------------------------------------------
# y is rounded to bf16 once (2^-8 of it) and sums in fp32: K products and the
# group's terms, each step off by at most 2^-23 (MFMA partial sums included) of
# the magnitudes s (q + z) |x| that it goes through.
def _check(Y, X, q, s, z, group):
    y, mag = og.linear(_f64(X), q, s, z, group)
    err = np.abs(_f64(Y) - y)
    K = q.shape[1]
    assert np.all(err <= np.abs(y) * 2.0 ** -8 + mag * (K + 8) * 2.0 ** -23 + 2.0 ** -133)
    if np.linalg.norm(y) > 0:
        assert np.linalg.norm(err) <= 2.0 ** -8 * np.linalg.norm(y)


@pytest.mark.parametrize("T", [1, 2, 15, 16, 17, 32, 33, 48, 64, 65, 150])
@pytest.mark.parametrize("N,K,group,sym,sd", [
    (48, 256, 128, False, torch.bfloat16),   # whole tiles and chunks
    (33, 1000, 32, True, torch.bfloat16),    # odd rows, a short last group
    (7, 136, 64, False, torch.float32),      # fewer rows than a tile, one value past a chunk
    (100, 2064, 128, True, torch.float32),   # more chunks than waves
    (16, 1096, 32, False, torch.float32),
    (70, 4160, 64, True, torch.bfloat16),
])
def test_linear(qn, T, N, K, group, sym, sd):
    w, q, s, z = _quantized(qn, _weight(N, K, N + K, False), group, sym, sd)
    X = workloads.bf16_normal((T, K), 1.0, T)
    _check(qn.q4g_linear_fwd(w, X.cuda()), X, q, s, z, group)


@pytest.mark.parametrize("N,K", [(1, 8), (1, 32), (2, 40), (17, 120), (1, 22016), (515, 8), (3, 128)])
@pytest.mark.parametrize("T", [1, 5, 40])
@pytest.mark.parametrize("group", [32, 64, 128])
def test_linear_small(qn, N, K, T, group):
    w, q, s, z = _quantized(qn, _weight(N, K, N + K, True), group, False, torch.bfloat16)
    X = workloads.bf16_normal((T, K), 1.0, T)
    _check(qn.q4g_linear_fwd(w, X.cuda()), X, q, s, z, group)


@pytest.mark.parametrize("T,N,K,group", [(1, 4096, 4096, 128), (1, 11008, 4096, 32), (16, 4096, 11008, 64),
                                         (37, 11008, 4096, 128), (64, 4096, 4096, 32), (200, 4096, 4096, 128)])
def test_linear_model_shapes(qn, T, N, K, group):
    w, q, s, z = _quantized(qn, _weight(N, K, 5, False), group, False, torch.bfloat16)
    X = workloads.bf16_normal((T, K), 1.0, 6)
    _check(qn.q4g_linear_fwd(w, X.cuda()), X, q, s, z, group)


@pytest.mark.parametrize("group", [32, 64, 128])
def test_each_code_at_each_place(qn, group):
    """One-hot tokens read single weights: every place of a row's chunk, with
    a short last group, exactly."""
    N, K = 20, 392
    w, q, s, z = _quantized(qn, _weight(N, K, 11, True), group, False, torch.bfloat16)
    want = torch.from_numpy(og.dequantize(q, s, z, group).T.copy()).to(torch.bfloat16)
    for t0 in range(0, K, 56):
        X = torch.zeros(56, K, dtype=torch.bfloat16)
        X[torch.arange(56), t0 + torch.arange(56)] = 1.0
        assert torch.equal(qn.q4g_linear_fwd(w, X.cuda()).cpu(), want[t0:t0 + 56])
        assert torch.equal(qn.q4g_linear_fwd(w, X[:9].cuda()).cpu(), want[t0:t0 + 9])


def test_non_finite_tokens(qn):
    """An infinite x gives the infinities and NaN of the sum of x w', its own
    token only; huge values that overflow as separate sums do not."""
    N, K = 40, 520
    w, q, s, z = _quantized(qn, _weight(N, K, 12, False), 64, False, torch.bfloat16)
    wd = og.dequantize(q, s, z, 64).astype(np.float64)
    X = workloads.bf16_normal((20, K), 1.0, 3)
    clean = qn.q4g_linear_fwd(w, X.cuda()).cpu()
    X[3, 100], X[4, 7], X[5, 519] = float("inf"), float("-inf"), float("nan")
    X[6, 8], X[6, 9] = float("inf"), float("-inf")
    X[7] = 0.0
    X[7, 70] = 3.3e38
    Y = qn.q4g_linear_fwd(w, X.cuda()).cpu()
    other = [i for i in range(20) if i not in (3, 4, 5, 6, 7)]
    assert torch.equal(Y[other], clean[other])
    for t, k in ((3, 100), (4, 7)):
        want = float(X[t, k]) * wd[:, k]  # NaN where the weight is zero
        assert np.array_equal(_f64(Y[t]), want, equal_nan=True)
    assert torch.isnan(Y[5]).all()
    with np.errstate(invalid="ignore"):
        want = np.inf * wd[:, 8] - np.inf * wd[:, 9]
    assert np.array_equal(_f64(Y[6]), want, equal_nan=True)
    want = float(X[7, 70]) * wd[:, 70]
    assert np.all(np.abs(_f64(Y[7]) - want) <= np.abs(want) * 2.0 ** -8)


@pytest.mark.parametrize("T", [2, 7])
def test_non_finite_tokens_decode(qn, T):
    """The same with few tokens (and one of them infinite throughout)."""
    N, K = 40, 520
    w, q, s, z = _quantized(qn, _weight(N, K, 12, False), 32, True, torch.float32)
    wd = og.dequantize(q, s, z, 32).astype(np.float64)
    X = workloads.bf16_normal((T, K), 1.0, 3)
    clean = qn.q4g_linear_fwd(w, X.cuda()).cpu()
    X[1] = 0.0
    X[1, 300] = float("inf")
    Y = qn.q4g_linear_fwd(w, X.cuda()).cpu()
    with np.errstate(invalid="ignore"):
        assert np.array_equal(_f64(Y[1]), np.inf * wd[:, 300], equal_nan=True)
    rest = [t for t in range(T) if t != 1]
    assert torch.equal(Y[rest], clean[rest])


@pytest.mark.parametrize("T,N,K,group,sd", [
    (1, 16500, 520, 64, torch.bfloat16),     # rows for two row tiles a workgroup, the last one ragged
    (7, 16500, 392, 32, torch.float32),
    (13, 16500, 264, 128, torch.bfloat16),
    (29, 8210, 520, 32, torch.float32),
    (45, 8210, 264, 64, torch.bfloat16),
    (70, 8210, 392, 128, torch.float32),
    (3, 40, 34000, 32, torch.bfloat16),      # more groups than a workgroup holds at a time
    (3, 40, 34000, 32, torch.float32),
    (12, 40, 34000, 64, torch.float32),
    (50, 40, 34000, 32, torch.float32),
    (40, 8210, 9000, 32, torch.float32),
    (2, 16500, 9000, 32, torch.float32),
])
@pytest.mark.parametrize("sym", [False, True])
def test_linear_variants(qn, T, N, K, group, sd, sym):
    """Each variant of the kernels against the expanded weight (tested above
    to be exact) in fp64."""
    W = (torch.randn(N, K, device="cuda", generator=torch.Generator("cuda").manual_seed(N + K)) * 0.02)
    w = qn.q4g_quantize(W, group=group, symmetric=sym, scale_dtype=sd)
    X = workloads.bf16_normal((T, K), 1.0, T).cuda()
    wd = qn.q4g_dequantize(w, torch.float32)
    y = X.double() @ wd.double().t().contiguous()
    z = (w.zero.double() if w.zero is not None else torch.full(w.scale.shape, 8.0, device="cuda", dtype=torch.float64))
    at = torch.arange(K, device="cuda") // group
    # s (q + z) |x| = (s (q - z) + 2 s z) |x|
    mag = X.double().abs() @ (wd.double() + 2 * (w.scale.double() * z)[:, at]).t().contiguous()
    err = (qn.q4g_linear_fwd(w, X).double() - y).abs()
    assert bool((err <= y.abs() * 2.0 ** -8 + mag * (K + 8) * 2.0 ** -23).all())
    assert float(err.norm()) <= 2.0 ** -8 * float(y.norm())


@pytest.mark.parametrize("T,N,K,group,sd", [
    (33, 4128, 1032, 64, torch.bfloat16),    # 259 workgroups of a row tile: two row tiles, 8 waves
    (100, 4090, 776, 128, torch.float32),    # 512
    (130, 4090, 776, 32, torch.bfloat16),    # 768: two row tiles, 4 waves
    (20, 16500, 264, 32, torch.float32),     # 1032 with short groups: 8 waves again
    (64, 16500, 1288, 32, torch.bfloat16),
])
@pytest.mark.parametrize("sym", [False, True])
def test_linear_workgroup_rule(qn, T, N, K, group, sd, sym):
    test_linear_variants(qn, T, N, K, group, sd, sym)


@pytest.mark.parametrize("T,N,K,group,sd", [
    (60, 10250, 1288, 32, torch.bfloat16),   # 641 row tiles: three a workgroup, 8 waves, the last tile alone
    (25, 11000, 520, 64, torch.float32),
    (37, 9000, 4104, 32, torch.float32),     # constants in slices
    (64, 8210, 9000, 32, torch.float32),
    (64, 8210, 17000, 32, torch.bfloat16),
    (16, 10250, 648, 128, torch.bfloat16),
    (9, 22000, 392, 128, torch.float32),     # 1375: three a workgroup, 4 waves
    (30, 22000, 264, 32, torch.bfloat16),
    (45, 22000, 392, 64, torch.float32),
    (64, 22000, 264, 32, torch.float32),     # 8 waves
    (64, 22000, 392, 128, torch.bfloat16),
    (33, 32000, 264, 32, torch.float32),     # 2000: two a workgroup
    (200, 4090, 520, 32, torch.bfloat16),
    (100, 6140, 520, 64, torch.bfloat16),    # three, over two token tiles
])
@pytest.mark.parametrize("sym", [False, True])
def test_linear_balance_rule(qn, T, N, K, group, sd, sym):
    test_linear_variants(qn, T, N, K, group, sd, sym)


def test_padding_and_memory_behind_the_arrays(qn):
    """Codes past K, rows behind the last token and behind the output do not
    matter and stay as they were."""
    N, K, T = 19, 72, 5
    w, q, s, z = _quantized(qn, _weight(N, K, 13, False), 64, False, torch.bfloat16)
    X = torch.full((16, K), float("nan"), dtype=torch.bfloat16, device="cuda")
    X[:T] = workloads.bf16_normal((T, K), 1.0, 4).cuda()
    out = torch.full((16, N), 7.0, dtype=torch.bfloat16, device="cuda")
    want = qn.q4g_linear_fwd(w, X[:T].clone())
    w.packed[:, K // 2:] = 0xFF
    got = qn.q4g_linear_fwd(w, X[:T], out=out[:T])
    assert torch.equal(got, want) and bool((out[T:] == 7).all())
    assert torch.equal(qn.q4g_dequantize(w, torch.float32).cpu(), torch.from_numpy(og.dequantize(q, s, z, 64)))


def test_no_tokens_and_repeatable(qn):
    w, *_ = _quantized(qn, _weight(33, 264, 14, False), 32, True, torch.bfloat16)
    assert qn.q4g_linear_fwd(w, torch.empty(0, 264, dtype=torch.bfloat16, device="cuda")).shape == (0, 33)
    X = workloads.bf16_normal((40, 264), 1.0, 5).cuda()
    one = qn.q4g_linear_fwd(w, X)
    for _ in range(3):
        assert torch.equal(qn.q4g_linear_fwd(w, X), one)


def test_infinite_scale(qn):
    """A weight brought from elsewhere may hold infinite scales: their rows
    become infinite or NaN, the others stay."""
    w, q, s, z = _quantized(qn, _weight(33, 264, 15, False), 32, False, torch.bfloat16)
    X = workloads.bf16_normal((3, 264), 1.0, 5).cuda()
    want = qn.q4g_linear_fwd(w, X)
    w.scale[4, 8] = float("inf")
    got = qn.q4g_linear_fwd(w, X)
    assert not torch.isfinite(got[:, 4]).any()
    rest = [i for i in range(33) if i != 4]
    assert torch.equal(got[:, rest], want[:, rest])


def test_captured_calls_replay(qn):
    N, K = 130, 520
    W = _weight(N, K, 16, False).cuda()
    X = workloads.bf16_normal((5, K), 1.0, 6).cuda()

    def step():
        w = qn.q4g_quantize(W, group=64)
        return qn.q4g_linear_fwd(w, X), qn.q4g_dequantize(w)

    step()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = step()
    for i in range(3):
        W.copy_(_weight(N, K, 20 + i, False).cuda())
        X.copy_(workloads.bf16_normal((5, K), 1.0, 30 + i).cuda())
        graph.replay()
        torch.cuda.synchronize()
        for a, b in zip(out, step()):
            assert torch.equal(a, b)


def test_two_streams(qn):
    ws = [_quantized(qn, _weight(1030, 2064, s, False), 128, False, torch.bfloat16)[0] for s in (1, 2)]
    X = workloads.bf16_normal((9, 2064), 1.0, 7).cuda()
    want = [qn.q4g_linear_fwd(w, X) for w in ws]
    torch.cuda.synchronize()
    got = []
    for w in ws:
        st = torch.cuda.Stream()
        st.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(st):
            got.append(qn.q4g_linear_fwd(w, X))
    torch.cuda.synchronize()
    for a, b in zip(got, want):
        assert torch.equal(a, b)


def test_merge_then_serve(qn):
    """Trained weight to 4 bits for serving: merge the adapter, quantize the
    merged weight, decode; the product is that of the expanded weight."""
    N, K, r = 136, 320, 8
    w4 = qn.quantize_weight(workloads.normal_weight(N, K, 0.02, 1).cuda())
    A, B = workloads.bf16_normal((r, K), 0.05, 2).cuda(), workloads.bf16_normal((N, r), 0.05, 3).cuda()
    merged = qn.qlora_merge(w4, A, B, 2.0)
    for group in (32, 128):
        w = qn.q4g_quantize(merged, group=group)
        q, s, z = og.quantize(merged.float().cpu().numpy(), group, False)
        X = workloads.bf16_normal((3, K), 1.0, 4)
        _check(qn.q4g_linear_fwd(w, X.cuda()), X, q, s, z, group)
        # nearest of sixteen values: half a step, and the scale's own rounding at the ends
        err = (qn.q4g_dequantize(w, torch.float32) - merged.float()).abs()
        step = w.scale.float().repeat_interleave(group, dim=1)[:, :K]
        assert bool((err <= step * (0.5 + 15 * 2.0 ** -8)).all())


def test_refusals(qn):
    W = torch.zeros(4, 64, dtype=torch.bfloat16, device="cuda")
    w = qn.q4g_quantize(W, group=32)
    X = torch.zeros(3, 64, dtype=torch.bfloat16, device="cuda")
    bad = [lambda: qn.q4g_quantize(W.half()), lambda: qn.q4g_quantize(W.cpu()), lambda: qn.q4g_quantize(W.t()),
           lambda: qn.q4g_quantize(W, group=48), lambda: qn.q4g_quantize(W, scale_dtype=torch.float16),
           lambda: qn.q4g_quantize(W[:, :20].contiguous()), lambda: qn.q4g_quantize(W[:0]),
           lambda: qn.q4g_dequantize(w, torch.float16), lambda: qn.q4g_dequantize(w, out=X),
           lambda: qn.q4g_linear_fwd(w, X.float()), lambda: qn.q4g_linear_fwd(w, X[:, :32].contiguous()),
           lambda: qn.q4g_linear_fwd(w, X.cpu()), lambda: qn.q4g_linear_fwd(w, X, out=X),
           lambda: qn.q4g_linear_fwd(qn.Q4GWeight(4, 64, 32, w.packed[:3], w.scale, w.zero), X),
           lambda: qn.q4g_linear_fwd(qn.Q4GWeight(4, 64, 64, w.packed, w.scale, w.zero), X),
           lambda: qn.q4g_linear_fwd(qn.Q4GWeight(4, 64, 32, w.packed, w.scale.half(), w.zero), X),
           lambda: qn.q4g_linear_fwd(qn.Q4GWeight(4, 64, 32, w.packed, w.scale, w.zero[:3]), X)]
    for call in bad:
        with pytest.raises(qn.QLoraError):
            call()
