"""The linear layer's epilogue at the ends of its range: infinite adapter terms,
and the activations' values to more bits than the result has."""

import math

import pytest
import torch

from test_gpu_epilogue import ACTS, BF16, _act

pytestmark = pytest.mark.gpu
INF = float("inf")


@pytest.fixture(scope="module")
def qn():
    import bit_nf4_quantized_16_amd as qn

    assert torch.cuda.is_available()
    return qn


def _positive(qn, T, N, K, r, seed):
    """A weight and adapters without zeros, of one sign: a token with an
    infinite activation has infinite outputs, not 0 times infinity."""
    g = torch.Generator(device="cuda").manual_seed(seed)
    u = lambda *s: 0.02 * (0.5 + torch.rand(*s, generator=g, device="cuda"))
    w = qn.quantize_weight(u(N, K))
    assert bool((qn.nf4_dequantize(w) > 0).all())
    return w, torch.randn(T, K, generator=g, device="cuda").to(BF16), u(r, K).to(BF16), u(N, r).to(BF16)


@pytest.mark.parametrize("r", [8, 16, 5, 33, 64, 128])
@pytest.mark.parametrize("T", [5, 20, 300])
def test_an_infinite_activation(qn, T, r):
    """Every path gives the plain forward's infinities: decode, U beside the
    launch, both terms in one rank step or in several."""
    w, X, A, B = _positive(qn, T, 264, 512, r, seed=r)
    X[2, 17], X[T - 1, 300] = INF, -INF
    Y0, U0 = qn.qlora_linear_fwd(w, X, A, B, 0.7)
    assert bool((Y0[2] == INF).all()) and bool((Y0[T - 1] == -INF).all()) and bool((U0[2] == INF).all())
    Y, U, Z = qn.qlora_linear_fwd_epilogue(w, X, A, B, 0.7, save_z=True)
    for t in (Y, Z):
        assert bool((t[2] == INF).all()) and bool((t[T - 1] == -INF).all())
        rows = torch.arange(T, device="cuda")
        assert bool(t[(rows != 2) & (rows != T - 1)].isfinite().all())
    assert torch.equal(U, U0)
    for act in ACTS[1:]:
        Y, _, _ = qn.qlora_linear_fwd_epilogue(w, X, A, B, 0.7, act=act)
        assert bool((Y[2] == INF).all()) and bool(Y[T - 1].isnan().all())


@pytest.mark.parametrize("N,K,T,r", [(1024, 512, 300, 16), (520, 256, 33, 8)])
@pytest.mark.parametrize("spin", [None, "-1"])
def test_an_infinite_activation_with_u_inside_the_launch(qn, monkeypatch, N, K, T, r, spin):
    monkeypatch.setenv("QLORA_NF4_GEMM_TILE", "256")
    assert qn.lib.qlora_linear_fwd_u_in_launch(N, K, T, r) == 1
    if spin:
        monkeypatch.setenv("QLORA_NF4_GEMM_SPIN", spin)  # a tile forms U itself
    w, X, A, B = _positive(qn, T, N, K, r, seed=r)
    X[2, 17], X[T - 1, 200] = INF, -INF
    Y, _, Z = qn.qlora_linear_fwd_epilogue(w, X, A, B, 0.7, save_z=True)
    rows = torch.arange(T, device="cuda")
    for t in (Y, Z):
        assert bool((t[2] == INF).all()) and bool((t[T - 1] == -INF).all())
        assert bool(t[(rows != 2) & (rows != T - 1)].isfinite().all())


@pytest.mark.parametrize("T", [5, 20])
def test_adapter_terms_past_the_bf16_range(qn, T):
    """s U between bf16's largest value and fp32's: bf16 makes it infinite, as
    in the plain forward; no NaN comes of the rest of it."""
    w, X, A, B = _positive(qn, T, 264, 512, 8, seed=3)
    X.abs_()
    U = torch.mm(X.float(), A.float().t())
    Y, _, Z = qn.qlora_linear_fwd_epilogue(w, X, A, B, 3.4e38 / float(U.max()), save_z=True)
    assert not bool(Y.isnan().any()) and not bool(Z.isnan().any())


@pytest.mark.parametrize("path", ["decode", "gemm", "q4g"])
@pytest.mark.parametrize("act", ACTS[1:])
def test_values_everywhere(qn, act, path):
    """act at every bf16 z from -30 to 30, beside the residual -bf16(act(z)), so
    that the sum shows 8 more bits of it: within 2^-15 of the value. The exponent
    (to 126) is formed with 2.5 roundings for GELU, 1.5 for SiLU, 5 for the tanh
    form: 2.7e-5 at most, GELU's 1.1e-5 of its polynomial among them. The factor
    of z may be zero where it is under the smallest normal fp32; bf16 results
    under 2^-126 are steps of 2^-133, rounded by 2^-134."""
    bits = torch.arange(1 << 16, dtype=torch.int32, device="cuda").to(torch.int16).view(BF16)
    bias = bits[bits.float().abs() <= 30]
    bias = bias[:bias.numel() // 8 * 8].contiguous()
    N, T = bias.numel(), 17 if path == "gemm" else 2
    z = bias.double()
    # torch's normal distribution function loses its lower tail
    v = z * 0.5 * torch.special.erfc(-z * math.sqrt(0.5)) if act == "gelu" else _act(z, act)[0]
    res = (-v).to(BF16).expand(T, N).contiguous()
    if path == "q4g":
        w = qn.q4g_quantize(torch.ones(N, 32, device="cuda"), 32)
        Y = qn.q4g_linear_fwd_epilogue(w, torch.zeros(T, 32, dtype=BF16, device="cuda"), bias, act, res)
    else:
        w = qn.quantize_weight(torch.ones(N, 64, device="cuda"))
        Y, _, _ = qn.qlora_linear_fwd_epilogue(w, torch.zeros(T, 64, dtype=BF16, device="cuda"), bias=bias, act=act,
                                               residual=res)
    want = v + res[0].double()
    bad = (Y.double() - want).abs() - (2.0 ** -8 * want.abs() + 2.0 ** -15 * v.abs() + 2.0 ** -126 * z.abs() + 2.0 ** -134)
    assert float(bad.max()) <= 0, (float(bad.max()), float(bias[int(bad.amax(0).argmax())]))
