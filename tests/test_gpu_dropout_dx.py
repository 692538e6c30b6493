"""dX of the layer's backward with dropout is rounded once: element by element
against the 64-bit formula, where dY W' and the masked adapter term cancel too."""

import numpy as np
import pytest
import torch

import workloads

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def qn():
    import bit_nf4_quantized_16_amd as qn

    assert torch.cuda.is_available()
    return qn


def _ints(shape, most, seed):
    g = torch.Generator().manual_seed(seed)
    return torch.randint(-most, most + 1, shape, generator=g).float()


class Case:
    """dY and B small whole numbers, scale a power of two: G = s dY B is exact
    in bf16 and in every fp32 sum, so dX's errors are the fp32 sums' and one
    rounding. ``cancel``: W' all 2^-3 (exact in NF4) and B A near -W'."""

    def __init__(self, qn, T, N, K, r, p, seed, cancel=False, dq=True):
        self.T, self.N, self.K, self.r, self.p, self.s = T, N, K, r, p, 0.5
        W = torch.full((N, K), 0.125) if cancel else workloads.normal_weight(N, K, 0.02, seed)
        self.w = qn.quantize_weight(W.cuda(), double_quant=dq and not cancel)
        self.X = workloads.bf16_normal((T, K), 1.0, seed + 1).cuda()
        # the sums of |dY| |B| stay under 256: G's values are whole multiples of s
        few = torch.rand(T, N, generator=torch.Generator().manual_seed(seed + 2)) < min(1.0, 60 / N)
        dY = _ints((T, N), 1, seed + 3) * few
        B = _ints((N, r), 1, seed + 4)
        A = 0.05 * torch.randn(r, K, generator=torch.Generator().manual_seed(seed + 5))
        if cancel:  # s B A c = -W' (1 + small) on the rank's first component
            B[:, 0] = 1.0
            B[:, 1:] = 0.0
            A[0] = -0.125 * (1 - p) / self.s * (1 + 0.02 * torch.randn(K, generator=torch.Generator().manual_seed(seed + 6)))
        self.dY, self.A, self.B = (t.bfloat16().cuda() for t in (dY, A, B))
        self.keep = workloads.keep_mask(T, K, p, seed + 7)
        self.bits = workloads.pack_keep_bits(self.keep).cuda()

    def exact(self, qn):
        """dX in 64 bits and its bound: 2^-8 of the value (one rounding to
        bf16), and for the fp32 sums over N and r, with c's rounding and
        product, (N + r + 4) 2^-23 of the sums of magnitudes."""
        f = lambda t: t.detach().cpu().double().numpy()
        d, A, B, W = f(self.dY), f(self.A), f(self.B), f(qn.nf4_dequantize(self.w))
        G = self.s * (d @ B)
        assert np.all(G * 2 == np.rint(G * 2)) and np.abs(G).max() < 128  # exact in bf16
        m = self.keep.numpy() / (1.0 - self.p)
        dX = d @ W + m * (G @ A)
        mags = np.abs(d) @ np.abs(W) + m * (np.abs(G) @ np.abs(A))
        return dX, 2.0 ** -8 * np.abs(dX) + (self.N + self.r + 4) * 2.0 ** -23 * mags + 2.0 ** -133


CASES = [(1, 64, 64, 1), (17, 72, 192, 5), (33, 264, 320, 16), (255, 136, 64, 33), (257, 520, 448, 64), (300, 320, 192, 128),
         (1000, 2048, 1024, 16)]


@pytest.mark.parametrize("T,N,K,r", CASES)
@pytest.mark.parametrize("p", [0.05, 0.5])
@pytest.mark.parametrize("cancel", [False, True])
def test_one_rounding(qn, T, N, K, r, p, cancel):
    c = Case(qn, T, N, K, r, p, seed=T + N + r, cancel=cancel, dq=r % 2 == 0)
    want, bound = c.exact(qn)
    dX = qn.qlora_linear_bwd(c.w, c.X, c.dY, c.A, c.B, c.s, need_da=False, need_db=False, keep=c.bits, p=p)[0]
    assert np.all(np.abs(dX.cpu().double().numpy() - want) <= bound)
    x8 = qn.qlora_linear_bwd_act8(c.w, None, c.dY, c.A, c.B, c.s, need_da=False, need_db=False, keep=c.bits, p=p)[0]
    assert torch.equal(dX, x8)


@pytest.mark.parametrize("tile,splits", [("128", None), ("256", "1"), ("256", "3")])
def test_every_plan(qn, monkeypatch, tile, splits):
    """Both tiles, the reduction whole and split (the mask is the first split's)."""
    monkeypatch.setenv("QLORA_NF4_GEMM_TILE", tile)
    if splits:
        monkeypatch.setenv("QLORA_NF4_GEMM_SPLITS", splits)
    for T, r, dq in ((300, 16, True), (130, 100, False)):
        c = Case(qn, T, 328, 384, r, 0.3, seed=T, dq=dq)
        want, bound = c.exact(qn)
        dX = qn.qlora_linear_bwd(c.w, c.X, c.dY, c.A, c.B, c.s, need_da=False, need_db=False, keep=c.bits, p=0.3)[0]
        assert np.all(np.abs(dX.cpu().double().numpy() - want) <= bound)


def test_error_like_without_dropout(qn):
    """Normwise the rounding alone. Spread evenly over a step of 2^-7 of the
    binade's start it is 2^-7 / sqrt(12) of that, root mean square, and with a
    density falling as v^-2 over the binade the values are sqrt(2) of it: 1.6e-3
    of the norm, so under 2^-9 (two independent ones come to 2.3e-3)."""
    c = Case(qn, 512, 1024, 512, 16, 0.1, seed=3)
    c.A = c.A / 16  # the adapter's term under the base's, as in a layer
    want, _ = c.exact(qn)
    dX = qn.qlora_linear_bwd(c.w, c.X, c.dY, c.A, c.B, c.s, need_da=False, need_db=False, keep=c.bits, p=0.1)[0]
    assert np.linalg.norm(dX.cpu().double().numpy() - want) <= 2.0 ** -9 * np.linalg.norm(want)


def test_dropped_entries_take_nothing_of_the_adapter(qn):
    """A NaN or infinite adapter term stays out of the masked entries."""
    c = Case(qn, 70, 136, 128, 8, 0.5, seed=5)
    want = qn.qlora_linear_bwd(c.w, c.X, c.dY, need_da=False, need_db=False)[0]
    A = c.A.clone()
    A[3] = float("nan")
    dX = qn.qlora_linear_bwd(c.w, c.X, c.dY, A, c.B, c.s, need_da=False, need_db=False, keep=c.bits, p=0.5)[0]
    dropped = c.keep.cuda() == 0
    assert torch.equal(dX[dropped], want[dropped]) and torch.isnan(dX[~dropped]).all()


def test_repeated_and_captured(qn):
    c = Case(qn, 300, 264, 320, 16, 0.2, seed=6)
    step = lambda: qn.qlora_linear_bwd(c.w, c.X, c.dY, c.A, c.B, c.s, keep=c.bits, p=0.2)
    one = step()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = step()
    for i in range(3):
        c.dY.copy_(workloads.bf16_normal((300, 264), 1.0, 60 + i).cuda())
        graph.replay()
        torch.cuda.synchronize()
        for a, b in zip(out, step()):
            assert torch.equal(a, b)
    assert one[0].shape == (300, 320)


def test_timers_count_the_masked_product(qn):
    c = Case(qn, 100, 136, 128, 8, 0.2, seed=7)
    timers = [qn.KernelTimer(k) for k in (qn._lib.QL_KERNEL_GEMM_DX, qn._lib.QL_KERNEL_DX_KEEP)]
    for bits, p, want in ((c.bits, 0.2, [1, 1]), (None, 0.0, [1, 0])):
        for t in timers:
            t.arm()
        qn.qlora_linear_bwd(c.w, c.X, c.dY, c.A, c.B, c.s, need_da=False, need_db=False, keep=bits, p=p)
        torch.cuda.synchronize()
        assert [t.read()[0] for t in timers] == want
        for t in timers:
            t.disarm()
