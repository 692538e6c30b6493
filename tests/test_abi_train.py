"""Refusals of the norms and the losses on logits, before any launch (no GPU)."""

import os

import pytest

from conftest import ROOT

LIB = os.path.join(ROOT, "bit_nf4_quantized_16_amd", "libqlora_nf4.so")
pytestmark = pytest.mark.skipif(not os.path.exists(LIB), reason="library not built")

P, MIS, ODD = 0x10000, 0x10004, 0x10001  # fake device addresses, never dereferenced
INF, NAN = float("inf"), float("nan")


@pytest.fixture(scope="module")
def L():
    from bit_nf4_quantized_16_amd import _lib

    return _lib


@pytest.fixture(scope="module")
def lib(L):
    return L.load(LIB)


def _each(call, L, **by_status):
    for status, cases in by_status.items():
        for kw in cases:
            assert call(**kw) == getattr(L, status), kw


def test_norm_forward(lib, L):
    def call(X=P, xd=L.QL_BF16, rows=4, cols=64, w=P, b=P, wd=L.QL_F32, eps=1e-5, rms=0, Y=P, mean=P, rstd=P):
        return lib.qlora_norm_fwd(X, xd, rows, cols, w, b, wd, eps, rms, Y, mean, rstd, None)

    _each(call, L,
          QL_ERR_SHAPE=[dict(rows=-1), dict(rows=1 << 22), dict(rows=1 << 62), dict(cols=0), dict(cols=-8), dict(cols=12),
                        dict(cols=16392)],
          QL_ERR_UNSUPPORTED=[dict(xd=2), dict(wd=-1), dict(eps=-1.0), dict(eps=INF), dict(eps=NAN), dict(rms=2)],
          QL_ERR_NULL=[dict(X=None), dict(w=None), dict(Y=None)],
          QL_ERR_ALIGN=[dict(X=MIS), dict(w=MIS), dict(b=MIS), dict(Y=MIS), dict(mean=ODD), dict(rstd=ODD)],
          QL_OK=[dict(rows=0, X=None, w=None, Y=None)])


def test_norm_backward(lib, L):
    def call(X=P, xd=L.QL_BF16, rows=4, cols=64, w=P, wd=L.QL_F32, dY=P, mean=P, rstd=P, dX=P, dW=P, dB=P, acc=0, ws=P,
             n=1 << 40):
        return lib.qlora_norm_bwd(X, xd, rows, cols, w, wd, dY, mean, rstd, dX, dW, dB, acc, ws, n, None)

    _each(call, L,
          QL_ERR_SHAPE=[dict(rows=-1), dict(cols=20), dict(cols=1 << 40)],
          QL_ERR_UNSUPPORTED=[dict(xd=7), dict(wd=7), dict(acc=2)],
          QL_ERR_NULL=[dict(X=None), dict(w=None), dict(dY=None), dict(rstd=None)],
          QL_ERR_ALIGN=[dict(X=MIS), dict(w=MIS), dict(dY=MIS), dict(dX=MIS), dict(dW=MIS), dict(dB=MIS), dict(rstd=ODD),
                        dict(ws=MIS)],
          QL_ERR_WORKSPACE=[dict(ws=None), dict(n=lib.qlora_norm_bwd_workspace(4, 64) - 1)],
          QL_OK=[dict(dX=None, dW=None, dB=None, X=None), dict(rows=0, dW=None, dB=None, X=None, rstd=None)])
    assert lib.qlora_norm_bwd_workspace(4, 64) > 0
    for rows, cols in ((0, 64), (-1, 64), (1 << 62, 64), (4, 0), (4, 1 << 40)):
        assert lib.qlora_norm_bwd_workspace(rows, cols) == 0


LOGITS = dict(QL_ERR_SHAPE=[dict(T=-1), dict(T=(1 << 22) + 1), dict(T=1 << 62), dict(V=0), dict(V=-1), dict(V=1 << 30, ld=1 << 30),
                            dict(V=1 << 62), dict(T=1 << 22, V=1 << 14, ld=1 << 14), dict(ld=99), dict(ld=1 << 62)],
              QL_ERR_UNSUPPORTED=[dict(dt=2), dict(dt=-1)],
              QL_ERR_NULL=[dict(z=None), dict(labels=None)],
              QL_ERR_ALIGN=[dict(z=ODD), dict(labels=MIS)])


def _and(base, **more):
    return {k: base.get(k, []) + more.get(k, []) for k in {*base, *more}}


def test_token_logp(lib, L):
    def call(z=P, dt=L.QL_BF16, T=4, V=100, ld=100, labels=P, out=P, ws=P, n=1 << 40):
        return lib.qlora_token_logp(z, dt, T, V, ld, labels, out, ws, n, None)

    big = dict(V=100000, ld=100000)
    _each(call, L, **_and(LOGITS, QL_ERR_NULL=[dict(out=None)], QL_ERR_ALIGN=[dict(out=ODD), dict(ws=MIS, **big)],
                          QL_ERR_WORKSPACE=[dict(ws=None, **big),
                                            dict(n=lib.qlora_token_logp_workspace(4, 100000, L.QL_BF16) - 1, **big)],
                          QL_OK=[dict(T=0, z=None, labels=None, out=None, ws=None)]))
    assert lib.qlora_token_logp_workspace(4, 100000, L.QL_BF16) > 0
    for T, V, dt in ((0, 100000, 1), (-1, 100000, 1), (4, 0, 1), (4, 100000, 9), (1 << 62, 1 << 62, 0)):
        assert lib.qlora_token_logp_workspace(T, V, dt) == 0


def test_preference(lib, L):
    def fwd(z=P, dt=L.QL_BF16, T=4, V=100, ld=100, labels=P, start=P, pairs=2, ref=P, beta=0.1, e=0.0, kind=0, avg=0, loss=P,
            sl=P, state=P, ws=P, n=1 << 40):
        return lib.qlora_preference_loss_fwd(z, dt, T, V, ld, labels, start, pairs, ref, beta, e, kind, avg, loss, sl, state,
                                             ws, n, None)

    _each(fwd, L, **_and(LOGITS, QL_ERR_SHAPE=[dict(pairs=-1), dict(pairs=1 << 40)],
                         QL_ERR_UNSUPPORTED=[dict(beta=0.0), dict(beta=-1.0), dict(beta=INF), dict(beta=NAN), dict(e=-0.1),
                                             dict(e=1.5), dict(e=NAN), dict(kind=3), dict(kind=1, e=0.1), dict(avg=2)],
                         QL_ERR_NULL=[dict(start=None), dict(ref=None), dict(loss=None), dict(sl=None), dict(state=None)],
                         QL_ERR_ALIGN=[dict(start=MIS), dict(ref=ODD), dict(loss=ODD), dict(sl=ODD), dict(state=ODD)],
                         QL_ERR_WORKSPACE=[dict(V=100000, ld=100000, n=0)],
                         QL_OK=[dict(T=0, pairs=0, z=None, labels=None, start=None, ref=None, loss=None, sl=None, state=None)]))

    def bwd(z=P, dt=L.QL_BF16, T=4, V=100, ld=100, labels=P, state=P, dloss=P, pairs=2, dz=P):
        return lib.qlora_preference_loss_bwd(z, dt, T, V, ld, labels, state, dloss, pairs, dz, None)

    _each(bwd, L, **_and(LOGITS, QL_ERR_SHAPE=[dict(pairs=-1)], QL_ERR_NULL=[dict(state=None), dict(dloss=None), dict(dz=None)],
                         QL_ERR_ALIGN=[dict(state=ODD), dict(dloss=ODD), dict(dz=ODD), dict(dz=P + 2), dict(z=P + 2)],
                         QL_OK=[dict(T=0, z=None, labels=None, state=None, dloss=None, dz=None)]))


def test_distill(lib, L):
    def call(z=P, dt=L.QL_BF16, T=4, V=100, ld=100, idx=P, top=P, td=L.QL_F32, K=8, labels=P, tau=1.0, a=0.5, w=P, loss=P,
             dz=P):
        return lib.qlora_distill_loss(z, dt, T, V, ld, idx, top, td, K, labels, tau, a, w, loss, dz, None)

    _each(call, L, **_and(LOGITS, QL_ERR_SHAPE=[dict(K=0), dict(K=257), dict(K=-1)],
                          QL_ERR_UNSUPPORTED=[dict(td=4), dict(tau=0.0), dict(tau=-1.0), dict(tau=INF), dict(tau=NAN), dict(tau=2.0 ** 21),
                                              dict(a=-0.1), dict(a=1.1), dict(a=NAN)],
                          QL_ERR_NULL=[dict(idx=None), dict(top=None)],
                          QL_ERR_ALIGN=[dict(idx=MIS), dict(top=0x10002), dict(w=ODD), dict(loss=ODD), dict(dz=P + 2),
                                        dict(a=0.0, labels=MIS)],
                          QL_OK=[dict(T=0, z=None), dict(loss=None, dz=None, z=None)]))


def test_python_refusals_need_no_gpu(L):
    """Host tensors are refused by name before the library is called."""
    import torch

    import bit_nf4_quantized_16_amd as qn

    z, lab = torch.zeros(4, 10), torch.zeros(4, dtype=torch.int64)
    for call in (lambda: qn.norm_fwd(z, torch.zeros(10)), lambda: qn.norm_bwd(z, torch.zeros(10), z, None, torch.zeros(4)),
                 lambda: qn.token_logp(z, lab), lambda: qn.token_logp(z.half(), lab), lambda: qn.token_logp(z[0], lab),
                 lambda: qn.preference_loss_fwd(z, lab, lab, torch.zeros(2)),
                 lambda: qn.preference_loss_bwd(z, lab, None, torch.zeros(2)),
                 lambda: qn.distill_loss(z, lab[:, None], z[:, :1]), lambda: qn.distill_loss(None, None, None)):
        with pytest.raises(qn.QLoraError):
            call()
