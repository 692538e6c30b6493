"""Refusals of the linear forwards with an epilogue and of its backward, before
any launch (no GPU)."""

import ctypes
import os

import pytest

from conftest import ROOT

LIB = os.path.join(ROOT, "bit_nf4_quantized_16_amd", "libqlora_nf4.so")
pytestmark = pytest.mark.skipif(not os.path.exists(LIB), reason="library not built")

P, MIS = 0x10000, 0x10004  # fake device addresses, never dereferenced


@pytest.fixture(scope="module")
def L():
    from bit_nf4_quantized_16_amd import _lib

    return _lib


@pytest.fixture(scope="module")
def lib(L):
    return L.load(LIB)


def _e(L, bias=P, act=2, residual=P, Z=P, z_dtype=0):
    return L.QlEpilogue(bias, act, residual, Z, z_dtype)


def test_linear(lib, L):
    w = L.QlNf4Weight(64, 128, 64, 256, P, P, P, P, P)

    def call(w=w, X=P, T=4, A=P, B=P, r=8, keep=None, p=0.0, e=_e(L), Y=P, U=P, ws=P, n=1 << 40):
        return lib.qlora_linear_fwd_epilogue(w, X, T, A, B, r, 1.0, keep, p, e, Y, U, ws, n, None)

    for status, cases in (
            ("QL_ERR_NULL", [dict(w=None), dict(X=None), dict(e=None), dict(Y=None), dict(A=None), dict(B=None)]),
            ("QL_ERR_SHAPE", [dict(T=-1), dict(r=-1), dict(r=1000), dict(w=L.QlNf4Weight(60, 128, 64, 256, P, P, P, P, P))]),
            ("QL_ERR_UNSUPPORTED", [dict(e=_e(L, act=4)), dict(e=_e(L, act=-1)), dict(e=_e(L, z_dtype=2)), dict(p=0.1), dict(keep=P, p=1.0),
                                    dict(e=_e(L, act=9), T=0)]),
            ("QL_ERR_ALIGN", [dict(e=_e(L, bias=MIS)), dict(e=_e(L, residual=MIS)), dict(e=_e(L, Z=MIS)), dict(X=MIS),
                              dict(Y=MIS), dict(ws=MIS), dict(U=MIS)]),
            ("QL_ERR_WORKSPACE", [dict(ws=None), dict(n=0)]),
            ("QL_OK", [dict(T=0, X=None, Y=None)])):
        for kw in cases:
            assert call(**kw) == getattr(L, status), kw


def test_q4g(lib, L):
    w = L.QlQ4GWeight(64, 128, 32, L.QL_BF16, P, P, P)

    def call(w=w, X=P, T=4, e=_e(L, Z=None), Y=P):
        return lib.q4g_linear_fwd_epilogue(w, X, T, e, Y, None)

    for status, cases in (
            ("QL_ERR_NULL", [dict(w=None), dict(X=None), dict(e=None), dict(Y=None)]),
            ("QL_ERR_SHAPE", [dict(T=-1), dict(T=(1 << 21) + 1)]),
            ("QL_ERR_UNSUPPORTED", [dict(e=_e(L)), dict(e=_e(L, act=4, Z=None))]),
            ("QL_ERR_ALIGN", [dict(e=_e(L, bias=MIS, Z=None)), dict(e=_e(L, residual=MIS, Z=None)), dict(X=MIS), dict(Y=MIS)]),
            ("QL_OK", [dict(T=0, X=None, Y=None)])):
        for kw in cases:
            assert call(**kw) == getattr(L, status), kw


def test_backward(lib, L):
    def call(dY=P, Z=P, zd=1, rows=4, cols=64, act=2, dZ=P, db=P, acc=0, ws=P, n=1 << 40):
        return lib.qlora_epilogue_bwd(dY, Z, zd, rows, cols, act, dZ, db, acc, ws, n, None)

    need = lib.qlora_epilogue_bwd_workspace(4, 64)
    assert need >= 256
    for status, cases in (
            ("QL_ERR_NULL", [dict(dY=None), dict(Z=None)]),
            ("QL_ERR_SHAPE", [dict(rows=-1), dict(rows=1 << 32), dict(cols=0), dict(cols=12), dict(cols=1 << 40),
                              dict(rows=1 << 20, cols=1 << 21)]),
            ("QL_ERR_UNSUPPORTED", [dict(act=4), dict(act=-1), dict(zd=2), dict(acc=3)]),
            ("QL_ERR_ALIGN", [dict(dY=MIS), dict(Z=MIS), dict(dZ=MIS), dict(db=MIS), dict(ws=MIS)]),
            ("QL_ERR_WORKSPACE", [dict(ws=None), dict(n=need - 1)]),
            ("QL_OK", [dict(dZ=None, db=None, dY=None, Z=None), dict(rows=0, db=None, dY=None)])):
        for kw in cases:
            assert call(**kw) == getattr(L, status), kw
    for rows, cols in ((0, 64), (-1, 64), (4, 0), (4, 20), (1 << 62, 64), (4, 1 << 62)):
        assert lib.qlora_epilogue_bwd_workspace(rows, cols) == 0


def test_the_struct_has_the_headers_layout(L):
    assert ctypes.sizeof(L.QlEpilogue) == 40 and L.QlEpilogue.residual.offset == 16


def test_python_refusals_need_no_gpu():
    import torch

    import bit_nf4_quantized_16_amd as qn

    z = torch.zeros(4, 64, dtype=torch.bfloat16)
    u8 = torch.zeros(64 * 32, dtype=torch.uint8)
    w = qn.NF4Weight(64, 64, u8, c8=u8, dq_scale=torch.zeros(1), dq_mean=torch.zeros(1))
    for call in (lambda: qn.qlora_linear_fwd_epilogue(w, z), lambda: qn.qlora_linear_fwd_epilogue(w, None),
                 lambda: qn.epilogue_bwd(z, z, "gelu"), lambda: qn.epilogue_bwd(z[0]),
                 lambda: qn.q4g_linear_fwd_epilogue(qn.Q4GWeight(64, 64, 32, u8.view(64, 32), z, None), z)):
        with pytest.raises(qn.QLoraError):
            call()


def test_backward_refuses_more_columns_than_a_launch_can_add(lib, L):
    last = (1 << 27) - 8
    assert lib.qlora_epilogue_bwd_workspace(1, last) == 4 * last
    assert lib.qlora_epilogue_bwd_workspace(1, last + 8) == 0
    assert lib.qlora_epilogue_bwd(P, P, 1, 1, last + 8, 2, P, P, 0, P, 1 << 40, None) == L.QL_ERR_SHAPE
