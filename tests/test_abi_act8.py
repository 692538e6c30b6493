"""Refusals of the 8-bit activation entry points, before any launch (no GPU)."""

import ctypes
import os

import pytest

from conftest import ROOT

LIB = os.path.join(ROOT, "bit_nf4_quantized_16_amd", "libqlora_nf4.so")
pytestmark = pytest.mark.skipif(not os.path.exists(LIB), reason="library not built")

P, P2, P3, MIS = 0x10000, 0x20000, 0x30000, 0x10004  # fake device addresses, never dereferenced


@pytest.fixture(scope="module")
def L():
    from bit_nf4_quantized_16_amd import _lib

    return _lib


@pytest.fixture(scope="module")
def lib(L):
    return L.load(LIB)


def _act(L, rows=4, cols=64, codes=P, scale=P2):
    return L.QlAct8(rows, cols, codes, scale)


def test_quantize_and_dequantize(lib, L):
    for call in (lambda a, p=P3: lib.act8_quantize(p, a, None), lambda a, p=P3: lib.act8_dequantize(a, p, L.QL_BF16, None)):
        assert call(None) == L.QL_ERR_NULL
        assert call(_act(L, rows=-1)) == L.QL_ERR_SHAPE
        assert call(_act(L, cols=0)) == L.QL_ERR_SHAPE
        assert call(_act(L, cols=48)) == L.QL_ERR_SHAPE
        assert call(_act(L, rows=(1 << 34) // 64 + 1)) == L.QL_ERR_SHAPE
        assert call(_act(L, rows=1 << 62, cols=1 << 40)) == L.QL_ERR_SHAPE
        assert call(_act(L, codes=None)) == L.QL_ERR_NULL
        assert call(_act(L, scale=None)) == L.QL_ERR_NULL
        assert call(_act(L, codes=MIS)) == L.QL_ERR_ALIGN
        assert call(_act(L, scale=MIS)) == L.QL_ERR_ALIGN
        assert call(_act(L), None) == L.QL_ERR_NULL
        assert call(_act(L), MIS) == L.QL_ERR_ALIGN
        assert call(_act(L, rows=0, codes=None, scale=None), None) == L.QL_OK
    assert lib.act8_dequantize(_act(L), P3, 9, None) == L.QL_ERR_UNSUPPORTED


def _weight(L, rows=256, cols=128, dq=256, **over):
    w = L.QlNf4Weight()
    w.rows, w.cols, w.blocksize, w.dq_blocksize = rows, cols, 64, dq
    w.packed, w.absmax, w.c8, w.dq_scale, w.dq_mean = 0x10000, 0x20000, 0x30000, 0x40000, 0x50000
    for k, v in over.items():
        setattr(w, k, v)
    return w


BIG = 1 << 40


def test_linear_bwd(lib, L):
    x8 = lambda **kw: _act(L, **dict(dict(rows=32, cols=128), **kw))
    need = lib.qlora_linear_bwd_act8_workspace(256, 128, 32, 8, 0)
    assert need > 0
    assert lib.qlora_linear_bwd_act8_workspace(256, 128, 0, 8, 0) == 0
    assert lib.qlora_linear_bwd_act8_workspace(256, 128, 32, 129, 0) == 0

    def call(w=None, x=x8(), dY=P, T=32, A=P, B=P, r=8, keep=None, p=0.0, U=P, dX=P, dA=P, dB=P, acc=0, ws=P, wsb=BIG):
        return lib.qlora_linear_bwd_act8(w or _weight(L), x, dY, T, A, B, r, 1.0, keep, p, U, dX, dA, dB, acc, ws, wsb, None)

    assert call(x=None) == L.QL_ERR_NULL
    assert call(x=x8(rows=31)) == L.QL_ERR_SHAPE and call(x=x8(cols=64)) == L.QL_ERR_SHAPE
    assert call(x=x8(codes=None)) == L.QL_ERR_NULL and call(x=x8(scale=MIS)) == L.QL_ERR_ALIGN
    assert call(U=None) == L.QL_ERR_NULL and "dB" in lib.qlora_last_error().decode()
    assert call(U=MIS) == L.QL_ERR_ALIGN
    assert call(T=-1) == L.QL_ERR_SHAPE
    assert call(r=129) == L.QL_ERR_SHAPE and call(r=-1) == L.QL_ERR_SHAPE
    assert call(r=0) == L.QL_ERR_SHAPE  # dA / dB with rank 0
    assert call(w=_weight(L, cols=96)) == L.QL_ERR_SHAPE
    assert call(w=_weight(L, rows=252)) == L.QL_ERR_SHAPE
    assert call(acc=2) == L.QL_ERR_UNSUPPORTED
    assert call(p=0.1) == L.QL_ERR_UNSUPPORTED  # no mask
    assert call(keep=P, p=1.0) == L.QL_ERR_UNSUPPORTED and call(keep=P, p=-0.1) == L.QL_ERR_UNSUPPORTED
    assert call(keep=MIS, p=0.1) == L.QL_ERR_ALIGN
    for k in ("dY", "A", "B"):
        assert call(**{k: None}) == L.QL_ERR_NULL
    for k in ("dY", "A", "B", "dX", "dA", "dB"):
        assert call(**{k: MIS}) == L.QL_ERR_ALIGN
    assert call(ws=None) == L.QL_ERR_WORKSPACE and call(wsb=need - 1) == L.QL_ERR_WORKSPACE
    assert call(ws=MIS) == L.QL_ERR_ALIGN
    assert call(T=0, x=x8(rows=0), dY=None, U=None, ws=None, wsb=0) == L.QL_OK
    assert call(dX=None, dA=None, dB=None, dY=None, x=None, U=None, ws=None, wsb=0) == L.QL_OK


def test_linear_bwd_group(lib, L):
    import ctypes

    ws = [_weight(L), _weight(L, rows=64)]
    rows = (ctypes.c_int64 * 2)(256, 64)
    need = lib.qlora_linear_bwd_group_act8_workspace(rows, 2, 128, 32, 8)
    assert need > 0
    assert lib.qlora_linear_bwd_group_act8_workspace(None, 2, 128, 32, 8) == 0
    assert lib.qlora_linear_bwd_group_act8_workspace(rows, 5, 128, 32, 8) == 0
    arr = lambda *v: (ctypes.c_void_p * len(v))(*v)
    wp = lambda: arr(*[ctypes.addressof(w) for w in ws])
    x8 = _act(L, rows=32, cols=128)

    def call(w=None, nw=2, x=x8, dY=arr(P, P), T=32, A=arr(P, P), B=arr(P, P), r=8, U=arr(P, P), dX=P, dA=arr(P, P),
             dB=arr(P, P), acc=0, s=P, sb=BIG):
        return lib.qlora_linear_bwd_group_act8(w or wp(), nw, x, dY, T, A, B, r, 1.0, U, dX, dA, dB, acc, s, sb, None)

    assert call(nw=0) == L.QL_ERR_SHAPE and call(nw=5) == L.QL_ERR_SHAPE
    assert call(x=None) == L.QL_ERR_NULL
    assert call(x=_act(L, rows=32, cols=64)) == L.QL_ERR_SHAPE
    for k in ("dY", "A", "B", "U"):
        assert call(**{k: None}) == L.QL_ERR_NULL
        assert call(**{k: arr(P, None)}) == L.QL_ERR_NULL
    assert call(dA=arr(P, MIS)) == L.QL_ERR_ALIGN
    assert call(s=None) == L.QL_ERR_WORKSPACE and call(sb=need - 1) == L.QL_ERR_WORKSPACE
    ws[1].cols = 64
    assert call() == L.QL_ERR_SHAPE
    ws[1].cols, ws[1].dq_blocksize = 128, 0
    assert call() == L.QL_ERR_UNSUPPORTED


def test_swiglu(lib, L):
    a = _act(L)
    fwd = lambda g=P, u=P2, rows=4, cols=64, h=P3, g8=a, u8=a, h8=a: lib.qlora_swiglu_fwd(g, u, rows, cols, h, g8, u8, h8, None)
    assert fwd(rows=-1) == L.QL_ERR_SHAPE
    assert fwd(cols=33) == L.QL_ERR_SHAPE
    for k in ("g8", "u8", "h8"):
        assert fwd(**{k: _act(L, rows=5)}) == L.QL_ERR_SHAPE
        assert fwd(**{k: _act(L, cols=32)}) == L.QL_ERR_SHAPE
        assert fwd(**{k: _act(L, codes=None)}) == L.QL_ERR_NULL
        assert fwd(**{k: _act(L, scale=MIS)}) == L.QL_ERR_ALIGN
    for k in ("g", "u", "h"):
        assert fwd(**{k: None}) == L.QL_ERR_NULL
        assert fwd(**{k: MIS}) == L.QL_ERR_ALIGN
    assert fwd(rows=0, g=None, u=None, h=None, g8=None, u8=None, h8=None) == L.QL_OK
    bwd = lambda g8=a, u8=a, d=P, dg=P2, du=P3: lib.qlora_swiglu_bwd(g8, u8, d, dg, du, None)
    assert bwd(g8=None) == L.QL_ERR_NULL and bwd(u8=None) == L.QL_ERR_NULL
    assert bwd(u8=_act(L, rows=5)) == L.QL_ERR_SHAPE
    for k in ("d", "dg", "du"):
        assert bwd(**{k: None}) == L.QL_ERR_NULL
        assert bwd(**{k: MIS}) == L.QL_ERR_ALIGN
