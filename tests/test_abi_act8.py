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
