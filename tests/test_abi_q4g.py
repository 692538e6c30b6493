"""Refusals of the 4-bit group-scale entry points, before any launch (no GPU)."""

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


def test_sizes(lib):
    assert lib.q4g_packed_bytes(3, 40) == 3 * 32
    assert lib.q4g_packed_bytes(4096, 4096) == 4096 * 2048
    assert lib.q4g_num_groups(3, 40, 32) == 6 and lib.q4g_num_groups(3, 136, 128) == 6
    assert lib.q4g_packed_bytes(0, 40) == 0 and lib.q4g_packed_bytes(3, 41) == 0
    assert lib.q4g_num_groups(3, 40, 48) == 0 and lib.q4g_num_groups(-3, 40, 32) == 0
    assert lib.q4g_packed_bytes(1 << 40, 1 << 40) == 0


def test_quantize(lib, L):
    def call(W=P, wd=L.QL_BF16, rows=4, cols=64, group=32, packed=P, scale=P2, sd=L.QL_BF16, zero=P3):
        return lib.q4g_quantize(W, wd, rows, cols, group, packed, scale, sd, zero, None)

    for rows, cols in ((0, 64), (-1, 64), (4, 0), (4, 60), (1 << 27, 64), (1, 1 << 34)):
        assert call(rows=rows, cols=cols) == L.QL_ERR_SHAPE
    assert call(wd=5) == L.QL_ERR_UNSUPPORTED and call(sd=5) == L.QL_ERR_UNSUPPORTED
    for g in (0, 16, 48, 256, -32):
        assert call(group=g) == L.QL_ERR_UNSUPPORTED
    for k in ("W", "packed", "scale"):
        assert call(**{k: None}) == L.QL_ERR_NULL
    for k in ("W", "packed", "scale", "zero"):
        assert call(**{k: MIS}) == L.QL_ERR_ALIGN


def _w(L, **kw):
    d = dict(dict(rows=4, cols=64, group=32, scale_dtype=L.QL_BF16, packed=P, scale=P2, zero=P3), **kw)
    return L.QlQ4GWeight(*[d[k] for k, _ in L.QlQ4GWeight._fields_])


def test_dequantize_and_linear(lib, L):
    for call in (lambda w, o=P: lib.q4g_dequantize(w, o, L.QL_BF16, None),
                 lambda w, o=P: lib.q4g_linear_fwd(w, P2, 3, o, None)):
        assert call(None) == L.QL_ERR_NULL
        for k in ("packed", "scale"):
            assert call(_w(L, **{k: None})) == L.QL_ERR_NULL
        for k in ("packed", "scale", "zero"):
            assert call(_w(L, **{k: MIS})) == L.QL_ERR_ALIGN
        assert call(_w(L, rows=0)) == L.QL_ERR_SHAPE and call(_w(L, cols=20)) == L.QL_ERR_SHAPE
        assert call(_w(L, rows=1 << 27)) == L.QL_ERR_SHAPE
        assert call(_w(L, group=96)) == L.QL_ERR_UNSUPPORTED and call(_w(L, scale_dtype=2)) == L.QL_ERR_UNSUPPORTED
        assert call(_w(L), None) == L.QL_ERR_NULL and call(_w(L), MIS) == L.QL_ERR_ALIGN
    assert lib.q4g_dequantize(_w(L), P, 3, None) == L.QL_ERR_UNSUPPORTED
    assert lib.q4g_linear_fwd(_w(L), P, -1, P2, None) == L.QL_ERR_SHAPE
    assert lib.q4g_linear_fwd(_w(L), P, (1 << 21) + 1, P2, None) == L.QL_ERR_SHAPE
    assert lib.q4g_linear_fwd(_w(L), None, 3, P2, None) == L.QL_ERR_NULL
    assert lib.q4g_linear_fwd(_w(L), MIS, 3, P2, None) == L.QL_ERR_ALIGN
    assert lib.q4g_linear_fwd(_w(L), None, 0, None, None) == L.QL_OK
