"""Workspace of the backward from a checkpoint by the outputs asked for (CPU:
sizes, and which sizes the calls accept before their first launch)."""

import ctypes
import itertools

import pytest
import torch

# the accepted calls stop at their first launch only where there is no GPU
pytestmark = pytest.mark.skipif(torch.cuda.device_count() > 0, reason="made-up addresses: for machines without a GPU")

P, P2, P3, P4 = (ctypes.c_void_p(0x10000 * i) for i in (1, 2, 3, 4))
BIG = 1 << 40


@pytest.fixture(scope="module")
def L():
    from bit_nf4_quantized_16_amd import _lib

    return _lib


@pytest.fixture(scope="module")
def lib(L):
    return L.load()


def _weight(L, rows, cols):
    w = L.QlNf4Weight()
    w.rows, w.cols, w.blocksize, w.dq_blocksize = rows, cols, 64, 256
    w.packed, w.c8, w.dq_scale, w.dq_mean = 0x10000, 0x30000, 0x40000, 0x50000
    return w


SHAPES = [(4096, 4096, 1024, 16), (11008, 4096, 1000, 16), (4096, 11008, 4096, 64), (72, 128, 33, 8), (64, 64, 2100, 128),
          (4096, 4096, 1, 0)]


def _wishes(r):
    return [w for w in itertools.product((0, 1), repeat=3) if any(w) and (r > 0 or not (w[1] or w[2]))]


@pytest.mark.parametrize("rows,cols,T,r", SHAPES)
@pytest.mark.parametrize("drop", [0, 1])
def test_single(lib, L, rows, cols, T, r, drop):
    full = lib.qlora_linear_bwd_act8_workspace(rows, cols, T, r, drop)
    size = lambda x, a, b: lib.qlora_linear_bwd_act8_workspace_for(rows, cols, T, r, drop, x | a << 1 | b << 2)
    assert size(1, 1, 1) == full and size(0, 0, 0) <= full
    w = _weight(L, rows, cols)
    x8 = L.QlAct8(T, cols, 0x60000, 0x70000)
    for x, a, b in _wishes(r):
        n = size(x, a, b)
        assert n <= full
        if not x:  # no more than G, the terms of two V (6 B a token and padded rank), partials of the sums, projection
            assert n < 64 << 20 and (T > 2048 or n <= 4 * T * r + 12 * (T + 32) * 128 + (4 << 20))

        def call(n):
            return lib.qlora_linear_bwd_act8(w, x8, P, T, P2, P3, r, 1.0, P4 if drop else None, 0.1 if drop else 0.0, P4,
                                             P if x else None, P2 if a else None, P3 if b else None, 0, P, n, None)

        if n > 0:
            assert call(n - 1) == L.QL_ERR_WORKSPACE
        assert call(n) in (L.QL_ERR_HIP, L.QL_OK)  # stops at its launch: no GPU here
    assert lib.qlora_linear_bwd_act8_workspace_for(rows, cols, 0, r, drop, 7) == 0


def test_first_layer_holds_no_partials_of_the_product(lib):
    assert lib.qlora_linear_bwd_act8_workspace(4096, 4096, 1024, 16, 0) > 64 << 20
    assert lib.qlora_linear_bwd_act8_workspace_for(4096, 4096, 1024, 16, 0, 6) < 1 << 20


@pytest.mark.parametrize("T,r", [(33, 8), (1024, 16), (2100, 64), (1, 0)])
def test_group(lib, L, T, r):
    rows = (ctypes.c_int64 * 2)(11008, 72)
    full = lib.qlora_linear_bwd_group_act8_workspace(rows, 2, 4096, T, r)
    size = lambda x, a, b: lib.qlora_linear_bwd_group_act8_workspace_for(rows, 2, 4096, T, r, x | a << 1 | b << 2)
    assert size(1, 1, 1) == full
    ws = [_weight(L, 11008, 4096), _weight(L, 72, 4096)]
    arr = lambda *v: (ctypes.c_void_p * 2)(*v)
    x8 = L.QlAct8(T, 4096, 0x60000, 0x70000)
    for x, a, b in _wishes(r):
        n = size(x, a, b)
        assert n <= full

        # a layer's own wishes within those named: the second one asks for nothing of its own
        def call(n, both=True):
            return lib.qlora_linear_bwd_group_act8(arr(*[ctypes.addressof(w) for w in ws]), 2, x8, arr(P, P), T, arr(P2, P2),
                                                   arr(P3, P3), r, 1.0, arr(P4, P4), P if x else None,
                                                   arr(P2, P2 if both else None) if a else None,
                                                   arr(P3, P3 if both else None) if b else None, 0, P, n, None)

        if n > 0:
            assert call(n - 1) == L.QL_ERR_WORKSPACE
        assert call(n) in (L.QL_ERR_HIP, L.QL_OK) and call(n, False) in (L.QL_ERR_HIP, L.QL_OK)
