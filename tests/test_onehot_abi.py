"""Host checks of the one-hot operators' C entries: every refusal comes before any device work (no GPU needed)."""
import ctypes

import pytest


@pytest.fixture(scope="module")
def L():
    from sparse_dense_matrix_spmm_gb300 import _lib, build
    build.build()
    return _lib.load()


def _route(T=10, k=2, E=4, order=16, pos=16, offsets=16, keys=16):
    from sparse_dense_matrix_spmm_gb300 import _lib
    return ctypes.byref(_lib.RouteT(T, k, E, order, pos, offsets, keys))


NULL, SHAPE, DTYPE, WORKSPACE, UNSUPPORTED = 1, 2, 3, 5, 8


def test_layout():
    from sparse_dense_matrix_spmm_gb300 import _lib
    assert ctypes.sizeof(_lib.RouteT) == 8 + 8 + 8 + 8 * 4


def test_build_route(L):
    b = L.spmm_build_route
    assert b(16, 8, 2, None, None, 0, None) == NULL
    assert b(None, 8, 2, _route(), None, 0, None) == NULL
    assert b(16, 8, 2, _route(order=None), None, 0, None) == NULL
    assert b(16, 8, 1, _route(), None, 0, None) == SHAPE              # pitch below k
    assert b(16, 8, 2, _route(k=0), None, 0, None) == SHAPE
    assert b(16, 8, 2, _route(E=0), None, 0, None) == SHAPE
    assert b(20, 8, 2, _route(), None, 0, None) == SHAPE              # ids not aligned
    assert b(16, 2, 2, _route(), None, 0, None) == DTYPE
    assert b(16, 8, 2, _route(T=1 << 30, k=2), None, 0, None) == UNSUPPORTED
    assert b(16, 8, 2, _route(E=512), None, 0, None) == WORKSPACE
    n = ctypes.c_size_t(0)
    assert L.spmm_build_route_workspace_size(10, 2, 511, ctypes.byref(n)) == 0 and n.value == 0
    assert L.spmm_build_route_workspace_size(10, 2, 512, ctypes.byref(n)) == 0 and n.value >= 10 * 2 * 8
    assert L.spmm_build_route_workspace_size(-1, 2, 512, ctypes.byref(n)) == SHAPE
    assert L.spmm_build_route_workspace_size(10, 2, 512, None) == NULL


def test_rows(L):
    bf16, i8 = 0, 2
    d, c, g = L.spmm_dispatch, L.spmm_combine, L.spmm_combine_grad
    assert d(None, 16, 64, 16, 64, 64, bf16, None) == NULL
    assert d(_route(), None, 64, 16, 64, 64, bf16, None) == NULL
    assert d(_route(), 16, 63, 16, 64, 64, bf16, None) == SHAPE
    assert d(_route(), 17, 64, 16, 64, 64, bf16, None) == SHAPE        # not aligned to its elements
    assert d(_route(), 16, 64, 16, 64, 64, i8, None) == DTYPE
    assert d(_route(T=0), None, 64, None, 64, 64, bf16, None) == 0     # nothing to write
    assert d(_route(), None, 0, None, 0, 0, bf16, None) == 0
    assert c(_route(), 16, 64, None, None, 64, 64, bf16, None) == NULL
    assert c(_route(), 16, 64, None, 16, 60, 64, bf16, None) == SHAPE
    assert c(_route(), 16, 64, 18, 16, 64, 64, bf16, None) == SHAPE    # weights not aligned
    assert c(_route(), 16, 64, None, 16, 64, 64, 7, None) == DTYPE
    assert g(_route(), 16, 64, 16, 64, None, 16, 64, 16, 64, bf16, None) == NULL
    assert g(_route(), 16, 64, 16, 64, 16, 16, 64, None, 64, bf16, None) == NULL
    assert g(_route(), 16, 64, 16, 8, 16, 16, 64, 16, 64, bf16, None) == SHAPE
    assert g(_route(pos=None), 16, 64, 16, 64, 16, 16, 64, 16, 64, bf16, None) == NULL


def test_embed(L):
    e, g = L.spmm_embed, L.spmm_embed_grad
    assert e(None, 10, 64, 64, 0, 16, 8, 4, 1.0, 16, 64, None) == NULL
    assert e(16, 10, 64, 60, 0, 16, 8, 4, 1.0, 16, 64, None) == SHAPE
    assert e(16, 0, 64, 64, 0, 16, 8, 4, 1.0, 16, 64, None) == SHAPE
    assert e(16, 10, 64, 64, 3, 16, 8, 4, 1.0, 16, 64, None) == DTYPE
    assert e(16, 10, 64, 64, 0, 16, 3, 4, 1.0, 16, 64, None) == DTYPE
    assert e(16, 10, 64, 64, 0, 20, 8, 4, 1.0, 16, 64, None) == SHAPE
    assert e(None, 10, 64, 64, 0, None, 8, 0, 1.0, None, 64, None) == 0
    one = dict(k=1)
    assert g(_route(), 16, 64, 64, 0, 1.0, 0, 16, 64, 0, 16, 1 << 30, None) == SHAPE          # k = 2
    assert g(_route(**one), 16, 64, 64, 0, 1.0, 2, 16, 64, 0, 16, 1 << 30, None) == SHAPE     # accumulate
    assert g(_route(**one), 16, 64, 64, 0, 1.0, 0, 16, 64, 1, 16, 1 << 30, None) == DTYPE     # bf16 to fp16
    assert g(_route(**one), 16, 64, 64, 0, 1.0, 0, None, 64, 0, 16, 1 << 30, None) == NULL
    assert g(_route(keys=None, **one), 16, 64, 64, 0, 1.0, 0, 16, 64, 0, 16, 1 << 30, None) == NULL
    assert g(_route(**one), 16, 64, 64, 0, 1.0, 0, 16, 64, 0, 16, 8, None) == WORKSPACE
    assert g(_route(**one), 16, 60, 64, 0, 1.0, 0, 16, 64, 0, 16, 1 << 30, None) == SHAPE


def test_experts(L):
    f, x, w = L.spmm_experts, L.spmm_experts_dx, L.spmm_experts_dw
    lde = 32 * 64
    for call in (f, x):
        assert call(None, 16, 64, 16, 64, lde, 32, 64, 0, 16, 64, None) == NULL
        assert call(_route(), 16, 64, 16, 64, lde, 32, 64, 5, 16, 64, None) == DTYPE       # fp32
        assert call(_route(), 16, 64, 16, 64, lde, 32, 60, 0, 16, 64, None) == SHAPE       # K % 8
        assert call(_route(), 16, 64, 16, 64, lde, 0, 64, 0, 16, 64, None) == SHAPE
        assert call(_route(), 16, 68, 16, 64, lde, 32, 64, 0, 16, 64, None) == SHAPE       # pitch % 8
        assert call(_route(), 16, 64, 16, 64, lde - 8, 32, 64, 0, 16, 64, None) == SHAPE   # experts overlap
        assert call(_route(), 24, 64, 16, 64, lde, 32, 64, 0, 16, 64, None) == SHAPE       # alignment
        assert call(_route(), 16, 64, None, 64, lde, 32, 64, 0, 16, 64, None) == NULL
        assert call(_route(E=70000), 16, 64, 16, 64, lde, 32, 64, 0, 16, 64, None) == UNSUPPORTED
        assert call(_route(T=(1 << 31) - 100, k=1), 16, 64, 16, 64, lde, 32, 64, 0, 16, 64, None) == UNSUPPORTED
        assert call(_route(), 16, 1 << 30, 16, 1 << 30, 1 << 36, 32, 1 << 30, 0, 16, 1 << 30, None) == UNSUPPORTED
        assert call(_route(T=0), None, 64, None, 64, lde, 32, 64, 0, None, 64, None) == 0
    assert w(_route(), 16, 32, 16, 64, 32, 64, 0, 16, 60, lde, None) == SHAPE
    assert w(_route(), 16, 32, 16, 64, 32, 64, 0, None, 64, lde, None) == NULL
    assert w(_route(), 16, 32, 16, 64, 32, 64, 2, 16, 64, lde, None) == DTYPE
