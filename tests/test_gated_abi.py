"""Host checks of the gated experts' C entries: every refusal comes before any device work (no GPU needed)."""
import ctypes

import pytest

from tests.test_onehot_abi import _route

NULL, SHAPE, DTYPE, WORKSPACE, UNSUPPORTED = 1, 2, 3, 5, 8
BF16, F16, I8, F32 = 0, 1, 2, 5


@pytest.fixture(scope="module")
def L():
    from sparse_dense_matrix_spmm_gb300 import _lib, build
    build.build()
    return _lib.load()


def _rows8(rows=20, cols=64, q=16, ldq=64, scale=16, lds=4):
    from sparse_dense_matrix_spmm_gb300 import _lib
    return ctypes.byref(_lib.Rows8T(rows, cols, q, ldq, scale, lds))


def test_layout():
    from sparse_dense_matrix_spmm_gb300 import _lib
    assert ctypes.sizeof(_lib.Rows8T) == 6 * 8


def test_topk(L):
    f = L.spmm_topk
    ok = dict(logits=16, T=10, E=40, ldl=40, dt=F32, k=4, renorm=1, ids=16, idb=8, w=16)

    def call(**kw):
        a = dict(ok, **kw)
        return f(a["logits"], a["T"], a["E"], a["ldl"], a["dt"], a["k"], a["renorm"], a["ids"], a["idb"], a["w"], None)

    assert call(T=0, logits=None, ids=None, w=None) == 0
    assert call(logits=None) == NULL and call(ids=None) == NULL and call(w=None) == NULL
    assert call(dt=I8) == DTYPE and call(idb=2) == DTYPE
    for bad in (dict(T=-1), dict(E=0), dict(k=0), dict(k=41), dict(renorm=2), dict(ldl=39), dict(ids=20), dict(w=18),
                dict(logits=18), dict(ldl=1 << 40)):
        assert call(**bad) == SHAPE, bad
    assert call(E=1025, ldl=1025) == UNSUPPORTED and call(k=33) == UNSUPPORTED
    assert call(T=1 << 31) == UNSUPPORTED and call(T=1 << 30, k=4) == UNSUPPORTED


def test_topk_grad(L):
    f = L.spmm_topk_grad
    ok = dict(logits=16, T=10, E=40, ldl=40, dt=F16, k=4, renorm=0, ids=16, idb=4, w=16, dw=16, d=16, ldd=40)

    def call(**kw):
        a = dict(ok, **kw)
        return f(a["logits"], a["T"], a["E"], a["ldl"], a["dt"], a["k"], a["renorm"], a["ids"], a["idb"], a["w"], a["dw"],
                 a["d"], a["ldd"], None)

    assert call(T=0, logits=None, ids=None, w=None, dw=None, d=None) == 0
    for name in ("logits", "ids", "w", "dw", "d"):
        assert call(**{name: None}) == NULL, name
    for bad in (dict(ldd=39), dict(k=41), dict(logits=17), dict(dw=18), dict(d=17), dict(ids=18)):
        assert call(**bad) == SHAPE, bad
    assert call(dt=7) == DTYPE and call(E=2000, ldl=2000, ldd=2000) == UNSUPPORTED


def test_rows8(L):
    p, u = L.spmm_pack_rows, L.spmm_unpack_rows

    def both(P, x=16, ld=64, dt=BF16):
        r = p(x, ld, dt, P, None), u(P, x, ld, dt, None)
        assert r[0] == r[1]
        return r[0]

    assert both(None) == NULL and both(_rows8(), x=None) == NULL
    assert both(_rows8(q=None)) == NULL and both(_rows8(scale=None)) == NULL
    assert both(_rows8(), dt=I8) == DTYPE
    assert both(_rows8(), ld=63) == SHAPE and both(_rows8(ldq=63)) == SHAPE and both(_rows8(lds=3)) == SHAPE
    assert both(_rows8(), x=17) == SHAPE and both(_rows8(), x=18, dt=F32) == SHAPE
    assert both(_rows8(rows=-1)) == SHAPE and both(_rows8(cols=-1)) == SHAPE
    assert both(_rows8(rows=1 << 31)) == UNSUPPORTED
    assert both(_rows8(rows=0), x=None) == 0 and both(_rows8(cols=0), x=None) == 0


def test_experts_gated(L):
    f = L.spmm_experts_gated
    N, K = 32, 64
    ok = dict(R=_route(), xs=16, ldx=K, W=16, ldw=K, lde=2 * N * K, N=N, K=K, dt=BF16, act=0, h=16, ldh=N, gu=None, ldgu=2 * N,
              P=None)

    def call(**kw):
        a = dict(ok, **kw)
        return f(a["R"], a["xs"], a["ldx"], a["W"], a["ldw"], a["lde"], a["N"], a["K"], a["dt"], a["act"], a["h"], a["ldh"],
                 a["gu"], a["ldgu"], a["P"], None)

    assert call(R=_route(T=0), xs=None, W=None, h=None) == 0
    for name in ("R", "xs", "W", "h"):
        assert call(**{name: None}) == NULL, name
    assert call(dt=F32) == DTYPE
    for bad in (dict(N=24), dict(N=0), dict(K=60), dict(ldx=60), dict(ldx=68), dict(ldh=24), dict(ldh=36), dict(lde=2 * N * K - 8),
                dict(ldw=56), dict(xs=24), dict(W=24), dict(h=24), dict(gu=24), dict(gu=16, ldgu=56), dict(gu=16, ldgu=68),
                dict(P=_rows8(rows=19)), dict(P=_rows8(cols=48)), dict(P=_rows8(ldq=72)), dict(P=_rows8(q=24)),
                dict(P=_rows8(lds=3))):
        assert call(**bad) == SHAPE, bad
    assert call(P=_rows8(q=None)) == NULL and call(P=_rows8(scale=None)) == NULL
    for bad in (dict(act=3), dict(act=-1), dict(gu=16, P=_rows8()), dict(R=_route(E=70000)), dict(N=1 << 29),
                dict(R=_route(T=(1 << 31) - 100, k=1))):
        assert call(**bad) == UNSUPPORTED, bad


def test_gated_grad(L):
    f = L.spmm_gated_grad
    N = 32
    ok = dict(R=_route(), dh=16, lddh=N, gu=16, ldgu=2 * N, P=None, N=N, dt=F16, act=2, dgu=16, lddgu=2 * N, h=None, ldh=N)

    def call(**kw):
        a = dict(ok, **kw)
        return f(a["R"], a["dh"], a["lddh"], a["gu"], a["ldgu"], a["P"], a["N"], a["dt"], a["act"], a["dgu"], a["lddgu"], a["h"],
                 a["ldh"], None)

    assert call(R=_route(T=0), dh=None, gu=None, dgu=None) == 0
    for name in ("R", "dh", "gu", "dgu"):
        assert call(**{name: None}) == NULL, name
    assert call(dt=F32) == DTYPE
    for bad in (dict(N=24), dict(N=0), dict(lddh=24), dict(lddh=36), dict(ldgu=56), dict(lddgu=60), dict(lddgu=68), dict(dh=24),
                dict(gu=24), dict(dgu=24), dict(h=24), dict(h=16, ldh=24), dict(gu=None, P=_rows8(rows=21)),
                dict(gu=None, P=_rows8(ldq=80, q=18))):
        assert call(**bad) == SHAPE, bad
    assert call(act=9) == UNSUPPORTED and call(P=_rows8()) == UNSUPPORTED and call(gu=None, P=_rows8(q=None)) == NULL


def test_experts_gated_grad(L):
    f = L.spmm_experts_gated_grad
    N, K = 32, 64
    ok = dict(R=_route(), dh=16, lddh=N, xs=16, ldx=K, xs8=None, W=16, ldw=K, lde=2 * N * K, gu=16, ldgu=2 * N, P=None, N=N, K=K,
              dt=BF16, act=0, dgu=16, lddgu=2 * N, dxs=16, lddx=K, dW=16, lddw=K, ldde=2 * N * K, ws=None, wsb=0)

    def call(**kw):
        a = dict(ok, **kw)
        return f(*(a[n] for n in ok), None)

    x8 = _rows8(cols=K, ldq=K)
    for name in ("R", "dh", "xs", "W", "gu", "dgu", "dxs", "dW"):
        assert call(**{name: None}) == NULL, name
    assert call(dt=F32) == DTYPE
    for bad in (dict(N=24), dict(K=60), dict(lddh=24), dict(ldx=56), dict(ldx=68), dict(ldw=56), dict(lde=2 * N * K - 8),
                dict(ldgu=56), dict(lddgu=56), dict(lddx=60), dict(lddw=60), dict(ldde=2 * N * K - 8), dict(xs=24), dict(W=24),
                dict(dxs=24), dict(dW=24), dict(gu=24), dict(dh=24), dict(dgu=24), dict(xs=None, xs8=_rows8(rows=19)),
                dict(xs=None, xs8=_rows8(cols=48)), dict(xs=None, xs8=x8, ws=24, wsb=1 << 20)):
        assert call(**bad) == SHAPE, bad
    assert call(xs8=x8) == UNSUPPORTED and call(P=_rows8()) == UNSUPPORTED and call(act=5) == UNSUPPORTED
    assert call(xs=None, xs8=x8) == WORKSPACE and call(xs=None, xs8=x8, ws=16, wsb=20 * K * 2 - 1) == WORKSPACE
    assert call(xs=None, xs8=_rows8(cols=K, ldq=K, q=None), ws=16, wsb=1 << 20) == NULL
    n = ctypes.c_size_t(0)
    size = L.spmm_experts_gated_grad_workspace_size
    assert size(_route(), N, K, 1, ctypes.byref(n)) == 0 and n.value == 20 * K * 2
    assert size(_route(), N, K, 0, ctypes.byref(n)) == 0 and n.value == 0
    assert size(_route(), N, K, 2, ctypes.byref(n)) == SHAPE and size(_route(), N, 60, 1, ctypes.byref(n)) == SHAPE
    assert size(_route(), 24, K, 1, ctypes.byref(n)) == SHAPE and size(_route(E=70000), N, K, 1, ctypes.byref(n)) == UNSUPPORTED
    assert size(_route(), N, K, 1, None) == NULL and size(None, N, K, 1, ctypes.byref(n)) == NULL


@pytest.mark.parametrize("rows,E,N,K", [(65536, 2, 128, 256), (16384, 2, 256, 512), (5000, 1, 64, 64), (50000, 12, 80, 248),
                                        (1 << 20, 3, 16, 8)])
def test_room_for_the_parts_of_dw(L, rows, E, N, K):
    """Parts fill the 76 CTA pairs (or 152 CTAs, up to 128 rows of dW) once at most, with 256 rows each on average; experts
    have 4096 on average."""
    n = ctypes.c_size_t(0)
    assert L.spmm_experts_gated_grad_workspace_size(_route(T=rows, k=1, E=E), N, K, 0, ctypes.byref(n)) == 0
    parts, rest = divmod(n.value, E * 2 * N * K * 4)
    side = 256 if 2 * N > 128 else 128
    units = E * -(-2 * N // side) * -(-K // 256)
    assert rest == 0 and parts == min((76 if side == 256 else 152) // units, rows // (256 * E)) and parts > 1
    assert n.value <= 20 << 20
    assert L.spmm_experts_gated_grad_workspace_size(_route(T=rows, k=1, E=E), N, K, 1, ctypes.byref(n)) == 0
    assert n.value == parts * E * 2 * N * K * 4 + rows * K * 2


def test_no_room_where_dw_is_large(L):
    n = ctypes.c_size_t(0)
    for rows, E, N, K in ((65536, 16, 1280, 3584), (900, 2, 64, 64), (65536, 64, 128, 512), (8, 2, 16, 64), (16384, 8, 256, 512)):
        assert L.spmm_experts_gated_grad_workspace_size(_route(T=rows, k=1, E=E), N, K, 0, ctypes.byref(n)) == 0
        assert n.value == 0
