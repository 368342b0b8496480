"""Routes (ids sorted by key) and the rows moved through them, against plain
64-bit definitions: order, places and offsets exact, sums within derived bounds."""
import numpy as np
import pytest

from tests.gpu_util import need_gpu
from tests.onehot_util import DT, check, f64, matrix, route

pytestmark = pytest.mark.gpu


def _ids(T, k, n_keys, seed, drop=0.0, skew=1.0):
    rng = np.random.default_rng(seed)
    ids = np.minimum((rng.random((T, k)) ** skew * n_keys).astype(np.int64), n_keys - 1)
    return np.where(rng.random((T, k)) < drop, -1 - rng.integers(0, 5, (T, k)), ids)


def _build(ids, n_keys, dtype=np.int64):
    import torch

    import sparse_dense_matrix_spmm_gb300 as spmm
    return spmm.spmm_build_route(torch.from_numpy(ids.astype(dtype)).cuda(), n_keys)


def _same_route(R, ids, n_keys):
    order, pos, offsets = route(ids, n_keys)
    assert np.array_equal(R.order.cpu().numpy(), order)
    assert np.array_equal(R.pos.cpu().numpy(), pos)
    assert np.array_equal(R.offsets.cpu().numpy(), offsets)
    if R.k == 1:
        flat = np.asarray(ids).reshape(-1)[order]
        assert np.array_equal(R.keys.cpu().numpy(), np.where((flat < 0) | (flat >= n_keys), n_keys, flat))


@pytest.mark.parametrize("dtype", [np.int32, np.int64])
@pytest.mark.parametrize("T,k,n_keys,drop,skew", [
    (1, 1, 1, 0.0, 1), (1, 8, 128, 0.0, 1), (7, 3, 2, 0.5, 1), (33, 1, 511, 0.0, 1), (1000, 3, 512, 0.1, 1),
    (1025, 1, 513, 0.0, 3), (4097, 2, 60, 0.05, 2), (16384, 8, 256, 0.01, 1), (70001, 1, 200000, 0.1, 8),
    (3001, 1, 300000, 0.0, 1), (140000, 2, 5, 0.0, 1), (5000, 1, 1 << 28, 0.0, 1)])
def test_route_is_the_stable_sort(dtype, T, k, n_keys, drop, skew):
    need_gpu()
    if n_keys > 1 << 27 and dtype == np.int32:
        pytest.skip("one run with a gigabyte of offsets")
    ids = _ids(T, k, n_keys, T + k, drop, skew)
    R = _build(ids, n_keys, dtype)
    if n_keys <= 1 << 27:
        _same_route(R, ids, n_keys)
        return
    # many more keys than ids: the offsets are compared where they step
    key = ids.reshape(-1)
    order = np.argsort(key, kind="stable")
    assert np.array_equal(R.order.cpu().numpy(), order)
    off = R.offsets.cpu().numpy()
    assert off[0] == 0 and off[-1] == T and (np.diff(off) >= 0).all()
    assert np.array_equal(off[np.sort(key)], np.searchsorted(np.sort(key), np.sort(key), side="left"))


@pytest.mark.parametrize("n_keys", [4, 5000])
def test_route_extremes(n_keys):
    """No tokens, every choice dropped, one key for all, ids in descending order, ids past
    the keys (dropped, and named in the error word), rows of a wider array."""
    torch = need_gpu()
    import sparse_dense_matrix_spmm_gb300 as spmm
    spmm.last_device_error()
    R = _build(np.zeros((0, 3), np.int64), n_keys)
    assert R.order.numel() == 0 and not R.offsets.cpu().numpy().any() and R.offsets.numel() == n_keys + 1
    for ids in (np.full((70, 2), -7), np.full((9000, 2), n_keys - 1), (np.arange(2000)[::-1] % n_keys).reshape(-1, 1)):
        _same_route(_build(ids, n_keys), ids, n_keys)
    assert spmm.last_device_error() == 0
    ids = _ids(500, 2, n_keys, 1)
    ids[3, 1], ids[77, 0] = n_keys, 1 << 40
    _same_route(_build(ids, n_keys), ids, n_keys)
    assert spmm.last_device_error() == spmm._lib.DEVERR_INDEX
    wide = torch.from_numpy(_ids(321, 7, n_keys, 2, 0.1)).cuda()
    _same_route(spmm.spmm_build_route(wide[:, 2:5], n_keys), wide[:, 2:5].cpu().numpy(), n_keys)
    _same_route(spmm.spmm_build_route(wide[:, 3], n_keys), wide[:, 3].cpu().numpy(), n_keys)
    flat = wide[:, 0].contiguous()
    _same_route(spmm.spmm_build_route(flat, n_keys), flat.cpu().numpy(), n_keys)


SHAPES = [(1, 1, 3, 8), (1, 8, 16, 4096), (19, 2, 3, 7), (64, 3, 5, 1), (257, 4, 31, 3584), (130, 9, 12, 520),
          (33, 5, 600, 2051), (40, 17, 20, 8200)]


@pytest.mark.parametrize("dtype", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("T,k,E,H", SHAPES)
@pytest.mark.parametrize("drop,pad", [(0.0, 0), (0.3, 8), (0.3, 3)])
def test_dispatch_copies_rows(dtype, T, k, E, H, drop, pad):
    torch = need_gpu()
    import sparse_dense_matrix_spmm_gb300 as spmm
    ids = _ids(T, k, E, T * k + H, drop)
    R = _build(ids, E)
    x = matrix((T, H), dtype, 5, pitch=H + pad if pad else None)
    x[0, 0], x[-1, -1] = float("inf"), float("nan")
    out = torch.full((T * k, H + pad), 7.0, dtype=DT[dtype], device="cuda")
    xs = spmm.spmm_dispatch(R, x, out[:, :H])
    order, _, offsets = route(ids, E)
    kept = offsets[-1]
    want = torch.zeros((T * k, H), dtype=DT[dtype])
    want[:kept] = x.cpu()[torch.from_numpy(order[:kept] // k)]
    bits = torch.int32 if dtype == "f32" else torch.int16
    assert torch.equal(xs.cpu().contiguous().view(bits), want.view(bits))
    if pad:
        assert (out[:, H:] == 7.0).all()


@pytest.mark.parametrize("dtype", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("T,k,E,H", SHAPES)
@pytest.mark.parametrize("drop,pad", [(0.0, 0), (0.3, 8), (0.3, 3)])
def test_combine_and_gradients(dtype, T, k, E, H, drop, pad):
    """y, dys, dw and dx against the formulas; rows past the kept places hold NaN and must not count."""
    torch = need_gpu()
    import sparse_dense_matrix_spmm_gb300 as spmm
    ids = _ids(T, k, E, T * k + H + 1, drop)
    if drop:
        ids[T // 2] = -1  # a token with nothing
    R = _build(ids, E)
    order, pos, offsets = route(ids, E)
    kept = offsets[-1]
    ys = matrix((T * k, H), dtype, 6, pitch=H + pad if pad else None)
    ys[kept:] = float("nan")
    w = torch.rand((T, k), generator=torch.Generator().manual_seed(7)).cuda()
    dy = matrix((T, H), dtype, 8, pitch=H + pad if pad else None)
    Y, W, D = f64(ys), f64(w), f64(dy)
    ref, mag, dx, dxm = (np.zeros((T, H)) for _ in range(4))
    dys, dw, dwm = np.zeros((T * k, H)), np.zeros((T, k)), np.zeros((T, k))
    for t in range(T):
        for j in range(k):
            p = pos[t, j]
            if p < 0:
                continue
            ref[t] += W[t, j] * Y[p]
            mag[t] += np.abs(W[t, j] * Y[p])
            dx[t] += Y[p]
            dxm[t] += np.abs(Y[p])
            dys[p] = W[t, j] * D[t]
            dw[t, j] = D[t] @ Y[p]
            dwm[t, j] = np.abs(D[t]) @ np.abs(Y[p])
    check(spmm.spmm_combine(R, ys, w), ref, mag, k, dtype, "y")
    check(spmm.spmm_dispatch_grad(R, ys), dx, dxm, k, dtype, "dx")
    buf = torch.full((T * k, H + pad), 7.0, dtype=DT[dtype], device="cuda")
    got_dys, got_dw = spmm.spmm_combine_grad(R, dy, ys, w, out=buf[:, :H])
    check(got_dys, dys, np.abs(dys), 0, dtype, "dys")
    check(got_dw, dw, dwm, H, "f32", "dw")
    if pad:
        assert (buf[:, H:] == 7.0).all()
    again = spmm.spmm_combine_grad(R, dy, ys, w)
    assert torch.equal(again[0].view(torch.uint8), got_dys.contiguous().view(torch.uint8))
    assert torch.equal(again[1], got_dw)


def test_combine_gradient_against_differences():
    """Central differences of L = sum(y * g) in w and ys (fp32 rows): y is linear in each, so the
    quotient is exact up to rounding: |L| is below 2^7 here, fp32 outputs carry 2^-23 of their terms."""
    torch = need_gpu()
    import sparse_dense_matrix_spmm_gb300 as spmm
    T, k, E, H = 6, 3, 4, 20
    ids = _ids(T, k, E, 3, 0.2)
    R = _build(ids, E)
    ys, g = matrix((T * k, H), "f32", 1), matrix((T, H), "f32", 2)
    w = torch.rand((T, k), generator=torch.Generator().manual_seed(3)).cuda()
    dys, dw = spmm.spmm_combine_grad(R, g, ys, w)

    def loss(ys, w):
        return float((f64(spmm.spmm_combine(R, ys, w)) * f64(g)).sum())

    tol = T * H * k * 2.0 ** -23 * 16
    for i in range(T * k):
        for t, grad in ((w.view(-1), dw.view(-1)), (ys[i], dys[i])):
            at = i if t.numel() == T * k else i % H
            old = t[at].item()
            t[at] = old + 0.5
            up = loss(ys, w)
            t[at] = old - 0.5
            down = loss(ys, w)
            t[at] = old
            assert abs((up - down) - grad[at].item()) <= tol


def test_side_stream_and_empty():
    """On a stream of its own while the current one is busy; shapes with nothing to write."""
    torch = need_gpu()
    import sparse_dense_matrix_spmm_gb300 as spmm
    s = torch.cuda.Stream()
    ids = _ids(300, 2, 700, 9)
    x = matrix((300, 256), "bf16", 3)
    d = torch.from_numpy(ids).cuda()
    torch.cuda.synchronize()
    R = spmm.spmm_build_route(d, 700, stream=s)
    xs = spmm.spmm_dispatch(R, x, stream=s)
    y = spmm.spmm_combine(R, xs, stream=s)
    s.synchronize()
    _same_route(R, ids, 700)
    assert torch.equal(y.float(), (x.float() * 2).to(torch.bfloat16).float())
    E = _build(np.zeros((0, 2), np.int64), 4)
    assert spmm.spmm_dispatch(E, x[:0]).shape == (0, 256)
    assert spmm.spmm_combine(E, x[:0]).shape == (0, 256)
    R = _build(ids[:4], 700)
    assert spmm.spmm_dispatch(R, x[:4, :0]).shape == (8, 0)
    torch.cuda.synchronize()
    assert spmm.last_device_error() == 0


def test_refusals():
    torch = need_gpu()
    import sparse_dense_matrix_spmm_gb300 as spmm
    R = _build(_ids(10, 2, 4, 1), 4)
    x, ys, w = matrix((10, 64), "bf16", 1), matrix((20, 64), "bf16", 2), torch.ones((10, 2), device="cuda")
    with pytest.raises(TypeError):
        spmm.spmm_build_route(x, 4)                                   # ids are no integers
    with pytest.raises(ValueError):
        spmm.spmm_build_route(torch.zeros((2, 3, 4), dtype=torch.int64, device="cuda"), 4)
    with pytest.raises(ValueError):
        spmm.spmm_build_route(torch.zeros((6, 4), dtype=torch.int64, device="cuda").t(), 4)
    with pytest.raises(ValueError):
        spmm.spmm_build_route(torch.zeros(4, dtype=torch.int64), 4)    # on the host
    with pytest.raises(spmm.SpmmError, match="SHAPE"):
        spmm.spmm_build_route(torch.zeros(4, dtype=torch.int64, device="cuda"), 0)
    with pytest.raises(spmm.SpmmError, match="WORKSPACE"):
        spmm.spmm_build_route(torch.zeros(4, dtype=torch.int64, device="cuda"), 600,
                              workspace=torch.empty(8, dtype=torch.uint8, device="cuda"))
    with pytest.raises(ValueError):
        spmm.spmm_dispatch(R, x[:9])                                   # rows
    with pytest.raises(TypeError):
        spmm.spmm_dispatch(R, x.to(torch.float64))
    with pytest.raises(ValueError):
        spmm.spmm_dispatch(R, x.t().contiguous().t())                  # columns contiguous
    with pytest.raises(TypeError):
        spmm.spmm_dispatch(R, x, out=torch.empty((20, 64), device="cuda"))
    with pytest.raises(spmm.SpmmError, match="SHAPE"):
        spmm.spmm_dispatch(R, x[:1].expand(10, 64))                    # a row pitch of 0
    with pytest.raises(TypeError):
        spmm.spmm_combine(R, ys, w.to(torch.bfloat16))
    with pytest.raises(ValueError):
        spmm.spmm_combine(R, ys, w[:, :1])
    with pytest.raises(ValueError):
        spmm.spmm_combine(R, ys, w.t().contiguous())                   # k x T
    with pytest.raises(ValueError):
        spmm.spmm_combine(R, ys, out=x[:9])
    with pytest.raises(TypeError):
        spmm.spmm_combine_grad(R, x, ys.to(torch.float16), w)
