"""Every width in which the row operators move their rows, against plain 64-bit
definitions.  Rows move in the widest pieces of 16, 8, 4 or 2 bytes that base, pitch
and length of every operand allow, so each case names what narrows it."""
import numpy as np
import pytest

from tests.gpu_util import need_gpu
from tests.onehot_util import DT, check, f64, matrix, route

pytestmark = pytest.mark.gpu

# row length, pitch of the inputs, pitch of the outputs, first column.  In 16-bit values: 4 per move by the
# length (4, 12, 100, 4100), 2 (2, 6, 4098), narrowed by a pitch or a base at an even or full length; in 32 bits
# the lengths 2, 6, 2050 move by 2 and the narrowed ones by 2 or 1.
WIDTHS = [(4, 4, 4, 0), (12, 12, 12, 0), (100, 100, 100, 0), (4100, 4100, 4100, 0), (2, 2, 2, 0), (6, 6, 6, 0),
          (2050, 2050, 2050, 0), (4098, 4098, 4098, 0), (64, 68, 64, 0), (64, 64, 66, 0), (520, 522, 528, 0),
          (520, 528, 528, 4), (264, 272, 272, 2), (264, 272, 272, 1), (96, 97, 96, 0),
          (96, 96, 97, 0)]


def _view(shape, dtype, seed, pitch, first):
    """A matrix of normal values whose rows start `first` columns into rows of `pitch` and more."""
    return matrix((shape[0], first + shape[1]), dtype, seed, pitch=max(pitch, first + shape[1]))[:, first:]


def _out(torch, shape, dtype, pitch, first):
    buf = torch.full((shape[0], max(pitch, first + shape[1])), 7.0, dtype=DT[dtype], device="cuda")
    return buf, buf[:, first:first + shape[1]]


def _untouched(buf, view, first):
    return bool((buf[:, :first] == 7.0).all() and (buf[:, first + view.shape[1]:] == 7.0).all())


@pytest.mark.parametrize("dtype", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("H,pitch,out_pitch,first", WIDTHS)
@pytest.mark.parametrize("k", [3, 6])
def test_dispatch_combine_and_gradients(dtype, H, pitch, out_pitch, first, k):
    """Three choices, and six (more than the rows in flight together)."""
    torch = need_gpu()
    import sparse_dense_matrix_spmm_gb300 as spmm
    T, E = 37, 9
    rng = np.random.default_rng(H + pitch + k)
    ids = np.where(rng.random((T, k)) < 0.2, -1, rng.integers(0, E, (T, k)))
    ids[4] = -1
    R = spmm.spmm_build_route(torch.from_numpy(ids).cuda(), E)
    order, pos, offsets = route(ids, E)
    kept = int(offsets[-1])
    x = _view((T, H), dtype, 1, pitch, first)
    ys = _view((T * k, H), dtype, 2, pitch, first)
    dy = _view((T, H), dtype, 3, pitch, first)
    ys[kept:] = float("nan")
    w = torch.rand((T, k), generator=torch.Generator().manual_seed(5)).cuda()

    buf, out = _out(torch, (T * k, H), dtype, out_pitch, first)
    spmm.spmm_dispatch(R, x, out=out)
    want = torch.zeros((T * k, H), dtype=DT[dtype])
    want[:kept] = x.cpu()[torch.from_numpy(order[:kept] // k)]
    assert torch.equal(out.cpu(), want) and _untouched(buf, out, first)

    Y, W, D, live = f64(ys), f64(w), f64(dy), pos >= 0
    rows = np.where(live[:, :, None], Y[np.maximum(pos, 0)], 0.0)   # T x k x H
    terms = W[:, :, None] * rows
    buf, out = _out(torch, (T, H), dtype, out_pitch, first)
    check(spmm.spmm_combine(R, ys, w, out=out), terms.sum(1), np.abs(terms).sum(1), k, dtype, "y")
    assert _untouched(buf, out, first)
    check(spmm.spmm_dispatch_grad(R, ys), rows.sum(1), np.abs(rows).sum(1), k, dtype, "dx")

    dys = np.zeros((T * k, H))
    dys[:kept] = D[order[:kept] // k] * W.reshape(-1)[order[:kept], None]
    dots = np.where(live, (D[:, None, :] * rows).sum(2), 0.0)
    buf, out = _out(torch, (T * k, H), dtype, out_pitch, first)
    got, dw = spmm.spmm_combine_grad(R, dy, ys, w, out=out)
    check(got, dys, np.abs(dys), 0, dtype, "dys")
    check(dw, dots, np.abs(D[:, None, :] * rows).sum(2), H, "f32", "dw")
    assert _untouched(buf, out, first)


@pytest.mark.parametrize("dtype", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("H,pitch,out_pitch,first", WIDTHS)
def test_embed(dtype, H, pitch, out_pitch, first):
    torch = need_gpu()
    import sparse_dense_matrix_spmm_gb300 as spmm
    T, V = 41, 23
    rng = np.random.default_rng(H + pitch)
    ids = np.where(rng.random(T) < 0.2, -1, rng.integers(0, V, T))
    table = _view((V, H), dtype, 4, pitch, first)
    buf, out = _out(torch, (T, H), dtype, out_pitch, first)
    ref = np.where(ids[:, None] >= 0, f64(table)[np.maximum(ids, 0)] * 0.75, 0.0)
    check(spmm.spmm_embed(table, torch.from_numpy(ids).cuda(), 0.75, out=out), ref, np.abs(ref), 0, dtype, "embed")
    assert _untouched(buf, out, first)


@pytest.mark.parametrize("dtype,out_dtype", [("bf16", "bf16"), ("bf16", "f32"), ("f16", "f16"), ("f16", "f32"),
                                             ("f32", "f32")])
@pytest.mark.parametrize("H,pitch,out_pitch,first", WIDTHS)
def test_embed_grad(dtype, out_dtype, H, pitch, out_pitch, first):
    """Rows with one token and with runs of 2900: 46 partial sums, past the 16 that one thread adds."""
    torch = need_gpu()
    import sparse_dense_matrix_spmm_gb300 as spmm
    T, V = 3001, 50
    rng = np.random.default_rng(H + pitch + 1)
    ids = np.where(np.arange(T) % 30 == 7, rng.integers(-1, V, T), 17)
    dy = _view((T, H), dtype, 6, pitch, first)
    R = spmm.spmm_build_route(torch.from_numpy(ids).cuda(), V)
    D = f64(dy)
    ref, mag = np.zeros((V, H)), np.zeros((V, H))
    for v in range(V):
        ref[v], mag[v] = D[ids == v].sum(0) * 0.5, np.abs(D[ids == v]).sum(0) * 0.5
    buf, out = _out(torch, (V, H), out_dtype, out_pitch, first)
    check(spmm.spmm_embed_grad(R, dy, 0.5, out=out), ref, mag, T, out_dtype, "dtable")
    assert _untouched(buf, out, first)
    base = matrix((V, H), out_dtype, 7)
    acc = base.clone()
    spmm.spmm_embed_grad(R, dy, 0.5, out=acc, accumulate=True)
    check(acc, f64(base) + ref, np.abs(f64(base)) + mag, T + 1, out_dtype, "accumulated")
