"""The router and its gradient against the definition in 64 bits."""
import numpy as np
import pytest

from tests.gpu_util import need_gpu
from tests.gated_util import near
from tests.onehot_util import DT, f64, matrix

pytestmark = pytest.mark.gpu

SIZES = [(1, 1, 1), (1, 5, 5), (3, 31, 2), (40, 32, 8), (41, 33, 7), (64, 60, 6), (17, 64, 1), (130, 65, 4), (33, 128, 8),
         (9, 200, 32), (300, 256, 8), (5, 511, 16), (6, 512, 3), (7, 1000, 10), (4, 1024, 32), (2, 40, 32)]


def _reference(x, k, renorm):
    """ids, w, p (the softmax that the gradient uses) of logits without NaN and +infinity, by sorting."""
    T, E = x.shape
    ids, w, p = np.full((T, k), -1, np.int64), np.zeros((T, k)), np.zeros((T, E))
    for t in range(T):
        order = sorted((e for e in range(E) if x[t, e] > -np.inf), key=lambda e: (-x[t, e], e))
        chosen = order[:k]
        if not chosen:
            continue
        over = chosen if renorm else order
        z = np.exp(x[t, over] - x[t, over].max())
        p[t, over] = z / z.sum()
        ids[t, :len(chosen)] = chosen
        w[t, :len(chosen)] = p[t, chosen]
    return ids, w, p


def _weight_error(x, w):
    """Relative: an exponent's difference is rounded (2^-24 of at most its own size), expf and the division take a
    few units, the sum one per term."""
    spread = np.where(np.isfinite(x), x, np.nan)
    spread = np.nan_to_num(np.nanmax(spread, axis=1) - np.nanmin(spread, axis=1)) if x.size else np.zeros(len(x))
    return w * (x.shape[1] + 8 + spread[:, None]) * 2.0 ** -22


def _check(torch, spmm, x, k, renorm, idt, seed=0):
    X = f64(x)
    T, E = X.shape
    ids, w = spmm.spmm_topk(x, k, renorm=renorm, id_dtype=idt)
    rids, rw, p = _reference(X, k, renorm)
    assert ids.dtype == idt and w.dtype == torch.float32
    assert np.array_equal(ids.cpu().numpy(), rids)
    with np.errstate(all="ignore"):
        near(w, rw, _weight_error(X, rw), "f32", "w")
    dw = torch.randn(T, k, generator=torch.Generator().manual_seed(seed)).cuda()
    dw[ids < 0] = float("nan")  # a dropped choice's gradient is not read
    got = spmm.spmm_topk_grad(x, ids, w, dw, renorm=renorm)
    name = {torch.bfloat16: "bf16", torch.float16: "f16", torch.float32: "f32"}[x.dtype]
    D = np.nan_to_num(f64(dw))
    ref, mag = np.zeros((T, E)), np.zeros((T, E))
    for t in range(T):
        on = rids[t] >= 0
        dot, adot = (rw[t] * D[t])[on].sum(), np.abs(rw[t] * D[t])[on].sum()
        ref[t], mag[t] = -p[t] * dot, p[t] * adot
        ref[t, rids[t][on]] += (rw[t] * D[t])[on]
        mag[t, rids[t][on]] += np.abs(rw[t] * D[t])[on]
    with np.errstate(all="ignore"):
        err = 3 * mag * np.nan_to_num(_weight_error(X, np.ones((T, 1))))
    near(got, ref, err, name, "dlogits")
    return ids, w


@pytest.mark.parametrize("dtype", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("renorm", [True, False])
@pytest.mark.parametrize("T,E,k", SIZES)
def test_against_sorting(dtype, renorm, T, E, k):
    torch = need_gpu()
    import sparse_dense_matrix_spmm_gb300 as spmm
    _check(torch, spmm, matrix((T, E), dtype, T + E, 2.0), k, renorm, torch.int64 if T % 2 else torch.int32)
    assert spmm.last_device_error() == 0


@pytest.mark.parametrize("renorm", [True, False])
@pytest.mark.parametrize("E", [6, 60, 300])
def test_ties_masks_and_extremes(renorm, E):
    """Equal logits, both zeros, logits of -infinity and of the type's lowest value, tokens with few or no experts left."""
    torch = need_gpu()
    import sparse_dense_matrix_spmm_gb300 as spmm
    g = torch.Generator().manual_seed(E)
    x = torch.randint(-2, 3, (50, E), generator=g).float()
    x[1] = 0.0
    x[1, ::2] = -0.0
    x[2:20].masked_fill_(torch.rand(18, E, generator=g) < 0.7, -float("inf"))
    x[20] = -float("inf")
    x[21] = -float("inf")
    x[21, E - 1] = -5.0
    x[22] = torch.finfo(torch.float32).min
    x[23, : E // 2] = torch.finfo(torch.float32).min
    x[24] = 88.0
    x[25, 3] = 3e38
    for t in (x.cuda(), x[:25].to(torch.bfloat16).cuda()):
        ids, w = _check(torch, spmm, t, 5, renorm, torch.int64)
        assert (ids[20] == -1).all() and (w[20] == 0).all()


@pytest.mark.parametrize("renorm", [True, False])
def test_nan_and_infinity(renorm):
    """NaN ranks first, then +infinity; both make the token's weights NaN, and no other token's."""
    torch = need_gpu()
    import sparse_dense_matrix_spmm_gb300 as spmm
    x = matrix((6, 50), "f32", 1)
    clean = spmm.spmm_topk(x, 4, renorm=renorm)
    x[1, 7], x[1, 9] = float("inf"), float("nan")
    x[3, 30] = float("inf")
    x[4, 12] = -float("nan")
    ids, w = spmm.spmm_topk(x, 4, renorm=renorm)
    assert ids[1, 0] == 9 and ids[1, 1] == 7 and ids[3, 0] == 30 and ids[4, 0] == 12
    assert w[[1, 4]].isnan().all() and w[3, 0].isnan()
    for t in (0, 2, 5):
        assert torch.equal(ids[t], clean[0][t]) and torch.equal(w[t], clean[1][t])
    d = spmm.spmm_topk_grad(x, ids, w, torch.ones_like(w), renorm=renorm)
    assert d[1, 9].isnan() and not d[[0, 2, 5]].isnan().any()


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_pitches(dtype):
    torch = need_gpu()
    import sparse_dense_matrix_spmm_gb300 as spmm
    x = matrix((21, 70), dtype, 2, pitch=77)
    ids, w = _check(torch, spmm, x, 4, False, torch.int32)
    wide = torch.full((21, 75), 7.0, dtype=DT[dtype], device="cuda")
    dw = torch.ones_like(w)
    got = spmm.spmm_topk_grad(x, ids, w, dw, renorm=False, out=wide[:, 3:73])
    assert torch.equal(got, spmm.spmm_topk_grad(x, ids, w, dw, renorm=False))
    assert (wide[:, :3] == 7).all() and (wide[:, 73:] == 7).all()


@pytest.mark.parametrize("renorm", [True, False])
def test_gradient_of_given_ids(renorm):
    """Ids of the caller's own: the same one twice is added up, one past the experts is dropped and flagged."""
    torch = need_gpu()
    import sparse_dense_matrix_spmm_gb300 as spmm
    x = matrix((3, 9), "f32", 8)
    p = torch.softmax(x.double(), 1).cpu()
    ids = torch.tensor([[2, 2, 5], [1, 9, -7], [8, 0, 8]]).cuda()
    w = torch.where(ids.cpu() % 10 < 9, p.gather(1, ids.cpu().clamp(0, 8)), 0.0).float().cuda()
    dw = matrix((3, 3), "f32", 9)
    got = spmm.spmm_topk_grad(x, ids, w, dw, renorm=renorm)
    assert spmm.last_device_error() == 2
    W, D, I = f64(w), f64(dw), ids.cpu().numpy()
    ref = np.zeros((3, 9))
    for t in range(3):
        on = [j for j in range(3) if 0 <= I[t, j] < 9]
        dot = sum(W[t, j] * D[t, j] for j in on)
        q = np.zeros(9) if renorm else p[t].numpy()
        for j in on:
            ref[t, I[t, j]] += W[t, j] * D[t, j]
            if renorm:
                q[I[t, j]] += W[t, j]
        ref[t] -= q * dot
    near(got, ref, np.full((3, 9), 64 * 2.0 ** -22), "f32", "dlogits")


@pytest.mark.parametrize("renorm", [True, False])
def test_gradient_against_differences(renorm):
    """Central differences of the definition, where a small step changes no choice."""
    torch = need_gpu()
    import sparse_dense_matrix_spmm_gb300 as spmm
    g = torch.Generator().manual_seed(3)
    x = torch.stack([torch.randperm(24, generator=g) for _ in range(8)]).float() / 8  # gaps of 1/8
    k, h = 5, 1e-3
    ids, w = spmm.spmm_topk(x.cuda(), k, renorm=renorm)
    dw = matrix((8, k), "f32", 4)
    got = f64(spmm.spmm_topk_grad(x.cuda(), ids, w, dw, renorm=renorm))
    X, D = x.double().numpy(), f64(dw)
    for e in range(24):
        up, down = X.copy(), X.copy()
        up[:, e] += h
        down[:, e] -= h
        slope = ((_reference(up, k, renorm)[1] - _reference(down, k, renorm)[1]) / (2 * h) * D).sum(1)
        # the difference's own error is a third derivative, below 1, times h^2 / 6 per term
        assert (np.abs(got[:, e] - slope) <= np.abs(D).sum(1) * (h * h + 64 * 2.0 ** -22)).all()


def test_many_tokens_and_none():
    torch = need_gpu()
    import sparse_dense_matrix_spmm_gb300 as spmm
    x = matrix((70001, 16), "bf16", 6)
    ids, w = spmm.spmm_topk(x, 2)
    top = torch.sort(x.float(), dim=1, descending=True, stable=True)
    assert torch.equal(ids, top.indices[:, :2])
    assert (w.sum(1) - 1).abs().max() < 1e-6
    ids, w = spmm.spmm_topk(x[:0], 2)
    assert ids.shape == w.shape == (0, 2)
    assert spmm.spmm_topk_grad(x[:0], ids, w, w).shape == (0, 16)
