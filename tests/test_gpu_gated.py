"""The experts' gated block, what it keeps for the way back, and its gradients, against 64 bits."""
import numpy as np
import pytest

from tests.gated_util import ACTS, act, act_error, act_slope, held, near
from tests.gpu_util import need_gpu
from tests.onehot_util import DT, check, f64, matrix, route

pytestmark = pytest.mark.gpu

# (rows per expert, dropped choices, N, K): one row, none, ragged counts around the tiles' edges, few rows in all and
# many, features around 64, 128 and 256
CASES = [
    ([1], 0, 16, 8), ([0, 1, 0], 2, 32, 24), ([0, 0], 5, 64, 64), ([1] * 8, 0, 144, 264), ([5, 0, 9], 1, 48, 520),
    ([16], 0, 80, 72), ([17], 3, 16, 136), ([15, 16, 17, 0, 31, 33], 3, 128, 64), ([63, 64, 65, 1], 0, 112, 200),
    ([127, 128, 129], 2, 256, 128), ([255, 3, 257, 300], 1, 272, 328), ([600, 0, 0, 37], 0, 528, 1000),
    ([5, 2, 0, 7, 1, 3, 6, 4] * 4, 9, 384, 512), ([1030], 0, 768, 520), ([0, 40], 0, 64, 2056), ([0] * 40 + [1, 30], 0, 32, 64),
    ([300] + [0] * 30 + [2] * 9, 1, 208, 200), ([2, 1], 13, 1040, 1032),
]


def _route(counts, dropped, seed):
    import torch

    import sparse_dense_matrix_spmm_gb300 as spmm
    ids = np.concatenate([np.full(c, e) for e, c in enumerate(counts)] + [np.full(dropped, -1)]).astype(np.int64)
    ids = np.random.default_rng(seed).permutation(ids)
    return spmm.spmm_build_route(torch.from_numpy(ids).cuda(), len(counts)), route(ids, len(counts))[2]


def _sums(X, V, offsets):
    """[g u] of every kept row in 64 bits, and the magnitude of its terms."""
    n = X.shape[0]
    gu, mag = np.zeros((n, V.shape[1])), np.zeros((n, V.shape[1]))
    for e in range(V.shape[0]):
        a, b = offsets[e], offsets[e + 1]
        gu[a:b], mag[a:b] = X[a:b] @ V[e].T, np.abs(X[a:b]) @ np.abs(V[e]).T
    return gu, mag


def _check_h(got, gu, mag, K, N, name, dtype):
    err = (K + 2) * 2.0 ** -23 * mag
    g, u, eg, eu = gu[:, :N], gu[:, N:], err[:, :N], err[:, N:]
    f = act(g, name)
    # |act'| < 1.2 for all three
    fe = 1.2 * eg + np.abs(f) * act_error(g)
    near(got, f * u, fe * (np.abs(u) + eu) + np.abs(f) * eu + 2.0 ** -23 * np.abs(f * u), dtype, "h")


def _check_packed(P, gu, mag, K):
    """The kept integers are the definition's for sums within their error of the exact ones."""
    q, s = P.q.cpu().numpy().astype(np.float64), P.scale.cpu().numpy()
    err = (K + 2) * 2.0 ** -23 * mag
    e = np.repeat(s.astype(np.float64) - 127, 16, axis=1)
    unit = 2.0 ** e
    assert (np.abs(q) <= 127).all() and (s >= 1).all() and (s <= 248).all()
    assert (np.abs(q * unit - gu) <= unit / 2 + err).all()
    v, ve = np.abs(gu).reshape(len(gu), -1, 16), err.reshape(len(gu), -1, 16)
    small = 2.0 ** (s.astype(np.float64) - 127)
    assert ((v - ve).max(2) <= 127.5 * small).all()  # it rounds to 127 at most
    assert (((v + ve).max(2) >= 127.5 * small / 2) | (s == 1)).all()  # and the next smaller exponent would not do


@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("pad", [0, 8])
@pytest.mark.parametrize("i", range(len(CASES)))
def test_forward(dtype, pad, i):
    """h, and the kept [g u] in both forms; rows of dropped choices hold NaN on the way in and zeros on the way out."""
    torch = need_gpu()
    import sparse_dense_matrix_spmm_gb300 as spmm
    counts, dropped, N, K = CASES[i]
    name = ACTS[(i + pad) % 3]
    R, offsets = _route(counts, dropped, N + K)
    n, kept, E = R.n_rows, int(offsets[-1]), len(counts)
    xs = matrix((n, K), dtype, 1, pitch=K + pad)
    W = matrix((E, 2 * N, K), dtype, 3, 1.5 * K ** -0.5, pitch=K + pad)
    xs[kept:] = float("nan")
    X, V = f64(xs), f64(W)
    X[kept:] = 0
    gu, mag = _sums(X, V, offsets)
    buf = torch.full((n, N + 8), 7.0, dtype=DT[dtype], device="cuda")
    h = spmm.spmm_experts_gated(R, xs, W, act=name, out=buf[:, :N])
    _check_h(h, gu, mag, K, N, name, dtype)
    assert (buf[:, N:] == 7.0).all() and not h[kept:].any()
    h16, kept16 = spmm.spmm_experts_gated(R, xs, W, act=name, save="rows")
    check(kept16, gu, mag, K, dtype, "gu")
    h8, kept8 = spmm.spmm_experts_gated(R, xs, W, act=name, save="packed")
    _check_packed(kept8, gu, mag, K)
    assert torch.equal(h16, h)
    _check_h(h8, gu, mag, K, N, name, dtype)
    assert dtype == "f16" or torch.equal(h8, h)  # fp16 sums kept in 8 bits are formed in halves
    assert not kept16[kept:].any() and not kept8.q[kept:].any() and (kept8.scale[kept:] == 1).all()
    torch.cuda.synchronize()
    assert spmm.last_device_error() == 0


@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("form", ["rows", "packed"])
@pytest.mark.parametrize("name", ACTS)
@pytest.mark.parametrize("counts,dropped,N,pad", [([1], 0, 16, 0), ([3, 0, 4], 5, 48, 8), ([40, 61], 2, 272, 0),
                                                  ([7, 2], 0, 2064, 8), ([0, 0], 3, 32, 0)])
def test_gradient_of_the_activation(dtype, form, name, counts, dropped, N, pad):
    """dgu and h from the kept [g u] as it is held, slopes by differences of the activation's definition."""
    torch = need_gpu()
    import sparse_dense_matrix_spmm_gb300 as spmm
    R, offsets = _route(counts, dropped, N)
    n, kept = R.n_rows, int(offsets[-1])
    dh = matrix((n, N), dtype, 4, pitch=N + pad)
    gu = matrix((n, 2 * N), dtype, 5, 2.0, pitch=2 * N + pad)
    gu[:kept, :8] = torch.tensor([0.0, -0.0, 1e-3, -1e-3, 9.0, -9.0, 20.0, -20.0], device="cuda").to(DT[dtype])
    saved = gu if form == "rows" else spmm.spmm_pack_rows(gu)
    V = f64(gu) if form == "rows" else held(saved.q.cpu().numpy(), saved.scale.cpu().numpy())
    dh[kept:], gu[kept:] = float("nan"), float("nan")
    if form == "packed":
        saved.scale[kept:] = 255
    D = f64(dh)
    D[kept:], V[kept:] = 0, 0
    wide = torch.full((n, 2 * N + 8), 7.0, dtype=DT[dtype], device="cuda")
    dgu, h = spmm.spmm_gated_grad(R, dh, saved, act=name, with_h=True, out=wide[:, :2 * N])
    g, u = V[:, :N], V[:, N:]
    f, d, e = act(g, name), act_slope(g, name), act_error(g)
    few = 4 * 2.0 ** -23
    near(dgu[:, :N], D * u * d, np.abs(D * u) * (e + few + 1e-9), dtype, "dg")
    near(dgu[:, N:], D * f, np.abs(D * f) * (e + few), dtype, "du")
    near(h, f * u, np.abs(f * u) * (e + few), dtype, "h")
    assert (wide[:, 2 * N:] == 7.0).all() and not dgu[kept:].any() and not h[kept:].any()
    assert torch.equal(spmm.spmm_gated_grad(R, dh, saved, act=name), dgu)


@pytest.mark.parametrize("form", ["rows", "packed"])
def test_all_gradients(form):
    """dgu, dxs and dW together, from a checkpoint of the rows too: the products of what is held."""
    torch = need_gpu()
    import sparse_dense_matrix_spmm_gb300 as spmm
    counts, dropped, N, K = [33, 0, 70, 5], 4, 144, 264
    R, offsets = _route(counts, dropped, 7)
    n, kept = R.n_rows, int(offsets[-1])
    xs, dh = matrix((n, K), "bf16", 1), matrix((n, N), "bf16", 2)
    W = matrix((4, 2 * N, K), "bf16", 3, K ** -0.5)
    xs[kept:], dh[kept:] = 0, 0
    h, gu = spmm.spmm_experts_gated(R, xs, W, act="silu", save=form)
    P = spmm.spmm_pack_rows(xs) if form == "packed" else xs
    X = held(P.q.cpu().numpy(), P.scale.cpu().numpy()) if form == "packed" else f64(xs)
    dgu, dxs, dW = spmm.spmm_experts_gated_grad(R, dh, P, W, gu, act="silu")
    assert torch.equal(dgu, spmm.spmm_gated_grad(R, dh, gu))
    D, V = f64(dgu), f64(W)
    dx, dxm, dw, dwm = np.zeros((n, K)), np.zeros((n, K)), np.zeros(V.shape), np.zeros(V.shape)
    for e in range(4):
        a, b = offsets[e], offsets[e + 1]
        dx[a:b], dxm[a:b] = D[a:b] @ V[e], np.abs(D[a:b]) @ np.abs(V[e])
        dw[e], dwm[e] = D[a:b].T @ X[a:b], np.abs(D[a:b]).T @ np.abs(X[a:b])
    check(dxs, dx, dxm, 2 * N, "bf16", "dxs")
    check(dW, dw, dwm, max(counts), "bf16", "dW")


@pytest.mark.parametrize("save", [None, "rows", "packed"])
def test_other_experts_do_not_leak(save):
    """Infinities and NaN in one expert's rows and weights stay in its own rows."""
    torch = need_gpu()
    import sparse_dense_matrix_spmm_gb300 as spmm
    counts = [5, 37, 11, 64, 1]
    R, offsets = _route(counts, 0, 1)
    N, K = 208, 136
    xs, W = matrix((R.n_rows, K), "bf16", 1), matrix((5, 2 * N, K), "bf16", 3, K ** -0.5)

    def run():
        r = spmm.spmm_experts_gated(R, xs, W, save=save)
        r = [r] if save is None else list(r)
        return r[:-1] + [r[-1].q, r[-1].scale] if save == "packed" else r

    before = run()
    for e, v in ((1, float("inf")), (3, float("nan"))):
        xs[offsets[e]:offsets[e + 1]], W[e] = v, v
    after = run()
    for x, y in zip(before, after):
        for e in (0, 2, 4):
            assert torch.equal(x[offsets[e]:offsets[e + 1]], y[offsets[e]:offsets[e + 1]])
    assert after[0][offsets[3]:offsets[4]].isnan().all()
    if save == "packed":
        assert (after[2][offsets[1]:offsets[2]] == 255).all() and (after[2][offsets[3]:offsets[4]] == 255).all()
    torch.cuda.synchronize()
    assert spmm.last_device_error() == 0


@pytest.mark.parametrize("save", [None, "rows", "packed"])
def test_large_block_sampled(save):
    """A prompt-sized block (2 x 4096 tokens over 8 experts): sampled rows, and the same bits on every run."""
    torch = need_gpu()
    import sparse_dense_matrix_spmm_gb300 as spmm
    rng = np.random.default_rng(4)
    E, N, K = 8, 1424, 2048
    R = spmm.spmm_build_route(torch.from_numpy(rng.integers(0, E, (4096, 2))).cuda(), E)
    offsets = R.offsets.cpu().numpy()
    xs, W = matrix((8192, K), "bf16", 1), matrix((E, 2 * N, K), "bf16", 3, K ** -0.5)
    r = spmm.spmm_experts_gated(R, xs, W, act="gelu_tanh", save=save)
    h = r if save is None else r[0]
    rows = np.unique(np.concatenate([offsets[:-1], offsets[1:] - 1, rng.integers(0, 8192, 64)]))
    e_of = np.searchsorted(offsets, rows, side="right") - 1
    X, V = f64(xs[torch.from_numpy(rows).cuda()]), f64(W)
    gu = np.stack([V[e] @ x for x, e in zip(X, e_of)])
    mag = np.stack([np.abs(V[e]) @ np.abs(x) for x, e in zip(X, e_of)])
    at = torch.from_numpy(rows).cuda()
    _check_h(h[at], gu, mag, K, N, "gelu_tanh", "bf16")
    again = spmm.spmm_experts_gated(R, xs, W, act="gelu_tanh", save=save)
    if save == "rows":
        check(r[1][at], gu, mag, K, "bf16", "gu")
        assert torch.equal(again[1], r[1])
    if save == "packed":
        P = spmm.Rows8(len(rows), 2 * N, r[1].dtype, r[1].q[at], r[1].scale[at])
        _check_packed(P, gu, mag, K)
        assert torch.equal(again[1].q, r[1].q) and torch.equal(again[1].scale, r[1].scale)
    assert torch.equal(again if save is None else again[0], h)
    assert spmm.last_device_error() == 0


def test_no_tokens():
    torch = need_gpu()
    import sparse_dense_matrix_spmm_gb300 as spmm
    R = spmm.spmm_build_route(torch.zeros(0, 2, dtype=torch.int64, device="cuda"), 3)
    xs, W = torch.empty(0, 64, dtype=torch.bfloat16, device="cuda"), matrix((3, 64, 64), "bf16", 1)
    h, gu = spmm.spmm_experts_gated(R, xs, W, save="packed")
    assert h.shape == (0, 32) and gu.q.shape == (0, 64)
    dgu, dxs, dW = spmm.spmm_experts_gated_grad(R, h, xs, W, gu)
    assert dgu.shape == (0, 64) and dxs.shape == (0, 64) and not dW.any()


@pytest.mark.parametrize("dtype,powers", [("bf16", (-100, -30, 0, 60, 119, 120, 121, 122, 126, 127)), ("f16", (-14, -7, 0, 3, 9, 15))])
@pytest.mark.parametrize("n", [10, 80, 300])
def test_packed_sums_exactly(dtype, powers, n):
    """Sums that are exact (one product each): the kept integers are the definition's bit for bit, ties, sums next to the
    largest fp32 and infinite ones among them, on CUDA cores and on the tensor cores."""
    torch = need_gpu()
    import sparse_dense_matrix_spmm_gb300 as spmm
    from tests.gated_util import packed
    rng = np.random.default_rng(n)
    N, K = 80, 16
    R = spmm.spmm_build_route(torch.zeros(n, dtype=torch.int64, device="cuda"), 1)
    xs, W = torch.zeros(n, K, dtype=torch.float64), torch.zeros(1, 2 * N, K, dtype=torch.float64)
    xs[:, 3] = torch.from_numpy(2.0 ** rng.choice(powers, n))
    W[0, :, 3] = torch.from_numpy(rng.integers(-255, 256, 2 * N) * rng.choice([0.5, 0.25, 1.0], 2 * N))
    W[0, 16:32] = 0
    W[0, 48:64, 3] = torch.arange(16) + 0.5
    W[0, 63, 3] = 127.0  # the unit is 1 at power 0: the others are ties
    with np.errstate(over="ignore"):
        g = (f64(xs) @ f64(W[0]).T).astype(np.float32).astype(np.float64)
    xs, W = xs.to(DT[dtype]).cuda(), W.to(DT[dtype]).cuda()
    q, scale = packed(g)
    _, P = spmm.spmm_experts_gated(R, xs, W, save="packed")
    assert np.array_equal(P.scale.cpu().numpy(), scale) and np.array_equal(P.q.cpu().numpy(), q)
    if dtype == "bf16":
        assert (scale == 255).any() and (scale == 248).any()
    assert spmm.last_device_error() == 0
