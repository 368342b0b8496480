"""The experts' products and their gradients against plain 64-bit products per expert."""
import numpy as np
import pytest

from tests.gpu_util import need_gpu
from tests.onehot_util import DT, check, f64, matrix, route

pytestmark = pytest.mark.gpu

# (tokens per expert, dropped choices, N, K): one token, no token, ragged counts around tile
# edges, odd multiples of 8, sizes past one tile in every direction
CASES = [
    ([1], 0, 8, 8), ([0, 1, 0], 0, 16, 24), ([1, 1, 1, 1, 1, 1, 1, 1], 0, 136, 264), ([0, 0, 0], 5, 64, 64),
    ([15, 16, 17, 0, 31, 33], 3, 128, 64), ([63, 64, 65, 1], 0, 72, 200), ([127, 128, 129], 2, 256, 128),
    ([255, 3, 257, 300], 1, 264, 328), ([600, 0, 0, 37], 0, 520, 1000), ([5, 2, 0, 7, 1, 3, 6, 4] * 4, 9, 384, 512),
    ([1030], 0, 1536, 520), ([5, 2, 0, 7], 2, 200, 584), ([0, 16], 0, 40, 2056), ([0] * 40 + [1, 3], 0, 24, 64),
    ([300] + [0] * 30 + [2] * 9, 1, 264, 200),
]


def _case(counts, dropped, seed):
    import torch

    import sparse_dense_matrix_spmm_gb300 as spmm
    ids = np.concatenate([np.full(c, e) for e, c in enumerate(counts)] + [np.full(dropped, -1)]).astype(np.int64)
    ids = np.random.default_rng(seed).permutation(ids)
    if ids.size == 0:
        ids = np.zeros(0, np.int64)
    R = spmm.spmm_build_route(torch.from_numpy(ids).cuda(), len(counts))
    return R, route(ids, len(counts))[2]


@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("pad", [0, 8])
@pytest.mark.parametrize("counts,dropped,N,K", CASES)
def test_experts_and_gradients(dtype, pad, counts, dropped, N, K):
    """Forward, dx and dw; rows of dropped choices hold NaN on the way in and zeros on the way out."""
    torch = need_gpu()
    import sparse_dense_matrix_spmm_gb300 as spmm
    E = len(counts)
    R, offsets = _case(counts, dropped, N + K)
    n, kept = R.n_rows, int(offsets[-1])
    xs = matrix((n, K), dtype, 1, pitch=K + pad)
    dys = matrix((n, N), dtype, 2, pitch=N + pad)
    W = matrix((E, N, K), dtype, 3, K ** -0.5, pitch=K + pad)
    xs[kept:], dys[kept:] = float("nan"), float("nan")
    X, D, V = f64(xs), f64(dys), f64(W)
    ys, ysm = np.zeros((n, N)), np.zeros((n, N))
    dx, dxm = np.zeros((n, K)), np.zeros((n, K))
    dw, dwm = np.zeros((E, N, K)), np.zeros((E, N, K))
    for e in range(E):
        a, b = offsets[e], offsets[e + 1]
        ys[a:b], ysm[a:b] = X[a:b] @ V[e].T, np.abs(X[a:b]) @ np.abs(V[e]).T
        dx[a:b], dxm[a:b] = D[a:b] @ V[e], np.abs(D[a:b]) @ np.abs(V[e])
        dw[e], dwm[e] = D[a:b].T @ X[a:b], np.abs(D[a:b]).T @ np.abs(X[a:b])
    buf = torch.full((n, N + 8), 7.0, dtype=DT[dtype], device="cuda")
    check(spmm.spmm_experts(R, xs, W, out=buf[:, :N]), ys, ysm, K, dtype, "ys")
    assert (buf[:, N:] == 7.0).all()
    got_dx, got_dw = spmm.spmm_experts_grad(R, dys, xs, W)
    check(got_dx, dx, dxm, N, dtype, "dxs")
    check(got_dw, dw, dwm, max(counts), dtype, "dW")
    wide = torch.full((E, N + 3, K + 8), 7.0, dtype=DT[dtype], device="cuda")
    check(spmm.spmm_experts_dw(R, dys, xs, out=wide[:, :N, :K]), dw, dwm, max(counts), dtype, "dW in a wider array")
    assert (wide[:, N:] == 7.0).all() and (wide[:, :, K:] == 7.0).all()
    torch.cuda.synchronize()
    assert spmm.last_device_error() == 0


@pytest.mark.parametrize("which", ["experts", "dx", "dw"])
def test_other_experts_do_not_leak(which):
    """Infinities and NaN in one expert's rows and weights stay in its own results."""
    torch = need_gpu()
    import sparse_dense_matrix_spmm_gb300 as spmm
    counts = [5, 37, 11, 64, 1]
    R, offsets = _case(counts, 0, 1)
    N, K = 200, 136
    xs, dys, W = matrix((R.n_rows, K), "bf16", 1), matrix((R.n_rows, N), "bf16", 2), matrix((5, N, K), "bf16", 3)
    clean = {"experts": lambda: spmm.spmm_experts(R, xs, W), "dx": lambda: spmm.spmm_experts_dx(R, dys, W),
             "dw": lambda: spmm.spmm_experts_dw(R, dys, xs)}[which]
    before = clean()
    for e in (1, 3):
        a, b = offsets[e], offsets[e + 1]
        xs[a:b], dys[a:b], W[e] = float("inf"), float("nan"), float("nan")
    after = clean()
    for e in (0, 2, 4):
        s = slice(e, e + 1) if which == "dw" else slice(offsets[e], offsets[e + 1])
        assert torch.equal(before[s], after[s])
    assert after[1 if which == "dw" else slice(offsets[1], offsets[2])].isnan().any()


def test_large_product_sampled():
    """A prompt-sized product (2 x 4096 tokens over 8 experts): sampled rows and weight rows."""
    torch = need_gpu()
    import sparse_dense_matrix_spmm_gb300 as spmm
    rng = np.random.default_rng(4)
    E, N, K = 8, 1408, 2048
    ids = torch.from_numpy(rng.integers(0, E, (4096, 2))).cuda()
    R = spmm.spmm_build_route(ids, E)
    offsets = R.offsets.cpu().numpy()
    xs, dys = matrix((8192, K), "bf16", 1), matrix((8192, N), "bf16", 2)
    W = matrix((E, N, K), "bf16", 3, K ** -0.5)
    ys, (dx, dw) = spmm.spmm_experts(R, xs, W), spmm.spmm_experts_grad(R, dys, xs, W)
    rows = np.unique(np.concatenate([offsets[:-1], offsets[1:] - 1, rng.integers(0, 8192, 64)]))
    e_of = np.searchsorted(offsets, rows, side="right") - 1
    X, D, V = f64(xs), f64(dys), f64(W)
    at = torch.from_numpy(rows).cuda()
    check(ys[at], np.stack([V[e] @ X[r] for r, e in zip(rows, e_of)]),
          np.stack([np.abs(V[e]) @ np.abs(X[r]) for r, e in zip(rows, e_of)]), K, "bf16", "ys")
    check(dx[at], np.stack([V[e].T @ D[r] for r, e in zip(rows, e_of)]),
          np.stack([np.abs(V[e]).T @ np.abs(D[r]) for r, e in zip(rows, e_of)]), N, "bf16", "dxs")
    for e in (0, 7):
        a, b = offsets[e], offsets[e + 1]
        check(dw[e], D[a:b].T @ X[a:b], np.abs(D[a:b]).T @ np.abs(X[a:b]), b - a, "bf16", "dW")
    # the same bits on every run
    assert torch.equal(spmm.spmm_experts(R, xs, W), ys)
    assert torch.equal(spmm.spmm_experts_dw(R, dys, xs), dw)


@pytest.mark.parametrize("N,K,rows", [(264, 328, 5), (520, 72, 70), (712, 200, 33)])
def test_many_units_per_cta(N, K, rows):
    """Hundreds of experts, so that every CTA stores many tiles in a row, with odd numbers of
    64-column and 32-row boxes in them (a staging buffer reused before its store had read it)."""
    torch = need_gpu()
    import sparse_dense_matrix_spmm_gb300 as spmm
    E = 300
    R, offsets = _case([rows + e % 3 for e in range(E)], 4, 5)
    xs, dys = matrix((R.n_rows, K), "bf16", 1), matrix((R.n_rows, N), "bf16", 2)
    W = matrix((E, N, K), "bf16", 3, K ** -0.5)
    ys, (dx, dw) = spmm.spmm_experts(R, xs, W), spmm.spmm_experts_grad(R, dys, xs, W)
    for _ in range(3):
        assert torch.equal(spmm.spmm_experts_dw(R, dys, xs), dw)
        assert torch.equal(spmm.spmm_experts(R, xs, W), ys)
    for e in range(E):
        a, b = offsets[e], offsets[e + 1]
        X, D, V = f64(xs[a:b]), f64(dys[a:b]), f64(W[e])
        check(ys[a:b], X @ V.T, np.abs(X) @ np.abs(V).T, K, "bf16", f"ys of {e}")
        check(dx[a:b], D @ V, np.abs(D) @ np.abs(V), N, "bf16", f"dxs of {e}")
        check(dw[e], D.T @ X, np.abs(D).T @ np.abs(X), b - a, "bf16", f"dW of {e}")


def test_many_experts_single_tokens():
    """One decoding step: 3 tokens with 8 choices among 300 experts."""
    torch = need_gpu()
    import sparse_dense_matrix_spmm_gb300 as spmm
    rng = np.random.default_rng(8)
    ids = np.stack([rng.choice(300, 8, replace=False) for _ in range(3)])
    R = spmm.spmm_build_route(torch.from_numpy(ids).cuda(), 300)
    offsets = R.offsets.cpu().numpy()
    xs, W = matrix((24, 640), "bf16", 1), matrix((300, 392, 640), "bf16", 2, 0.04)
    ys, X, V = spmm.spmm_experts(R, xs, W), f64(xs), f64(W)
    e_of = np.searchsorted(offsets, np.arange(24), side="right") - 1
    check(ys, np.stack([V[e] @ X[r] for r, e in enumerate(e_of)]),
          np.stack([np.abs(V[e]) @ np.abs(X[r]) for r, e in enumerate(e_of)]), 640, "bf16", "ys")


def test_empty_and_side_stream():
    torch = need_gpu()
    import sparse_dense_matrix_spmm_gb300 as spmm
    R, _ = _case([0, 0], 0, 1)
    W = matrix((2, 64, 128), "bf16", 1)
    z = torch.zeros((0, 128), dtype=torch.bfloat16, device="cuda")
    assert spmm.spmm_experts(R, z, W).shape == (0, 64)
    dw = spmm.spmm_experts_dw(R, torch.zeros((0, 64), dtype=torch.bfloat16, device="cuda"), z,
                              out=torch.ones_like(W))
    assert not dw.any()
    R, offsets = _case([3, 40], 0, 2)
    xs = matrix((43, 128), "bf16", 2)
    here = spmm.spmm_experts(R, xs, W)
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    there = spmm.spmm_experts(R, xs, W, stream=s)
    s.synchronize()
    assert torch.equal(here, there)


def test_refusals():
    torch = need_gpu()
    import sparse_dense_matrix_spmm_gb300 as spmm
    R, _ = _case([3, 5], 0, 1)
    xs, W = matrix((8, 64), "bf16", 1), matrix((2, 32, 64), "bf16", 2)
    with pytest.raises(TypeError):
        spmm.spmm_experts(R, xs.float(), W)                             # types differ
    with pytest.raises(spmm.SpmmError, match="DTYPE"):
        spmm.spmm_experts(R, xs.float(), W.float())
    with pytest.raises(ValueError):
        spmm.spmm_experts(R, xs[:7], W)
    with pytest.raises(ValueError):
        spmm.spmm_experts(R, xs, W[:1])
    with pytest.raises(ValueError):
        spmm.spmm_experts(R, xs, W.transpose(1, 2).contiguous().transpose(1, 2))
    with pytest.raises(spmm.SpmmError, match="SHAPE"):
        spmm.spmm_experts(R, matrix((8, 60), "bf16", 1), matrix((2, 32, 60), "bf16", 2))   # K % 8
    with pytest.raises(spmm.SpmmError, match="SHAPE"):
        spmm.spmm_experts(R, matrix((8, 64), "bf16", 1, pitch=68), W)                      # pitch % 8
    with pytest.raises(spmm.SpmmError, match="SHAPE"):
        spmm.spmm_experts(R, matrix((8, 72), "bf16", 1)[:, 4:68], W)                       # base not 16-byte aligned
    with pytest.raises(spmm.SpmmError, match="SHAPE"):
        spmm.spmm_experts(R, xs, W[:1].expand(2, 32, 64))                                  # overlapping experts
