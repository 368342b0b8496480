"""The weights' gradient of few rows per expert on average (sums on CUDA cores), where
one expert has more rows than are staged at a time and where a row is longer than a CTA
covers in one go, against plain 64-bit products."""
import numpy as np
import pytest

from tests.gpu_util import need_gpu
from tests.onehot_util import DT, check, f64, matrix, route

pytestmark = pytest.mark.gpu

# rows per expert, dropped rows, N, K: 16 rows are staged at a time, 1024 columns taken in one go; the form
# is chosen by rows <= 4 experts, dropped ones included
CASES = [([40] + [0] * 30, 3, 24, 1032), ([17, 1] + [0] * 20, 2, 16, 2056), ([3, 0, 5, 2], 1, 40, 2056),
         ([16, 0, 0, 0], 0, 8, 1024), ([0, 33, 32, 0, 31] + [0] * 30, 5, 56, 3080), ([0, 0, 12], 0, 136, 1040),
         ([500] + [0] * 130, 7, 8, 24), ([1] * 60 + [15, 16, 17], 4, 72, 1032)]


@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("pad", [0, 8])
@pytest.mark.parametrize("counts,dropped,N,K", CASES)
def test_dw_of_skewed_batches(dtype, pad, counts, dropped, N, K):
    torch = need_gpu()
    import sparse_dense_matrix_spmm_gb300 as spmm
    E = len(counts)
    ids = np.concatenate([np.full(c, e) for e, c in enumerate(counts)] + [np.full(dropped, -1)]).astype(np.int64)
    ids = np.random.default_rng(N + K).permutation(ids)
    assert ids.size <= 4 * E
    R, offsets = spmm.spmm_build_route(torch.from_numpy(ids).cuda(), E), route(ids, E)[2]
    kept = int(offsets[-1])
    xs = matrix((ids.size, K), dtype, 1, pitch=K + pad)
    dys = matrix((ids.size, N), dtype, 2, pitch=N + pad)
    xs[kept:], dys[kept:] = float("nan"), float("nan")
    X, D = f64(xs), f64(dys)
    dw, mag = np.zeros((E, N, K)), np.zeros((E, N, K))
    for e in range(E):
        a, b = offsets[e], offsets[e + 1]
        dw[e], mag[e] = D[a:b].T @ X[a:b], np.abs(D[a:b]).T @ np.abs(X[a:b])
    wide = torch.full((E, N + 1, K + pad), 7.0, dtype=DT[dtype], device="cuda")
    check(spmm.spmm_experts_dw(R, dys, xs, out=wide[:, :N, :K]), dw, mag, max(counts), dtype, "dW")
    assert (wide[:, N:] == 7.0).all() and (wide[:, :, K:] == 7.0).all()
    assert torch.equal(spmm.spmm_experts_dw(R, dys, xs), wide[:, :N, :K])
