"""The weight gradient's tails: what follows an expert's last row belongs to the next one and is cleared in both CTAs
of a pair before it is multiplied, in many units on each pair and again and again."""
import numpy as np
import pytest

from tests.gpu_util import need_gpu
from tests.onehot_util import DT, check, f64, matrix

pytestmark = pytest.mark.gpu

COUNTS = [601, 47, 1, 130, 63, 575, 15, 17, 333, 65, 2, 255, 31, 401, 129, 90]


@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("N,K", [(1032, 1544), (2560, 3584), (120, 2048)])
def test_neighbours_of_nan(dtype, N, K):
    """Every other expert's rows are NaN: the experts between them keep their bits."""
    torch = need_gpu()
    import sparse_dense_matrix_spmm_gb300 as spmm
    E, n = len(COUNTS), sum(COUNTS)
    ids = torch.from_numpy(np.repeat(np.arange(E), COUNTS)).cuda()
    R = spmm.spmm_build_route(ids, E)
    xs, dys = matrix((n, K), dtype, 1), matrix((n, N), dtype, 2)
    first = spmm.spmm_experts_dw(R, dys, xs)
    start = np.concatenate([[0], np.cumsum(COUNTS)])
    for odd in (0, 1):
        x, d = xs.clone(), dys.clone()
        for e in range(1 - odd, E, 2):
            x[start[e]:start[e + 1]] = float("nan")
            d[start[e]:start[e + 1]] = float("nan")
        for _ in range(8):
            again = torch.full((E, N, K), 7.0, dtype=DT[dtype], device="cuda")
            spmm.spmm_experts_dw(R, d, x, out=again)
            assert torch.equal(again[odd::2], first[odd::2])
            assert again[1 - odd::2].isnan().all()
    assert spmm.last_device_error() == 0


def test_sums_of_ragged_experts():
    torch = need_gpu()
    import sparse_dense_matrix_spmm_gb300 as spmm
    E, n, N, K = len(COUNTS), sum(COUNTS), 520, 776
    R = spmm.spmm_build_route(torch.from_numpy(np.repeat(np.arange(E), COUNTS)).cuda(), E)
    xs, dys = matrix((n, K), "f16", 1), matrix((n, N), "f16", 2)
    X, D, start = f64(xs), f64(dys), np.concatenate([[0], np.cumsum(COUNTS)])
    rows = [slice(start[e], start[e + 1]) for e in range(E)]
    want = np.stack([D[r].T @ X[r] for r in rows])
    check(spmm.spmm_experts_dw(R, dys, xs), want, np.stack([np.abs(D[r]).T @ np.abs(X[r]) for r in rows]), max(COUNTS),
          "f16", "dW")
