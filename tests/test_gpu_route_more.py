"""Routes at sizes and key counts where the sort changes its form, against the stable sort."""
import numpy as np
import pytest

from tests.gpu_util import need_gpu
from tests.onehot_util import route

pytestmark = pytest.mark.gpu


def _ids(T, k, n_keys, seed, drop):
    rng = np.random.default_rng(seed)
    ids = np.minimum((rng.random((T, k)) ** 2 * n_keys).astype(np.int64), n_keys - 1)
    return np.where(rng.random((T, k)) < drop, -1, ids)


def _check(ids, n_keys):
    import torch

    import sparse_dense_matrix_spmm_gb300 as spmm
    R = spmm.spmm_build_route(torch.from_numpy(ids).cuda(), n_keys)
    order, pos, offsets = route(ids, n_keys)
    assert np.array_equal(R.order.cpu().numpy(), order)
    assert np.array_equal(R.pos.cpu().numpy(), pos)
    assert np.array_equal(R.offsets.cpu().numpy(), offsets)
    if R.k == 1:
        flat = ids.reshape(-1)[order]
        assert np.array_equal(R.keys.cpu().numpy(), np.where((flat < 0) | (flat >= n_keys), n_keys, flat))


@pytest.mark.parametrize("n_keys", [1, 2, 7, 15, 16, 31, 32])
@pytest.mark.parametrize("n", [2049, 4096, 5000, 12289, 16383, 16384])
def test_clusters_with_few_keys(n, n_keys):
    """Two to eight tiles, one digit with fewer values than a warp has threads."""
    need_gpu()
    _check(_ids(n, 1, n_keys, n + n_keys, 0.1), n_keys)
    _check(_ids(n // 3, 3, n_keys, n - n_keys, 0.02), n_keys)


@pytest.mark.parametrize("T,k,n_keys,drop", [(300001, 1, 5000, 0.0), (300001, 1, 200000, 0.1), (150001, 2, 200000, 0.0),
                                             (300001, 1, 300000, 0.3), (100003, 7, 1000, 0.01)])
def test_many_elements_over_many_keys(T, k, n_keys, drop):
    """More than 262144 elements in two or three passes: a CTA takes several tiles, and the counts of the
    next pass go to the CTA that will read the element there."""
    need_gpu()
    _check(_ids(T, k, n_keys, T + n_keys, drop), n_keys)
