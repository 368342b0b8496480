"""The gated block at depths of one and two steps of 64, with several units per SM whose row counts differ: the border
between the epilogue's warps moves from unit to unit."""
import numpy as np
import pytest

from tests.gpu_util import need_gpu
from tests.onehot_util import f64, matrix
from tests.test_gpu_gated import _check_h, _check_packed, _route, _sums

pytestmark = pytest.mark.gpu


# experts, their rows at most, N (2 N <= 128: single CTAs; else pairs), K
@pytest.mark.parametrize("experts,most,N", [(400, 60, 32), (420, 300, 48), (260, 300, 128), (120, 250, 272), (700, 30, 144)])
@pytest.mark.parametrize("K", [8, 64, 72, 128])
@pytest.mark.parametrize("dtype", ["f16", "bf16"])
def test_ragged_units(experts, most, N, K, dtype):
    torch = need_gpu()
    import sparse_dense_matrix_spmm_gb300 as spmm
    rng = np.random.default_rng(experts + K)
    counts = [int(c) for c in rng.integers(0, most + 1, experts)]
    R, offsets = _route(counts, 5, K)
    n, kept = R.n_rows, int(offsets[-1])
    xs, W = matrix((n, K), dtype, 1), matrix((experts, 2 * N, K), dtype, 3, 1.5 * K ** -0.5)
    runs = [spmm.spmm_experts_gated(R, xs, W, save="packed") for _ in range(4)]
    h, P = runs[0]
    for h2, P2 in runs[1:]:
        assert torch.equal(h2, h) and torch.equal(P2.q, P.q) and torch.equal(P2.scale, P.scale)
    X = f64(xs)
    X[kept:] = 0
    gu, mag = _sums(X, f64(W), offsets)
    _check_h(h, gu, mag, K, N, "silu", dtype)
    _check_packed(P, gu, mag, K)
    assert not h[kept:].any() and not P.q[kept:].any() and (P.scale[kept:] == 1).all()
    if K <= 64 or dtype == "bf16":  # one sum in every form
        assert torch.equal(h, spmm.spmm_experts_gated(R, xs, W))
    assert spmm.last_device_error() == 0
