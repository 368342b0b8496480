"""The weight gradient of long experts: stores by threads and by TMA, by where the gradient lies."""
import numpy as np
import pytest

from tests.gpu_util import need_gpu
from tests.onehot_util import DT, check, f64, matrix, route

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("counts,N,K", [
    ([513], 8, 8), ([1030], 136, 264), ([700, 0, 1500], 72, 200), ([600, 513, 530], 264, 72), ([2049, 1, 0, 37], 520, 584),
    ([0, 1281], 256, 512)])
def test_both_ways_of_storing_give_the_same_bits(dtype, counts, N, K):
    """dW on 32 bytes, dW 16 bytes past them, and rows of dW that are not whole sectors; what lies around stays."""
    torch = need_gpu()
    import sparse_dense_matrix_spmm_gb300 as spmm
    E, n = len(counts), sum(counts)
    ids = np.random.default_rng(n + K).permutation(np.repeat(np.arange(E), counts)).astype(np.int64)
    R, offsets = spmm.spmm_build_route(torch.from_numpy(ids).cuda(), E), route(ids, E)[2]
    xs, dys = matrix((n, K), dtype, 1), matrix((n, N), dtype, 2)
    X, D = f64(xs), f64(dys)
    dw, dwm = np.zeros((E, N, K)), np.zeros((E, N, K))
    for e in range(E):
        rows = slice(offsets[e], offsets[e + 1])
        dw[e], dwm[e] = D[rows].T @ X[rows], np.abs(D[rows]).T @ np.abs(X[rows])
    pitch = (K + 15) // 16 * 16 + 16
    first = None
    for ld, at in ((pitch, 0), (pitch, 8), (pitch + 8, 0), (pitch + 8, 8)):
        wide = torch.full((E, N + 2, ld), 7.0, dtype=DT[dtype], device="cuda")
        out = wide[:, :N, at:at + K]
        spmm.spmm_experts_dw(R, dys, xs, out=out)
        check(out, dw, dwm, max(counts), dtype, "dW")
        assert (wide[:, N:] == 7.0).all() and (wide[:, :, :at] == 7.0).all() and (wide[:, :, at + K:] == 7.0).all()
        first = out.clone() if first is None else first
        assert torch.equal(out, first)
    torch.cuda.synchronize()
    assert spmm.last_device_error() == 0


def test_past_32_bits():
    """An expert's gradient that begins past 2^31 elements."""
    torch = need_gpu()
    import sparse_dense_matrix_spmm_gb300 as spmm
    n, N, K = 2080, 264, 72
    ids = torch.arange(n, device="cuda") % 2
    R = spmm.spmm_build_route(ids, 2)
    xs, dys = matrix((n, K), "bf16", 1), matrix((n, N), "bf16", 2)
    apart = (1 << 31) + 16
    store = torch.empty(apart + N * 80, dtype=torch.bfloat16, device="cuda")
    out = torch.as_strided(store, (2, N, K), (apart, 80, 1))
    spmm.spmm_experts_dw(R, dys, xs, out=out)
    assert torch.equal(out, spmm.spmm_experts_dw(R, dys, xs))
