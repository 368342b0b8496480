"""Forms of the row operators that need a case of their own, against plain definitions."""
import numpy as np
import pytest

from tests.gpu_util import need_gpu
from tests.onehot_util import DT

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dtype", ["bf16", "f16", "f32"])
def test_rows_without_columns(dtype):
    """H = 0: nothing to move, and the weights' gradient is a sum of nothing."""
    torch = need_gpu()
    import sparse_dense_matrix_spmm_gb300 as spmm
    T, k = 5, 3
    ids = np.random.default_rng(1).integers(-1, 4, (T, k))
    R = spmm.spmm_build_route(torch.from_numpy(ids).cuda(), 4)
    x, ys = torch.empty((T, 0), dtype=DT[dtype], device="cuda"), torch.empty((T * k, 0), dtype=DT[dtype], device="cuda")
    w = torch.ones((T, k), device="cuda")
    assert spmm.spmm_dispatch(R, x).shape == (T * k, 0)
    assert spmm.spmm_combine(R, ys, w).shape == (T, 0)
    junk = torch.full((T, k), 9.0, device="cuda")  # what dw's memory may hold before
    del junk
    dys, dw = spmm.spmm_combine_grad(R, x, ys, w)
    assert dys.shape == (T * k, 0) and dw.shape == (T, k) and not dw.any()
    assert spmm.last_device_error() == 0


@pytest.mark.parametrize("H", [256 * 65536 + 1, 256 * 65536 * 4 + 8])
def test_table_gradient_of_very_long_rows(H):
    """More pieces of the columns than a grid has rows, for a run that crosses a chunk of tokens."""
    torch = need_gpu()
    import sparse_dense_matrix_spmm_gb300 as spmm
    torch.cuda.empty_cache()
    T = 70
    ids = torch.ones(T, dtype=torch.int64, device="cuda")
    ids[5] = 0
    dy = torch.empty((T, H), dtype=torch.bfloat16, device="cuda")
    for t in range(T):  # small integers: the sums are exact in fp32
        dy[t] = torch.randint(-2, 3, (H,), device="cuda", dtype=torch.int8)
    got = spmm.spmm_embed_grad(spmm.spmm_build_route(ids, 2), dy, out=torch.empty((2, H), device="cuda"))
    want = torch.zeros(H, device="cuda")
    for t in range(T):
        if t != 5:
            want += dy[t]
    assert torch.equal(got[1], want) and torch.equal(got[0], dy[5].float())


@pytest.mark.parametrize("dtype", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("H", [64, 7])
def test_weights_that_are_not_finite(dtype, H):
    """An infinite or NaN weight of a dropped choice does not count, of a kept one it reaches its token only."""
    torch = need_gpu()
    import sparse_dense_matrix_spmm_gb300 as spmm
    ids = np.array([[0, 2, -1], [1, 0, 2], [-1, -1, -1], [2, -1, 0], [1, 2, 0], [0, 1, -1]])
    T, k = ids.shape
    R = spmm.spmm_build_route(torch.from_numpy(ids).cuda(), 3)
    ys = torch.ones((T * k, H), dtype=DT[dtype], device="cuda")
    dy = torch.ones((T, H), dtype=DT[dtype], device="cuda")
    w = torch.full((T, k), 0.5, device="cuda")
    clean = [spmm.spmm_combine(R, ys, w), *spmm.spmm_combine_grad(R, dy, ys, w)]
    for value in (float("inf"), float("nan")):
        v = w.clone()
        v[torch.from_numpy(ids < 0).cuda()] = value
        for a, b in zip(clean, [spmm.spmm_combine(R, ys, v), *spmm.spmm_combine_grad(R, dy, ys, v)]):
            assert torch.equal(a, b)
        v = w.clone()
        v[4, 1] = value
        y, (dys, dw) = spmm.spmm_combine(R, ys, v), spmm.spmm_combine_grad(R, dy, ys, v)
        at = int(R.pos[4, 1])
        assert not y[4].isfinite().any() and not dys[at].isfinite().any()
        others = [t for t in range(T) if t != 4]
        assert torch.equal(y[others], clean[0][others]) and torch.equal(dw, clean[2])
        rows = [p for p in range(T * k) if p != at]
        assert torch.equal(dys[rows], clean[1][rows])
