"""The largest fp16 values in 8 bits.  A group whose largest magnitude is 65280 or more has the unit 2^10, and 65024 and
more are held as 64 units, 65536, which fp16 does not have: they read back as its largest value, 65504, within half a unit of
what they were."""
import numpy as np
import pytest

from tests.gpu_util import need_gpu
from tests.onehot_util import f64, matrix

pytestmark = pytest.mark.gpu

TOP = [65504.0, 65472.0, 65280.0, 65056.0, 65024.0, 64992.0, 64512.0, 64480.0, 63488.0, 0.0]


@pytest.mark.parametrize("cols", [64, 33, 2051])
@pytest.mark.parametrize("shift", [0, 1])
def test_finite_values_stay_finite(cols, shift):
    torch = need_gpu()
    import sparse_dense_matrix_spmm_gb300 as spmm
    x = matrix((6, cols), "f16", cols, pitch=cols + shift)
    x[0, 0], x[1, 5], x[2, cols - 1] = 65504.0, -65504.0, 65280.0
    x[3, :10] = torch.tensor(TOP)
    x[4, 16:26] = -torch.tensor(TOP)
    x[5, 3] = 65248.0  # rounds to 127 units of 2^9
    out = torch.zeros(6, cols + shift, dtype=torch.float16, device="cuda")[:, shift:]
    P = spmm.spmm_pack_rows(x)
    y = spmm.spmm_unpack_rows(P, out=out)
    assert y.isfinite().all()
    unit = 2.0 ** (np.repeat(P.scale.cpu().numpy().astype(np.float64), 16, axis=1)[:, :cols] - 127)
    assert (np.abs(f64(y) - f64(x)) <= unit / 2).all()
    assert y[0, 0] == 65504 and y[1, 5] == -65504 and y[5, 3] == 65024
    wide = spmm.spmm_unpack_rows(P, out=torch.empty(6, cols, device="cuda"))  # exact in fp32
    assert wide[0, 0] == 65536 and wide[1, 5] == -65536
    assert torch.equal(y, wide.clamp(-65504, 65504).half())


def test_what_no_fp16_value_is_held_as_stays_infinite():
    """From rows of fp32: an overflow is not hidden.  Infinities and NaN read back as NaN."""
    torch = need_gpu()
    import sparse_dense_matrix_spmm_gb300 as spmm
    x = torch.zeros(1, 96)
    x[0, 0], x[0, 16], x[0, 32], x[0, 33], x[0, 48], x[0, 64], x[0, 80] = 1e5, -3e38, 65536.0, 1.0, float("inf"), 67584.0, float("nan")
    y = spmm.spmm_unpack_rows(spmm.spmm_pack_rows(x.cuda()), out=torch.empty(1, 96, dtype=torch.float16, device="cuda"))[0].cpu()
    assert y[0] == float("inf") and y[16] == -float("inf") and y[64] == float("inf")
    assert y[32] == 65504 and y[48:64].isnan().all() and y[80:].isnan().all()


def test_gradient_from_a_checkpoint_of_them():
    """dW = dgu^T xs with the rows as the checkpoint reads back: finite where a row holds the largest value."""
    torch = need_gpu()
    import sparse_dense_matrix_spmm_gb300 as spmm
    N, K, n = 48, 64, 40
    R = spmm.spmm_build_route(torch.zeros(n, dtype=torch.int64, device="cuda"), 1)
    xs, W = matrix((n, K), "f16", 1), matrix((1, 2 * N, K), "f16", 2, 2.0 ** -14)
    xs[3, 7], xs[9, 40] = 65504.0, -65504.0
    dh = matrix((n, N), "f16", 3, 2.0 ** -8)
    _, gu = spmm.spmm_experts_gated(R, xs, W, save="rows")
    P = spmm.spmm_pack_rows(xs)
    _, _, dW = spmm.spmm_experts_gated_grad(R, dh, P, W, gu)
    assert dW.isfinite().all()
    assert torch.equal(dW, spmm.spmm_experts_gated_grad(R, dh, spmm.spmm_unpack_rows(P), W, gu)[2])
