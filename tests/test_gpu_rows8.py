"""Rows in 8 bits and back: bit for bit against the definition."""
import numpy as np
import pytest

from tests.gated_util import held, packed
from tests.gpu_util import need_gpu
from tests.onehot_util import DT, f64, matrix

pytestmark = pytest.mark.gpu


def _same(torch, spmm, x, out=None):
    P = spmm.spmm_pack_rows(x, out)
    q, scale = packed(f64(x))
    assert (P.rows, P.cols, P.dtype) == (*x.shape, x.dtype)
    assert np.array_equal(P.scale.cpu().numpy(), scale)
    assert np.array_equal(P.q.cpu().numpy(), q)
    y = spmm.spmm_unpack_rows(P)
    ref = torch.from_numpy(held(q, scale)).to(x.dtype)
    assert y.dtype == x.dtype and torch.equal(y.cpu().nan_to_num(nan=7.0), ref.nan_to_num(nan=7.0))
    return P


@pytest.mark.parametrize("dtype", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("rows,cols", [(1, 1), (1, 16), (3, 15), (2, 17), (5, 31), (7, 64), (4, 130), (33, 264), (3, 1000),
                                       (2, 2051), (2, 4100), (9, 36)])
def test_against_the_definition(dtype, rows, cols):
    torch = need_gpu()
    import sparse_dense_matrix_spmm_gb300 as spmm
    g = torch.Generator().manual_seed(rows * cols)
    size = torch.exp(2 * torch.randn(rows, cols, generator=g))  # groups of unequal size
    x = (torch.randn(rows, cols, generator=g) * size).to(DT[dtype]).cuda()
    _same(torch, spmm, x)
    assert spmm.last_device_error() == 0


@pytest.mark.parametrize("dtype", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("pad,shift", [(1, 0), (2, 2), (8, 0), (3, 5)])
def test_pitches_and_alignments(dtype, pad, shift):
    """Rows inside wider ones, at odd places; what lies around the results stays."""
    torch = need_gpu()
    import sparse_dense_matrix_spmm_gb300 as spmm
    rows, cols = 11, 208
    x = matrix((rows, cols + shift), dtype, 5, pitch=cols + shift + pad)[:, shift:]
    q = torch.full((rows, cols + pad), 99, dtype=torch.int8, device="cuda")
    scale = torch.full((rows, 13 + pad), 99, dtype=torch.uint8, device="cuda")
    P = spmm.Rows8(rows, cols, x.dtype, q[:, :cols], scale[:, :13])
    _same(torch, spmm, x, P)
    assert (q[:, cols:] == 99).all() and (scale[:, 13:] == 99).all()
    wide = torch.full((rows, cols + shift + pad), 7.0, dtype=x.dtype, device="cuda")
    y = spmm.spmm_unpack_rows(P, out=wide[:, shift:shift + cols])
    assert torch.equal(y, spmm.spmm_unpack_rows(P))
    assert (wide[:, :shift] == 7).all() and (wide[:, shift + cols:] == 7).all()


@pytest.mark.parametrize("dtype", ["bf16", "f16", "f32"])
def test_borders(dtype):
    """Zeros, infinities, NaN, the type's largest and smallest values, ties, and magnitudes that round to 128."""
    torch = need_gpu()
    import sparse_dense_matrix_spmm_gb300 as spmm
    f = torch.finfo(DT[dtype])
    x = torch.zeros(16, 48, dtype=DT[dtype])
    x[1, 3], x[1, 20] = float("inf"), float("-inf")
    x[2, 47] = float("nan")
    x[3, :16], x[3, 16:32], x[3, 40] = f.max, f.min, f.max
    x[4, 0], x[4, 17], x[4, 33] = f.tiny, -f.tiny, f.smallest_normal
    x[5, 0], x[5, 1] = f.smallest_normal * f.eps, -f.smallest_normal * f.eps  # the smallest subnormal
    x[6] = torch.linspace(-127.5, 127.5, 48).to(DT[dtype])
    x[7, 0], x[7, 16], x[7, 32] = 127.5, 127.0, -127.5
    x[8, :16] = torch.tensor([127.0] + [i + 0.5 for i in range(15)])  # ties go to the even integer
    x[9, :16] = torch.tensor([255.0, -254.0] + [2.0 * i + 1 for i in range(14)])
    x[10, 5] = -0.0
    x[11, :3] = torch.tensor([1.0, f.eps, 2.0 ** -9])
    x[12, ::2] = f.max
    x[13, :2] = torch.tensor([f.max, 1.0])
    _same(torch, spmm, x.cuda())


@pytest.mark.parametrize("source", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("target", ["bf16", "f16", "f32"])
def test_read_as_another_type(source, target):
    torch = need_gpu()
    import sparse_dense_matrix_spmm_gb300 as spmm
    x = matrix((6, 100), source, 3, 1e4)
    P = spmm.spmm_pack_rows(x)
    y = spmm.spmm_unpack_rows(P, out=torch.empty(6, 100, dtype=DT[target], device="cuda"))
    assert torch.equal(y.cpu(), torch.from_numpy(held(P.q.cpu().numpy(), P.scale.cpu().numpy())).to(DT[target]))


def test_error_bound():
    """At most half a unit 2^e.  e is the smallest for which the group's largest magnitude rounds to 127 at most, so at
    e - 1 it rounds to 128 or more: it is at least 127.5 2^(e - 1), and half a unit is at most 1 / 127.5 of it."""
    torch = need_gpu()
    import sparse_dense_matrix_spmm_gb300 as spmm
    x = matrix((64, 512), "f32", 9)
    y = f64(spmm.spmm_unpack_rows(spmm.spmm_pack_rows(x)))
    v = f64(x).reshape(64, -1, 16)
    top = np.abs(v).max(2, keepdims=True)
    assert (np.abs(y.reshape(v.shape) - v) <= top / 127.5).all()


def test_nothing_to_do():
    torch = need_gpu()
    import sparse_dense_matrix_spmm_gb300 as spmm
    for shape in ((0, 64), (0, 5), (3, 0)):
        x = torch.empty(shape, dtype=torch.bfloat16, device="cuda")
        assert spmm.spmm_unpack_rows(spmm.spmm_pack_rows(x)).shape == shape


def test_offsets_past_32_bits():
    """Rows whose byte offsets pass 2^32: the last ones come back."""
    torch = need_gpu()
    import sparse_dense_matrix_spmm_gb300 as spmm
    rows, cols = 4, (1 << 30) + 40
    x = torch.zeros(rows, cols, dtype=torch.bfloat16, device="cuda")
    tail = matrix((rows, 56), "bf16", 4)
    x[:, -56:] = tail
    P = spmm.spmm_pack_rows(x)
    y = spmm.spmm_unpack_rows(P)
    q, scale = packed(f64(x[:, -56:]))  # cols - 56 is a multiple of 16
    assert np.array_equal(P.q[:, -56:].cpu().numpy(), q) and np.array_equal(P.scale[:, -4:].cpu().numpy(), scale)
    assert torch.equal(y[:, -56:].cpu(), torch.from_numpy(held(q, scale)).to(torch.bfloat16))
    assert not y[:, :-56].any()
