"""The gated experts' C entries with pitches that the Python wrappers do not use: wider rows of [g u], of its 8-bit form, of
h, of the gradients and of the weights' gradient; and 8-bit rows at odd addresses.  What lies between the rows stays."""
import ctypes as C

import numpy as np
import pytest

from tests.gpu_util import need_gpu
from tests.onehot_util import DT, matrix

pytestmark = pytest.mark.gpu


def _wide(torch, rows, cols, pad, dtype, fill=7):
    full = torch.full((rows, cols + pad), fill, dtype=dtype, device="cuda")
    return full, full[:, :cols]


@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("tokens,experts", [(3, 4), (200, 4), (90, 40), (4200, 2)])
def test_wider_rows(dtype, tokens, experts):
    torch = need_gpu()
    import sparse_dense_matrix_spmm_gb300 as spmm
    from sparse_dense_matrix_spmm_gb300 import _lib
    N, K, t = 144, 264, DT[dtype]
    code = {"bf16": _lib.SPMM_BF16, "f16": _lib.SPMM_F16}[dtype]
    ids = np.random.default_rng(tokens).integers(-1, experts, (tokens, 2))
    R = spmm.spmm_build_route(torch.from_numpy(ids).cuda(), experts)
    n = R.n_rows
    xs, W, dh = matrix((n, K), dtype, 1), matrix((experts, 2 * N, K), dtype, 2, K ** -0.5), matrix((n, N), dtype, 3)
    h, gu = spmm.spmm_experts_gated(R, xs, W, act="gelu", save="rows")
    h8, P = spmm.spmm_experts_gated(R, xs, W, act="gelu", save="packed")
    stream = spmm._handle(None, xs.device)
    room = torch.empty(spmm.spmm_experts_gated_grad_workspace_size(R, N, K, False) + 16, dtype=torch.uint8, device="cuda")
    fh, wh = _wide(torch, n, N, 24, t)
    fg, wg = _wide(torch, n, 2 * N, 40, t)
    _lib.call("spmm_experts_gated", R._ref, xs.data_ptr(), K, W.data_ptr(), K, 2 * N * K, N, K, code, _lib.ACT_GELU, wh.data_ptr(),
              N + 24, wg.data_ptr(), 2 * N + 40, None, stream)
    assert torch.equal(wh, h) and torch.equal(wg, gu) and (fh[:, N:] == 7).all() and (fg[:, 2 * N:] == 7).all()
    fq, wq = _wide(torch, n, 2 * N, 48, torch.int8)
    fs, ws = _wide(torch, n, N // 8, 5, torch.uint8)
    Q = spmm.Rows8(n, 2 * N, t, wq, ws)
    _lib.call("spmm_experts_gated", R._ref, xs.data_ptr(), K, W.data_ptr(), K, 2 * N * K, N, K, code, _lib.ACT_GELU, wh.data_ptr(),
              N + 24, None, 0, Q._ref, stream)
    assert torch.equal(wh, h8) and torch.equal(wq, P.q) and torch.equal(ws, P.scale)
    assert (fq[:, 2 * N:] == 7).all() and (fs[:, N // 8:] == 7).all()
    for kept, wide, pitch in ((gu, wg, 2 * N + 40), (P, Q, 0)):
        dgu, h2 = spmm.spmm_gated_grad(R, dh, kept, act="gelu", with_h=True)
        fd, wd = _wide(torch, n, 2 * N, 8, t)
        f2, w2 = _wide(torch, n, N, 16, t)
        rows = wide.data_ptr() if pitch else None
        _lib.call("spmm_gated_grad", R._ref, dh.data_ptr(), N, rows, pitch or 2 * N, None if pitch else wide._ref, N, code,
                  _lib.ACT_GELU, wd.data_ptr(), 2 * N + 8, w2.data_ptr(), N + 16, stream)
        assert torch.equal(wd, dgu) and torch.equal(w2, h2) and (fd[:, 2 * N:] == 7).all() and (f2[:, N:] == 7).all()
        want = spmm.spmm_experts_gated_grad(R, dh, xs, W, kept, act="gelu")
        fx, wx = _wide(torch, n, K, 8, t)
        fw = torch.full((experts, 2 * N + 3, K + 16), 7, dtype=t, device="cuda")
        _lib.call("spmm_experts_gated_grad", R._ref, dh.data_ptr(), N, xs.data_ptr(), K, None, W.data_ptr(), K, 2 * N * K, rows,
                  pitch or 2 * N, None if pitch else wide._ref, N, K, code, _lib.ACT_GELU, wd.data_ptr(), 2 * N + 8, wx.data_ptr(),
                  K + 8, fw.data_ptr(), K + 16, (2 * N + 3) * (K + 16), room.data_ptr(), C.c_size_t(room.numel()), stream)
        assert torch.equal(wd, want[0]) and torch.equal(wx, want[1]) and torch.equal(fw[:, :2 * N, :K], want[2])
        assert (fx[:, K:] == 7).all() and (fw[:, 2 * N:] == 7).all() and (fw[:, :, K:] == 7).all()
    torch.cuda.synchronize()
    assert spmm.last_device_error() == 0


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("shift", [1, 2, 4, 8])
def test_integers_at_odd_addresses(dtype, shift):
    torch = need_gpu()
    import sparse_dense_matrix_spmm_gb300 as spmm
    x = matrix((13, 70), dtype, 4)
    want = spmm.spmm_pack_rows(x)
    q = torch.full((13, 112), 99, dtype=torch.int8, device="cuda")
    scale = torch.full((13, 9), 99, dtype=torch.uint8, device="cuda")
    P = spmm.Rows8(13, 70, x.dtype, q[:, shift:shift + 70], scale[:, 3:8])
    spmm.spmm_pack_rows(x, P)
    assert torch.equal(P.q, want.q) and torch.equal(P.scale, want.scale)
    assert (q[:, :shift] == 99).all() and (q[:, shift + 70:] == 99).all()
    assert (scale[:, :3] == 99).all() and (scale[:, 8:] == 99).all()
    assert torch.equal(spmm.spmm_unpack_rows(P), spmm.spmm_unpack_rows(want))


def test_refused_before_a_launch():
    """Limits and shapes that only real tensors reach."""
    torch = need_gpu()
    import sparse_dense_matrix_spmm_gb300 as spmm
    with pytest.raises(spmm.SpmmError, match="UNSUPPORTED"):
        spmm.spmm_topk(matrix((2, 1025), "f32", 1), 2)
    with pytest.raises(spmm.SpmmError, match="UNSUPPORTED"):
        spmm.spmm_topk(matrix((2, 64), "f32", 1), 33)
    with pytest.raises(spmm.SpmmError, match="SHAPE"):
        spmm.spmm_topk(matrix((1, 64), "f32", 1).expand(5, 64), 2)  # every token the same row
    R = spmm.spmm_build_route(torch.zeros(4, dtype=torch.int64, device="cuda"), 1)
    xs, W = matrix((4, 64), "bf16", 1), matrix((1, 96, 64), "bf16", 2)
    for bad in (lambda: spmm.spmm_experts_gated(R, xs, W[:, :80]),                     # N = 40
                lambda: spmm.spmm_experts_gated(R, xs, W, out=matrix((4, 56), "bf16", 3)[:, 4:52]),
                lambda: spmm.spmm_experts_gated(R, matrix((4, 68), "bf16", 3)[:, :64], W),
                lambda: spmm.spmm_experts_gated(R, xs[:, :60], W[:, :, :60])):
        with pytest.raises(spmm.SpmmError, match="SHAPE"):
            bad()
    h, gu = spmm.spmm_experts_gated(R, xs, W, save="packed")
    other = spmm.Rows8(4, 96, torch.float16, gu.q, gu.scale)
    with pytest.raises(ValueError, match="gu must hold"):
        spmm.spmm_gated_grad(R, h, other)
    tight = spmm.Rows8(4, 96, torch.bfloat16, torch.zeros(4, 104, dtype=torch.int8, device="cuda")[:, :96], gu.scale)
    with pytest.raises(spmm.SpmmError, match="SHAPE"):
        spmm.spmm_gated_grad(R, h, tight)  # a pitch of 104
    assert spmm.last_device_error() == 0
