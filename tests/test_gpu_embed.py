"""Embedding lookup and its gradient by sorted tokens against plain 64-bit definitions."""
import numpy as np
import pytest

from tests.gpu_util import need_gpu
from tests.onehot_util import DT, check, f64, matrix

pytestmark = pytest.mark.gpu


def _ids(T, V, seed, pad=0.0, hot=0.0):
    rng = np.random.default_rng(seed)
    ids = np.minimum((rng.random(T) ** 4 * V).astype(np.int64), V - 1)
    ids = np.where(rng.random(T) < hot, V // 2, ids)
    return np.where(rng.random(T) < pad, -1, ids)


@pytest.mark.parametrize("dtype", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("T,V,H,pitch", [(1, 1, 1, 0), (1, 50021, 4096, 0), (9, 17, 7, 0), (300, 1000, 520, 528),
                                         (300, 1000, 520, 523), (65, 40, 8200, 0)])
@pytest.mark.parametrize("scale", [1.0, 22.627417])
def test_embed(dtype, T, V, H, pitch, scale):
    torch = need_gpu()
    import sparse_dense_matrix_spmm_gb300 as spmm
    ids = _ids(T, V, T + V, 0.2 if T > 1 else 0.0)
    table = matrix((V, H), dtype, 4, 0.05, pitch or None)
    s32 = float(np.float32(scale))
    ref = np.where(ids[:, None] >= 0, f64(table)[np.maximum(ids, 0)] * s32, 0.0)
    for it in (torch.int32, torch.int64):
        out = torch.full((T, H + 5), 7.0, dtype=DT[dtype], device="cuda")
        got = spmm.spmm_embed(table, torch.from_numpy(ids).to(it).cuda(), scale, out=out[:, :H])
        check(got, ref, np.abs(ref), 0, dtype, "embed")
        assert (out[:, H:] == 7.0).all()
        check(spmm.spmm_embed(table, torch.from_numpy(ids).to(it).cuda(), scale), ref, np.abs(ref), 0, dtype, "embed")


def test_embed_ids_past_the_table():
    torch = need_gpu()
    import sparse_dense_matrix_spmm_gb300 as spmm
    spmm.last_device_error()
    table = matrix((10, 64), "bf16", 1)
    out = spmm.spmm_embed(table, torch.tensor([3, 10, -1, 1 << 40], device="cuda"))
    assert torch.equal(out[0], table[3]) and not out[1:].any()
    assert spmm.last_device_error() == spmm._lib.DEVERR_INDEX
    assert spmm.spmm_embed(table, torch.zeros(0, dtype=torch.int64, device="cuda")).shape == (0, 64)


def _grad_ref(ids, V, dy, scale):
    D = f64(dy)
    ref, mag = np.zeros((V, D.shape[1])), np.zeros((V, D.shape[1]))
    live = ids >= 0
    np.add.at(ref, ids[live], D[live])
    np.add.at(mag, ids[live], np.abs(D[live]))
    s = float(np.float32(scale))
    return ref * s, mag * abs(s)


@pytest.mark.parametrize("dtype,out_dtype", [("bf16", "bf16"), ("bf16", "f32"), ("f16", "f16"), ("f16", "f32"),
                                             ("f32", "f32")])
@pytest.mark.parametrize("T,V,H,pitch,hot", [
    (1, 1, 1, 0, 0.0), (1, 700, 64, 0, 0.0), (63, 5, 7, 0, 0.0), (64, 1, 96, 0, 0.0), (129, 3, 520, 528, 0.9),
    (1000, 600, 40, 0, 0.5), (1025, 4, 523, 0, 1.0), (777, 2000, 520, 523, 0.3), (4096, 33, 264, 0, 0.6)])
def test_embed_grad(dtype, out_dtype, T, V, H, pitch, hot):
    """Rows with no token, with one, and with runs that span many tokens (all of them on one row as well)."""
    torch = need_gpu()
    import sparse_dense_matrix_spmm_gb300 as spmm
    ids = _ids(T, V, 3 * T + V, 0.1 if T > 1 else 0.0, hot)
    dy = matrix((T, H), dtype, 9, pitch=pitch or None)
    R = spmm.spmm_build_route(torch.from_numpy(ids).cuda(), V)
    scale = 1.5
    ref, mag = _grad_ref(ids, V, dy, scale)
    buf = torch.full((V, H + 8), 7.0, dtype=DT[out_dtype], device="cuda")
    got = spmm.spmm_embed_grad(R, dy, scale, out=buf[:, :H])
    check(got, ref, mag, T, out_dtype, "dtable")
    assert (buf[:, H:] == 7.0).all()
    # accumulated onto a table of values: rows without tokens keep their bits
    base = matrix((V, H), out_dtype, 11)
    acc = base.clone()
    spmm.spmm_embed_grad(R, dy, scale, out=acc, accumulate=True)
    check(acc, f64(base) + ref, np.abs(f64(base)) + mag, T + 1, out_dtype, "accumulated")
    idle = np.setdiff1d(np.arange(V), ids)
    assert torch.equal(acc[idle], base[idle])
    # the same bits on every run
    assert torch.equal(spmm.spmm_embed_grad(R, dy, scale, out=torch.empty_like(base)), got)


def test_embed_grad_large_offsets():
    """A gradient of more than 2^31 elements (bf16, 4.8 GB): rows past the 32-bit offset."""
    torch = need_gpu()
    import sparse_dense_matrix_spmm_gb300 as spmm
    V, H, T = 294000, 8192, 257
    ids = np.linspace(0, V - 1, T).astype(np.int64)
    dy = matrix((T, H), "bf16", 2)
    R = spmm.spmm_build_route(torch.from_numpy(ids).cuda(), V)
    got = spmm.spmm_embed_grad(R, dy)
    d = torch.from_numpy(ids).cuda()
    assert torch.equal(got[d], dy)
    assert not got[d[:-1] + 1].any() and not got[V - 2].any()
    # and a lookup in it
    assert torch.equal(spmm.spmm_embed(got, d), dy)


def test_gradient_against_differences():
    """L = sum(embed(table) * g) is linear in the table: a step of 1 in one entry changes it by the gradient."""
    torch = need_gpu()
    import sparse_dense_matrix_spmm_gb300 as spmm
    T, V, H = 40, 6, 12
    ids = _ids(T, V, 5, 0.2)
    d = torch.from_numpy(ids).cuda()
    table, g = matrix((V, H), "f32", 1), matrix((T, H), "f32", 2)
    grad = spmm.spmm_embed_grad(spmm.spmm_build_route(d, V), g, 2.0)

    def loss(t):
        return float((f64(spmm.spmm_embed(t, d, 2.0)) * f64(g)).sum())

    tol = T * H * 16 * 2.0 ** -23
    for v in range(V):
        old = table[v, v].item()
        table[v, v] = old + 0.5
        up = loss(table)
        table[v, v] = old - 0.5
        down = loss(table)
        table[v, v] = old
        assert abs((up - down) - grad[v, v].item()) <= tol


def test_refusals():
    torch = need_gpu()
    import sparse_dense_matrix_spmm_gb300 as spmm
    table, ids = matrix((10, 64), "bf16", 1), torch.zeros(4, dtype=torch.int64, device="cuda")
    dy = matrix((4, 64), "bf16", 2)
    R = spmm.spmm_build_route(ids, 10)
    with pytest.raises(TypeError):
        spmm.spmm_embed(table.to(torch.float64), ids)
    with pytest.raises(TypeError):
        spmm.spmm_embed(table, ids.float())
    with pytest.raises(ValueError):
        spmm.spmm_embed(table, ids.cpu())
    with pytest.raises(ValueError):
        spmm.spmm_embed(table, torch.zeros((2, 2), dtype=torch.int64, device="cuda"))
    with pytest.raises(ValueError):
        spmm.spmm_embed_grad(R, dy, accumulate=True)                    # nothing to add to
    with pytest.raises(spmm.SpmmError, match="DTYPE"):
        spmm.spmm_embed_grad(R, dy, out=torch.empty((10, 64), dtype=torch.float16, device="cuda"))
    with pytest.raises(ValueError):
        spmm.spmm_embed_grad(R, dy, out=torch.empty((9, 64), dtype=torch.bfloat16, device="cuda"))
    with pytest.raises(spmm.SpmmError, match="SHAPE"):
        spmm.spmm_embed_grad(R, dy[:1].expand(4, 64))                   # a row pitch of 0
    R2 = spmm.spmm_build_route(torch.zeros((2, 2), dtype=torch.int64, device="cuda"), 10)
    with pytest.raises(spmm.SpmmError, match="SHAPE"):
        spmm.spmm_embed_grad(R2, dy[:2])                                # k = 2
