"""The operators of a gated mixture-of-experts layer run together: forward pass and gradients of the example layer
against the same layer in 64 bits (autograd), and the example itself."""
import numpy as np
import pytest

from tests.gpu_util import need_gpu

pytestmark = pytest.mark.gpu

# What is rounded on the way is rounded to bf16 with a relative error of 2^-8 at most: forward logits, h, ys, the sum,
# y; backward dys, dh, dgu (from g and u, rounded too), h again, dxs, dlogits, the sums.  Twelve of them at most are
# passed through by any one result, each in norm.
TOL = 12 * 2.0 ** -8
# A value in 8 bits is off by half a unit, 1 / 127.5 of its group's largest magnitude at most; uniform over the unit, in norm
# by 1 / sqrt(3) of that where every group's values were as small as 1 / 3 of its largest in the mean square: 3 / 127.5
# / sqrt(3) < 2^-6.  Three such values (the rows, g and u) meet in a gradient.
TOL8 = TOL + 3 * 2.0 ** -6


def _example():
    from examples import gated_moe_layer
    return gated_moe_layer


def _reference(torch, layer, x, ids, dy):
    p = [t.detach().double().cpu().requires_grad_() for t in (x, layer.router, layer.up, layer.down)]
    X, router, up, down = p
    ids = ids.cpu()
    F = up.shape[1] // 2
    w = torch.softmax((X @ router.t()).gather(1, ids), dim=1)
    out = X
    for j in range(ids.shape[1]):
        e = ids[:, j]
        gu = torch.einsum("tfh,th->tf", up[e], X)
        out = out + w[:, j, None] * torch.einsum("thf,tf->th", down[e], torch.nn.functional.silu(gu[:, :F]) * gu[:, F:])
    (out * dy.double().cpu()).sum().backward()
    return out.detach(), [t.grad for t in p]


@pytest.mark.parametrize("keep", ["rows", "packed"])
@pytest.mark.parametrize("T,E,H,F,top", [(41, 6, 64, 96, 2), (300, 5, 136, 208, 3), (3, 4, 72, 32, 2)])
def test_layer_against_64_bits(keep, T, E, H, F, top):
    torch = need_gpu()
    import sparse_dense_matrix_spmm_gb300 as spmm
    m = _example()
    layer = m.Layer.random(E, H, F, top, seed=3)
    g = torch.Generator(device="cuda").manual_seed(T)
    x, dy = (torch.randn(T, H, generator=g, device="cuda").to(torch.bfloat16) for _ in range(2))
    y, saved = m.forward(layer, x, keep)
    got = m.backward(layer, saved, dy)
    out, grads = _reference(torch, layer, x, saved[2], dy)
    tol = TOL8 if keep == "packed" else TOL
    for name, a, b, t in [("y", y, out, TOL)] + [(n, a, b, tol) for n, a, b in zip(("dx", "drouter", "dup", "ddown"), got, grads)]:
        a = a.double().cpu()
        assert torch.linalg.vector_norm(a - b) <= t * torch.linalg.vector_norm(b), name
    served, none = m.forward(layer, x)
    assert none is None and torch.equal(served, y)
    assert spmm.last_device_error() == 0


@pytest.mark.parametrize("keep", ["rows", "packed"])
def test_example_runs(keep, capsys):
    need_gpu()
    import sparse_dense_matrix_spmm_gb300 as spmm
    losses = _example().main(["--tokens", "300", "--experts", "8", "--width", "256", "--hidden", "192", "--steps", "2", "--keep",
                              keep])
    assert len(losses) == 2 and np.isfinite(losses).all()
    assert "one decoded token" in capsys.readouterr().out
    assert spmm.last_device_error() == 0


@pytest.mark.parametrize("xs_packed", [False, True])
@pytest.mark.parametrize("gu_packed", [False, True])
def test_the_whole_way_back_is_its_parts(xs_packed, gu_packed):
    """spmm_experts_gated_grad gives the bits of its parts, with a workspace of the caller's too."""
    torch = need_gpu()
    import sparse_dense_matrix_spmm_gb300 as spmm
    from tests.onehot_util import matrix
    R = spmm.spmm_build_route(torch.from_numpy(np.random.default_rng(1).integers(-1, 5, (90, 2))).cuda(), 5)
    xs, W, dh = matrix((180, 136), "f16", 1), matrix((5, 160, 136), "f16", 2, 0.1), matrix((180, 80), "f16", 3)
    h, gu = spmm.spmm_experts_gated(R, xs, W, act="gelu", save="packed" if gu_packed else "rows")
    P = spmm.spmm_pack_rows(xs) if xs_packed else xs
    got = spmm.spmm_experts_gated_grad(R, dh, P, W, gu, act="gelu")
    dgu = spmm.spmm_gated_grad(R, dh, gu, act="gelu")
    rows = spmm.spmm_unpack_rows(P) if xs_packed else xs
    want = dgu, spmm.spmm_experts_dx(R, dgu, W), spmm.spmm_experts_dw(R, dgu, rows)
    need = spmm.spmm_experts_gated_grad_workspace_size(R, 80, 136, xs_packed)
    assert need == (180 * 136 * 2 if xs_packed else 0)
    ws = torch.empty(need + 16, dtype=torch.uint8, device="cuda")
    for a, b, c in zip(got, want, spmm.spmm_experts_gated_grad(R, dh, P, W, gu, act="gelu", workspace=ws)):
        assert torch.equal(a, b) and torch.equal(a, c)
    if xs_packed:
        with pytest.raises(spmm.SpmmError, match="WORKSPACE"):
            spmm.spmm_experts_gated_grad(R, dh, P, W, gu, act="gelu", workspace=ws[:need - 16])


@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("xs_packed", [False, True])
@pytest.mark.parametrize("counts,dropped,N,K", [([5000, 0, 9000], 40, 128, 248), ([8000, 400], 0, 64, 64), ([1, 9000], 5, 80, 520),
                                                ([4500], 0, 16, 8), ([64 * 69, 64 * 67 + 1, 0, 0, 12000], 3, 144, 136)])
def test_dw_in_parts(dtype, xs_packed, counts, dropped, N, K):
    """Few experts with small matrices: dW's rows are summed in parts.  Experts of unequal length, one with fewer rows
    than there are parts, one without any; NaN behind the kept rows; the same bits on every run."""
    torch = need_gpu()
    import sparse_dense_matrix_spmm_gb300 as spmm
    from tests.gated_util import held
    from tests.onehot_util import DT, check, f64, matrix
    ids = np.concatenate([np.full(c, e) for e, c in enumerate(counts)] + [np.full(dropped, -1)])
    R = spmm.spmm_build_route(torch.from_numpy(np.random.default_rng(2).permutation(ids)).cuda(), len(counts))
    n, kept, E = R.n_rows, sum(counts), len(counts)
    offsets = np.concatenate([[0], np.cumsum(counts)])
    xs, W, dh = matrix((n, K), dtype, 1), matrix((E, 2 * N, K), dtype, 2, K ** -0.5), matrix((n, N), dtype, 3)
    gu = matrix((n, 2 * N), dtype, 4)
    xs[kept:], dh[kept:], gu[kept:] = float("nan"), float("nan"), float("nan")
    P = spmm.spmm_pack_rows(xs) if xs_packed else xs
    X = held(P.q.cpu().numpy(), P.scale.cpu().numpy()) if xs_packed else f64(xs)
    need = spmm.spmm_experts_gated_grad_workspace_size(R, N, K, xs_packed) - (n * K * 2 if xs_packed else 0)
    assert need >= 2 * E * 2 * N * K * 4
    ws = torch.full((need + n * K * 2,), 255, dtype=torch.uint8, device="cuda")  # NaN everywhere
    dgu, dxs, dW = spmm.spmm_experts_gated_grad(R, dh, P, W, gu, workspace=ws)
    D = f64(dgu)
    dw, dwm = np.zeros((E, 2 * N, K)), np.zeros((E, 2 * N, K))
    for e in range(E):
        a, b = offsets[e], offsets[e + 1]
        dw[e], dwm[e] = D[a:b].T @ X[a:b], np.abs(D[a:b]).T @ np.abs(X[a:b])
    check(dW, dw, dwm, max(counts), dtype, "dW")
    assert torch.equal(dxs, spmm.spmm_experts_dx(R, dgu, W))
    for _ in range(2):
        assert torch.equal(spmm.spmm_experts_gated_grad(R, dh, P, W, gu)[2], dW)
    torch.cuda.synchronize()
    assert spmm.last_device_error() == 0
