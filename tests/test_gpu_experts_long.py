"""The experts' products at depths whose one unit of work takes longer than 2 s: no
wait of the kernel may give up on it, and the sums are those of the few nonzeros."""
import pytest

from tests.gpu_util import need_gpu

pytestmark = pytest.mark.gpu


def _route(torch, spmm, n):
    """All n rows belong to the one expert; the products read nothing but the offsets."""
    i32 = torch.int32
    none = torch.zeros(1, dtype=i32, device="cuda")
    return spmm.Route(n, 1, 1, none, none, torch.tensor([0, n], dtype=i32, device="cuda"))


def _places(n):
    return [0, 63, 64, n // 2 + 5, n - 65, n - 1]


@pytest.mark.parametrize("which", ["dw", "experts", "dx"])
def test_units_of_seconds(which):
    """Small integers in a few places of the depth, zeros elsewhere: the sums are exact in every type."""
    torch = need_gpu()
    import sparse_dense_matrix_spmm_gb300 as spmm
    bf16, m = torch.bfloat16, 8
    torch.cuda.empty_cache()
    spmm.last_device_error()
    if which == "dw":
        n = 512 * 1000 * 1000 + 37                       # rows of one expert, 0.33 us per 64 of them
        R = _route(torch, spmm, n)
        a, b = (torch.zeros((n, m), dtype=bf16, device="cuda") for _ in range(2))
        want = torch.zeros((1, m, m))
        for i, p in enumerate(_places(n)):
            a[p, i % m], b[p, (3 * i + 1) % m] = i + 1, 2
            want[0, i % m, (3 * i + 1) % m] += 2 * (i + 1)
        got = spmm.spmm_experts_dw(R, a, b)
    else:
        K, n = 600 * 1000 * 1000 + 8, 17                 # the depth, 0.26 us per 64
        R = _route(torch, spmm, n)
        a = torch.zeros((n, K), dtype=bf16, device="cuda")
        W = torch.zeros((1, m, K) if which == "experts" else (1, K, m), dtype=bf16, device="cuda")
        want = torch.zeros((n, m))
        for i, p in enumerate(_places(K)):
            a[i * 3 % n, p] = i + 1
            if which == "experts":
                W[0, i % m, p] = 2
            else:
                W[0, p, i % m] = 2
            want[i * 3 % n, i % m] += 2 * (i + 1)
        got = spmm.spmm_experts(R, a, W) if which == "experts" else spmm.spmm_experts_dx(R, a, W)
    torch.cuda.synchronize()
    assert spmm.last_device_error() == 0
    assert torch.equal(got.float().cpu(), want)
