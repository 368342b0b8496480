"""A thread's row and features in the gradient of the activation (csrc/gated.cu): one multiplication by 2^64 / threads of a
row, then a difference modulo 2^32.  Exact for every grid that the launcher accepts, read and computed without a GPU."""
import random
import re

import pytest

from tests.test_warp_convergence import _body, _code

M32, M64 = (1 << 32) - 1, (1 << 64) - 1


def _most(per):
    """Threads that the launcher accepts: fewer than 2^31 blocks of 256, and by `per` of a row below 2^64."""
    return min(((1 << 31) - 1) * 256, M64 // per)


def test_the_arithmetic_is_unsigned():
    """A signed product overflows, which is undefined, from 2^31 threads on."""
    body = _body(_code("gated.cu"), r"gated_grad_kernel\(")
    assert not re.search(r"static_cast<int>\((p|thread)\)", body)
    assert "static_cast<uint32_t>(p) * static_cast<uint32_t>(a.N / 8)" in body
    assert "static_cast<int>(static_cast<uint32_t>(thread) - before) * 8" in body


@pytest.mark.parametrize("N", [16, 32, 48, 80, 112, 1792, 2064, (1 << 20) + 16, (1 << 26) + 32, (1 << 29) - 16])
def test_row_and_features(N):
    per = N // 8
    factor = M64 // per + 1
    rng = random.Random(N)
    rows = min(_most(per) // per, (1 << 31) - 1)
    threads = {0, 1, per - 1, per, per + 1, rows * per - 1, (1 << 31) - 1, 1 << 31, (1 << 31) + 1, (1 << 32) - 1, 1 << 32}
    threads |= {rng.randrange(rows) * per + d for _ in range(2000) for d in (0, 1, per - 1)}
    for t in threads:
        if t >= rows * per:
            continue
        p = (t * factor) >> 64
        assert p == t // per
        c = ((t & M32) - (((p & M32) * per) & M32)) & M32
        assert c == t % per and c * 8 < 1 << 31


def test_more_is_refused():
    """Before any device work: the first by its threads of a row, the second by its blocks."""
    import ctypes

    from sparse_dense_matrix_spmm_gb300 import _lib, build
    build.build()
    f, N = _lib.load().spmm_gated_grad, (1 << 29) - 16
    for rows in (6000, 1 << 15):
        R = _lib.RouteT(rows, 1, 1, 16, 16, 16, None)
        P = _lib.Rows8T(rows, 2 * N, 16, 2 * N, 16, N // 8)
        assert f(ctypes.byref(R), 16, N, None, 2 * N, ctypes.byref(P), N, 0, 0, 16, 2 * N, None, N, None) == 8


@pytest.mark.gpu
def test_more_than_two_to_the_31_threads():
    """2^34 features of h in all: the last rows are those of a small call, and what is zero stays zero."""
    from tests.gpu_util import need_gpu
    from tests.onehot_util import matrix
    torch = need_gpu()
    import sparse_dense_matrix_spmm_gb300 as spmm
    rows, N, few = 1 << 14, (1 << 20) + 16, 3
    if torch.cuda.mem_get_info()[0] + torch.cuda.memory_reserved() < 170 << 30:
        pytest.skip("needs 150 GB of device memory")
    torch.cuda.empty_cache()
    dh = torch.zeros(rows, N, dtype=torch.bfloat16, device="cuda")
    P = spmm.Rows8(rows, 2 * N, torch.bfloat16, torch.zeros(rows, 2 * N, dtype=torch.int8, device="cuda"),
                   torch.ones(rows, N // 8, dtype=torch.uint8, device="cuda"))
    small = matrix((few, 2 * N), "bf16", 1)
    kept = spmm.spmm_pack_rows(small)
    dh[-few:] = matrix((few, N), "bf16", 2)
    P.q[-few:], P.scale[-few:] = kept.q, kept.scale
    R = spmm.spmm_build_route(torch.zeros(rows, dtype=torch.int64, device="cuda"), 1)
    r = spmm.spmm_build_route(torch.zeros(few, dtype=torch.int64, device="cuda"), 1)
    dgu = spmm.spmm_gated_grad(R, dh, P)
    assert torch.equal(dgu[-few:], spmm.spmm_gated_grad(r, dh[-few:], kept))
    assert dgu[-few:].any() and not any(bool(part.any()) for part in dgu[:-few].split(1 << 11))
    assert spmm.last_device_error() == 0
    del dh, P, dgu
    torch.cuda.empty_cache()
