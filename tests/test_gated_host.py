"""What the gated experts' wrappers refuse on the host, without a GPU."""
import copy
import inspect
from types import SimpleNamespace

import pytest
import torch

import sparse_dense_matrix_spmm_gb300 as spmm


def _cuda(shape, dtype=torch.bfloat16, stride=None):
    """Looks like a CUDA tensor to the checks; no memory behind it."""
    t = torch.empty(shape, dtype=dtype, device="meta")
    t = t if stride is None else t.as_strided(shape, stride)
    dev = torch.device("cuda", 0)
    return SimpleNamespace(shape=t.shape, dtype=dtype, device=dev, is_cuda=True, stride=t.stride, numel=t.numel, dim=t.dim,
                           is_contiguous=t.is_contiguous, data_ptr=lambda: 256)


def _R(T=5, k=2, E=3):
    return SimpleNamespace(T=T, k=k, n_keys=E, n_rows=T * k, device=torch.device("cuda", 0), shape=(T, k), _ref=None)


def test_every_wrapper_asks_for_the_handle():
    for f in (spmm.spmm_topk, spmm.spmm_topk_grad, spmm.spmm_pack_rows, spmm.spmm_unpack_rows, spmm.spmm_experts_gated,
              spmm.spmm_gated_grad, spmm.spmm_experts_gated_grad):
        assert "_handle(stream, " in inspect.getsource(f), f.__name__


def test_host_tensors_are_refused():
    x = torch.zeros(4, 16)
    for f in (lambda: spmm.spmm_topk(x, 2), lambda: spmm.spmm_pack_rows(x),
              lambda: spmm.Rows8(4, 16, x.dtype, x.to(torch.int8), x[:, :1].to(torch.uint8))):
        with pytest.raises(ValueError, match="no CPU path"):
            f()


def test_topk_arguments():
    x = _cuda((4, 16))
    for k in (0, 17, -1):
        with pytest.raises(ValueError, match="k must be"):
            spmm.spmm_topk(x, k)
    with pytest.raises(TypeError, match="int32 or int64"):
        spmm.spmm_topk(x, 2, id_dtype=torch.int16)
    with pytest.raises(TypeError, match="row dtype"):
        spmm.spmm_topk(_cuda((4, 16), torch.int8), 2)
    with pytest.raises(ValueError, match="contiguous rows"):
        spmm.spmm_topk(_cuda((4, 16), stride=(1, 4)), 2)
    ids, w = _cuda((4, 2), torch.int64), _cuda((4, 2), torch.float32)
    with pytest.raises(ValueError, match="ids must be"):
        spmm.spmm_topk_grad(x, _cuda((3, 2), torch.int64), w, w)
    with pytest.raises(TypeError, match="dw must be float32"):
        spmm.spmm_topk_grad(x, ids, w, _cuda((4, 2)))
    with pytest.raises(ValueError, match="w must be a contiguous"):
        spmm.spmm_topk_grad(x, ids, _cuda((4, 3), torch.float32), w)
    with pytest.raises(ValueError, match="out must be"):
        spmm.spmm_topk_grad(x, ids, w, w, out=_cuda((4, 15)))


def test_rows8_arguments():
    q, s = _cuda((4, 40), torch.int8), _cuda((4, 3), torch.uint8)
    c = spmm.Rows8(4, 40, torch.bfloat16, q, s).c()
    assert (c.rows, c.cols, c.ldq, c.lds) == (4, 40, 40, 3)
    c = spmm.Rows8(1, 40, torch.bfloat16, _cuda((1, 40), torch.int8), _cuda((1, 3), torch.uint8)).c()
    assert (c.ldq, c.lds) == (48, 3)
    for cols, q1, s1 in ((40, q, _cuda((4, 2), torch.uint8)), (41, q, s), (40, _cuda((4, 40), torch.uint8), s),
                         (40, _cuda((4, 40), torch.int8, (1, 4)), s), (40, q, _cuda((4, 3), torch.uint8, (1, 4)))):
        with pytest.raises(ValueError, match="must"):
            spmm.Rows8(4, cols, torch.bfloat16, q1, s1)
    with pytest.raises(ValueError, match="out must hold"):
        spmm.spmm_pack_rows(_cuda((4, 39)), spmm.Rows8(4, 40, torch.bfloat16, q, s))


@pytest.mark.parametrize("name", ["rows", "cols", "dtype", "q", "scale", "device"])
def test_rows8_fields_cannot_be_replaced(name):
    """The C struct holds the tensors' addresses: a replaced tensor would leave the kernels on freed memory."""
    P = spmm.Rows8(4, 40, torch.bfloat16, _cuda((4, 40), torch.int8, (48, 1)), _cuda((4, 3), torch.uint8))
    before = getattr(P, name)
    with pytest.raises(AttributeError, match="addresses"):
        setattr(P, name, before)
    with pytest.raises(AttributeError, match="addresses"):
        delattr(P, name)
    c = copy.copy(P)
    assert getattr(c, name) is before and c._ref is not P._ref and (c.c().ldq, c.c().lds, c.c().q) == (48, 3, 256)


def test_gated_arguments():
    R, xs, W = _R(), _cuda((10, 64)), _cuda((3, 96, 64))
    with pytest.raises(ValueError, match="act must be one of"):
        spmm.spmm_experts_gated(R, xs, W, act="relu")
    with pytest.raises(ValueError, match="save must be"):
        spmm.spmm_experts_gated(R, xs, W, save="fp8")
    with pytest.raises(ValueError, match="W must be"):
        spmm.spmm_experts_gated(R, xs, _cuda((3, 97, 64)))  # an odd number of weight rows
    with pytest.raises(ValueError, match="W must be"):
        spmm.spmm_experts_gated(R, xs, _cuda((4, 96, 64)))
    with pytest.raises(TypeError, match="W must be"):
        spmm.spmm_experts_gated(R, xs, _cuda((3, 96, 64), torch.float16))
    with pytest.raises(ValueError, match="xs must be"):
        spmm.spmm_experts_gated(R, _cuda((9, 64)), W)
    dh = _cuda((10, 48))
    with pytest.raises(ValueError, match="gu must be"):
        spmm.spmm_gated_grad(R, dh, _cuda((10, 48)))
    with pytest.raises(ValueError, match="gu must hold"):
        spmm.spmm_gated_grad(R, dh, spmm.Rows8(10, 48, torch.bfloat16, _cuda((10, 48), torch.int8), _cuda((10, 3), torch.uint8)))
    with pytest.raises(TypeError, match="gu must be"):
        spmm.spmm_gated_grad(R, dh, _cuda((10, 96), torch.float16))
    gu = _cuda((10, 96))
    with pytest.raises(ValueError, match="xs must be"):
        spmm.spmm_experts_gated_grad(R, dh, _cuda((10, 63)), W, gu)
    with pytest.raises(ValueError, match="xs must hold"):
        spmm.spmm_experts_gated_grad(R, dh, spmm.Rows8(10, 48, torch.bfloat16, _cuda((10, 48), torch.int8), _cuda((10, 3), torch.uint8)),
                                     W, gu)
    with pytest.raises(ValueError, match="W must be"):
        spmm.spmm_experts_gated_grad(R, dh, xs, _cuda((3, 80, 64)), gu)
    with pytest.raises(ValueError, match="gu must be"):
        spmm.spmm_experts_gated_grad(R, dh, xs, W, _cuda((10, 64)))
