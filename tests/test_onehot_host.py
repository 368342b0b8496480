"""What the one-hot wrappers do on the host, without a GPU."""
import copy
import ctypes
import inspect
import pickle
from types import SimpleNamespace

import pytest
import torch

import sparse_dense_matrix_spmm_gb300 as spmm


def test_calls_on_another_device_are_refused(monkeypatch):
    """A launch goes to the current device: operands or a stream of another one raise before it."""
    monkeypatch.setattr(torch._C, "_cuda_getDevice", lambda: 0, raising=False)
    monkeypatch.setattr(torch._C, "_cuda_getCurrentRawStream", lambda d: 100 + d, raising=False)
    here, there = torch.device("cuda", 0), torch.device("cuda", 1)
    assert spmm._handle(None, here) == 100
    assert spmm._handle(SimpleNamespace(device_index=0, cuda_stream=7), here) == 7
    with pytest.raises(ValueError, match="current device is cuda:0"):
        spmm._handle(None, there)
    with pytest.raises(ValueError, match="operands are on cuda:1"):
        spmm._handle(SimpleNamespace(device_index=1, cuda_stream=7), there)
    with pytest.raises(ValueError, match="stream belongs to cuda:1"):
        spmm._handle(SimpleNamespace(device_index=1, cuda_stream=7), here)


def test_every_wrapper_asks_for_the_handle():
    for f in (spmm.spmm_build_route, spmm.spmm_dispatch, spmm.spmm_combine, spmm.spmm_combine_grad, spmm.spmm_embed,
              spmm.spmm_embed_grad, spmm.spmm_experts, spmm.spmm_experts_dx, spmm.spmm_experts_dw):
        assert "_handle(stream, " in inspect.getsource(f), f.__name__


def _route(keys=True):
    i32 = torch.int32
    return spmm.Route(5, 1, 3, torch.arange(5, dtype=i32), torch.arange(5, dtype=i32),
                      torch.tensor([0, 2, 3, 5], dtype=i32), torch.zeros(5, dtype=i32) if keys else None)


def _holds_its_own(R):
    c = R.c()
    assert (c.T, c.k, c.n_keys) == (R.T, R.k, R.n_keys) and R.n_rows == R.T * R.k
    assert c.order == R.order.data_ptr() and c.pos == R.pos.data_ptr() and c.offsets == R.offsets.data_ptr()
    assert c.keys == (None if R.keys is None else R.keys.data_ptr())


@pytest.mark.parametrize("name", ["T", "k", "n_keys", "n_rows", "order", "pos", "offsets", "keys", "device", "shape"])
def test_route_fields_cannot_be_replaced(name):
    """The C struct holds the tensors' addresses: a replaced tensor would leave the kernels on freed memory."""
    R = _route()
    _holds_its_own(R)
    before = getattr(R, name)
    with pytest.raises(AttributeError, match="does not change"):
        setattr(R, name, before)
    with pytest.raises(AttributeError, match="does not change"):
        delattr(R, name)
    assert getattr(R, name) is before
    _holds_its_own(R)


@pytest.mark.parametrize("keys", [True, False])
def test_routes_are_copied_with_structs_of_their_own(keys):
    R = _route(keys)
    shallow, deep, thawed = copy.copy(R), copy.deepcopy(R), pickle.loads(pickle.dumps(R))
    for S in (shallow, deep, thawed):
        _holds_its_own(S)
        assert torch.equal(S.order, R.order) and torch.equal(S.pos, R.pos) and torch.equal(S.offsets, R.offsets)
        assert S.shape == R.shape and S.device == R.device
    assert shallow.pos is R.pos
    assert deep.pos.data_ptr() != R.pos.data_ptr() and thawed.pos.data_ptr() != R.pos.data_ptr()


def test_combine_grad_of_rows_without_columns_is_accepted():
    """As spmm_dispatch and spmm_combine accept them.  Without tokens nothing is launched."""
    from sparse_dense_matrix_spmm_gb300 import build
    build.build()
    L = spmm._lib.load()
    R = ctypes.byref(spmm._lib.RouteT(0, 2, 4, 16, 16, 16, 16))
    assert L.spmm_combine_grad(R, None, 0, None, 0, 16, None, 0, 16, 0, 0, None) == 0
    assert L.spmm_combine_grad(R, None, 0, None, 0, 16, None, 0, 16, -1, 0, None) == 2
    R = ctypes.byref(spmm._lib.RouteT(3, 2, 4, 16, 16, 16, 16))
    assert L.spmm_combine_grad(R, None, 0, None, 0, None, None, 0, 16, 0, 0, None) == 1   # w
    assert L.spmm_combine_grad(R, None, 0, None, 0, 16, None, 0, None, 0, 0, None) == 1   # dw
    assert L.spmm_combine_grad(R, None, 8, 16, 8, 16, 16, 8, 16, 8, 0, None) == 1         # dy, with columns


def test_more_choices_than_32_bits_are_refused():
    """2^32 + 5 choices of one token must not become 5."""
    for k in (1 << 31, (1 << 32) + 5):
        with pytest.raises(spmm.SpmmError, match="UNSUPPORTED"):
            spmm.spmm_build_route_workspace_size(1, k, 4)
    ids = SimpleNamespace(is_cuda=True, dtype=torch.int32, shape=(1, (1 << 32) + 5), stride=lambda d: 1)
    with pytest.raises(spmm.SpmmError, match="UNSUPPORTED"):
        spmm.spmm_build_route(ids, 4)
