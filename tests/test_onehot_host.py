"""What the one-hot wrappers do on the host, without a GPU."""
import inspect
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
