"""The communicator's operators on the host: a closed communicator, and
gradients of another GPU than its own."""
import os
from types import SimpleNamespace

import pytest
import torch


@pytest.fixture(scope="module")
def api():
    from collective_communication_ring_amd import api
    if not os.path.exists(api.LIB_PATH) or not os.path.exists(os.path.join(api.HERE, "_binding.so")):
        import __graft_entry__
        __graft_entry__.build()
    api.lib()
    return api


def _closed(api):
    """A communicator as close() leaves it, made without a GPU."""
    c = api.Comm.__new__(api.Comm)
    c.R, c.dtype, c.device, c._ws_stream = 2, api.AR_FLOAT32, torch.device("cuda:0"), 0
    c.handle = c.workspace = None
    return c


STREAM = SimpleNamespace(cuda_stream=0)


def test_reduce_scatter_norm_on_a_closed_comm(api):
    """Refused as the collectives refuse it."""
    send, w, y = torch.zeros(2, 16), torch.zeros(4), torch.zeros(2, 8)
    with pytest.raises(api.ArError) as e:
        _closed(api).reduce_scatter_rmsnorm(send, w, y, stream=STREAM)
    assert e.value.status == api.AR_ERR_INVALID_ARG


def _open(api, index):
    c = _closed(api)
    c.handle, c.workspace = 1, SimpleNamespace(get_device=lambda: index)
    c.close = lambda: None  # the handle is none of the library's
    return c


def _list(api, index):
    """A list of gradients of one GPU, made without one."""
    t = api.TensorList([])
    t.spans = lambda: t._array
    t.index = index
    return t


@pytest.mark.parametrize("norm_at,grads_at", [(1, 1), (1, 0), (0, 1), (1, -1)])
def test_gradients_of_another_gpu(api, monkeypatch, norm_at, grads_at):
    """Gradients or norm beside the communicator's GPU: refused before the call."""
    def called(*a):
        raise AssertionError("the library was called")
    monkeypatch.setattr(api, "ar_grad_norm", called)
    monkeypatch.setattr(api, "ar_grad_clip", called)
    norm = SimpleNamespace(numel=lambda: 1, dtype=torch.float32, is_cuda=True,
                           get_device=lambda: norm_at, data_ptr=lambda: 4096)
    c = _open(api, 0)
    c._stream = lambda s: 0
    for call in (lambda: c.grad_norm(_list(api, grads_at), norm),
                 lambda: c.grad_clip(_list(api, grads_at), norm, 1.0)):
        with pytest.raises(ValueError):
            call()


def test_gradients_of_the_comms_gpu_and_a_closed_comm(api, monkeypatch):
    seen = []
    monkeypatch.setattr(api, "ar_grad_norm", lambda *a: seen.append("norm"))
    monkeypatch.setattr(api, "ar_grad_clip", lambda *a: seen.append("clip"))
    norm = SimpleNamespace(numel=lambda: 1, dtype=torch.float32, is_cuda=True,
                           get_device=lambda: 1, data_ptr=lambda: 4096)
    c = _open(api, 1)
    c._stream = lambda s: 0
    for index in (1, -1):
        c.grad_norm(_list(api, index), norm)
        c.grad_clip(_list(api, index), norm, 1.0)
    assert seen == ["norm", "clip"] * 2
    monkeypatch.undo()
    with pytest.raises(api.ArError) as e:
        _closed(api).grad_norm(_list(api, 1), norm, stream=STREAM)
    assert e.value.status == api.AR_ERR_INVALID_ARG
