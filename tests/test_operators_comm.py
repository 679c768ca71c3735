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
