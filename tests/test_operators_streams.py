"""The operators' own temporary memory belongs to the stream they run on."""
import contextlib
from types import SimpleNamespace

import pytest
import torch


def test_backward_workspace_is_allocated_on_the_given_stream(monkeypatch):
    """Without a GPU: which stream is current when the workspace that the call
    makes for itself is allocated, and that the kernels get that stream."""
    from collective_communication_ring_amd import api
    current, seen = ["the current one"], []

    @contextlib.contextmanager
    def on(stream):
        current.append(stream)
        yield
        current.pop()

    def allocate(*size):
        seen.append((current[-1], size))
        return SimpleNamespace(record_stream=lambda s: None)

    def marshal(*args):
        seen.append(args[-1])
        return api.AR_SUCCESS
    monkeypatch.setattr(torch.cuda, "stream", on)
    monkeypatch.setattr(api, "rmsnorm_backward_workspace", allocate)
    monkeypatch.setattr(api, "_bound", (SimpleNamespace(rmsnorm_backward=marshal), None))
    x, w, r, dw = torch.zeros(6, 8), torch.zeros(8), torch.zeros(6), torch.zeros(2, 8)
    given = SimpleNamespace(cuda_stream=77)
    api.rmsnorm_backward(x, x, w, r, x.clone(), dw, stream=given)
    assert seen == [(given, (2, 6, 8, x.device)), 77]
    del seen[:]
    api.rmsnorm_backward(x, x, w, r, x.clone(), dw)
    assert seen[0] == ("the current one", (2, 6, 8, x.device))


@pytest.mark.gpu
def test_backward_on_a_stream_beside_pending_work():
    """A block of the workspace's size, freed on the current stream while work
    on it is still queued there, and the backward pass on another stream: both
    come out whole."""
    from collective_communication_ring_amd import api
    dev = torch.device("cuda:0")
    rows, cols = 2048, 1024
    g = torch.Generator(device=dev).manual_seed(5)
    dy, x = (torch.randn((rows, cols), generator=g, device=dev) for _ in range(2))
    w, rstd = torch.rand(cols, generator=g, device=dev) + 0.5, torch.rand(rows, generator=g, device=dev)
    want_dx, want_dw = torch.empty_like(x), torch.empty((1, cols), device=dev)
    api.rmsnorm_backward(dy, x, w, rstd, want_dx, want_dw)
    nbytes = api.rmsnorm_backward_workspace(1, rows, cols).numel()
    side = torch.cuda.Stream()
    kept = torch.empty(nbytes, dtype=torch.uint8, device=dev)
    dx, dw = torch.empty_like(x), torch.empty_like(want_dw)
    for _ in range(3):
        torch.cuda.synchronize()
        block = torch.empty(nbytes, dtype=torch.uint8, device=dev)
        block.fill_(7)
        torch.cuda._sleep(20_000_000)
        kept.copy_(block)
        del block
        api.rmsnorm_backward(dy, x, w, rstd, dx, dw, stream=side)
        torch.cuda.synchronize()
        assert bool((kept == 7).all())
        assert torch.equal(dx, want_dx) and torch.equal(dw, want_dw)
