"""Operators on tensors of another GPU than the current one, by its default stream, whose
handle is 0 on every GPU."""
import pytest
import torch

pytestmark = pytest.mark.gpu


def _calls(dev):
    """Operator -> (call, its outputs), all on `dev`."""
    from collective_communication_ring_amd import api
    g = torch.Generator().manual_seed(3)
    make = lambda *s: torch.randn(s, generator=g).to(dev)  # noqa: E731
    x, q, dy, w, big = make(5, 64), make(7, 3, 64), make(7, 3, 64), make(64), make(70, 90)
    turn, at = api.Rotation(64, device=dev), torch.arange(7, device=dev)
    y, rstd, dx, dw = torch.empty_like(x), torch.empty(5, device=dev), torch.empty_like(x), torch.empty(1, 64, device=dev)
    o, n, dq, dqw, z = (torch.empty_like(t) for t in (q, q, q, dw, big))
    return [
        (lambda: api.rmsnorm(x, w, y, rstd=rstd), [y, rstd]),
        (lambda: api.rmsnorm_backward(x, x, w, rstd, dx, dw), [dx, dw]),
        (lambda: api.rotary(q, at, turn, o), [o]),
        (lambda: api.head_rmsnorm(q, w, n, positions=at, rotation=turn), [n]),
        (lambda: api.head_rmsnorm_backward(dy, q, w, dq, dqw, positions=at, rotation=turn), [dq, dqw]),
        (lambda: api.orthogonalize(big, z), [z])]


def _run(dev):
    out = []
    for call, outputs in _calls(dev):
        call()
        out += outputs
    torch.cuda.synchronize(dev)
    return [t.cpu() for t in out]


def test_current_gpu_stays():
    with torch.cuda.device(0):
        _run("cuda:0")
        assert torch.cuda.current_device() == 0


@pytest.mark.skipif(torch.cuda.device_count() < 2, reason="needs two GPUs")
def test_other_gpu():
    want = _run("cuda:0")
    with torch.cuda.device(0):
        got = _run("cuda:1")
        assert torch.cuda.current_device() == 0
    assert all(torch.equal(a, b) for a, b in zip(got, want))
