"""The workspace that api.orthogonalize makes for itself: for all matrices where that is
little, else for as many as keep the GPU busy; the call takes them in parts."""
import os

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


class Binding:
    def orthogonalize(self, *a):
        self.workspace = a[5]
        return 0


@pytest.mark.parametrize("count,m,n,room", [
    (1, 4096, 8192, 1), (128, 4096, 8192, None), (40, 4096, 4096, None), (1, 16384, 65536, 1),
    (3, 65536, 16384, 1), (12, 1024, 1024, 12), (128, 512, 512, 128), (500, 200, 200, 128)])
def test_its_size(api, monkeypatch, count, m, n, room):
    fake = Binding()
    monkeypatch.setattr(api, "_bound", (fake, api.lib()))
    monkeypatch.setattr(api, "orthogonalize_workspace",
                        lambda c, r, k, t=None, d=None: api.ar_orthogonalize_workspace(c, r, k))
    x = torch.empty((count, m, n), device="meta")
    api.orthogonalize(x, x)
    api.orthogonalize(list(x), list(x))
    f = api.ar_orthogonalize_workspace
    assert f(1, m, n) <= fake.workspace <= max(f(1, m, n), 2 << 30)
    if room:
        assert fake.workspace == f(room, m, n)
    else:  # as many as fit
        assert fake.workspace + f(2, m, n) - f(1, m, n) > 2 << 30


@pytest.mark.gpu
def test_parts(api):
    """Matrices past what the workspace holds: the bits of a call with the caller's own
    workspace of that many, and no more memory than that."""
    x = torch.randn((5, 3000, 6000), generator=torch.Generator(device="cuda").manual_seed(1), device="cuda")
    y, z = torch.empty_like(x), torch.empty_like(x)
    before = torch.cuda.memory_allocated()
    torch.cuda.reset_peak_memory_stats()
    api.orthogonalize(x, y, 2)
    torch.cuda.synchronize()
    assert torch.cuda.max_memory_allocated() - before <= 2 << 30
    f = api.ar_orthogonalize_workspace
    room = max(k for k in range(1, 6) if f(k, 3000, 6000) <= 2 << 30)
    assert 1 < room < 5
    api.orthogonalize(x, z, 2, workspace=api.orthogonalize_workspace(room, 3000, 6000))
    torch.cuda.synchronize()
    assert torch.equal(y, z)
