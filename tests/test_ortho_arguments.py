"""Forms of api.orthogonalize's arguments that are no lists of 2-D tensors and tuples
of numbers: taken, or a ValueError."""
import os

import numpy as np
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
        self.coefficients = a[2]
        return 0


KS = [[4.0, -6.0, 3.0], [1.5, -0.5, 0.25]]


@pytest.mark.parametrize("form", (
    tuple, list, torch.tensor, lambda k: torch.tensor(k, dtype=torch.float64), np.array,
    lambda k: [torch.tensor(v) for v in k], lambda k: tuple(np.array(v) for v in k)))
def test_coefficients(api, monkeypatch, form):
    fake = Binding()
    monkeypatch.setattr(api, "_bound", (fake, api.lib()))
    x = torch.empty((4, 5), device="meta")
    api.orthogonalize(x, x, 2, form(KS), workspace=x)
    assert fake.coefficients == KS[0] + KS[1]
    api.orthogonalize(x, x, 3, form(KS[1]), workspace=x)
    assert fake.coefficients == KS[1] * 3
    with pytest.raises(ValueError):
        api.orthogonalize(x, x, 3, form(KS), workspace=x)


def test_matrices_that_are_none(api):
    for x in (torch.zeros(3), torch.zeros(2, 3, 4), torch.zeros(())):
        with pytest.raises(ValueError):
            api.orthogonalize([x], [x])
        with pytest.raises(ValueError):
            api.orthogonalize([torch.zeros(3, 4), x], [torch.zeros(3, 4), x])
