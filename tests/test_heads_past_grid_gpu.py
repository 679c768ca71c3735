"""As many heads as take more than 2^32 threads: those of one launch and those of the
next.  (184 GB, rotated in place; 2^30 heads of 86 elements, 8 threads each, by two.)"""
import pytest
import torch

from tests import head_forms as hf
from tests import operator_bounds as ob

pytestmark = pytest.mark.gpu


def test_past_one_launch():
    from collective_communication_ring_amd import api
    B, S, D = 1 << 15, (1 << 15) + 1, 86
    torch.cuda.empty_cache()
    if torch.cuda.mem_get_info()[0] < B * S * D * 2 + (8 << 30):
        pytest.skip("needs 193 GB of the GPU's memory")
    x = torch.empty((B, S, 1, D), dtype=torch.bfloat16, device="cuda")
    positions, turn = torch.arange(S, device="cuda"), api.Rotation(D, device="cuda")
    # launches of 2^23 workgroups of 4 waves, 2 rounds of 8 heads: 2^29 heads
    rows = [0, 1, (1 << 29) - 1, 1 << 29, (1 << 29) + 1, (1 << 30) - 1, 1 << 30, B * S - 2, B * S - 1]
    host = torch.randn((len(rows), 1, 1, D), generator=torch.Generator().manual_seed(2)).bfloat16()
    flat = x.view(B * S, 1, 1, D)
    for r, h in zip(rows, host):
        flat[r] = h.cuda()
    api.rotary(x, positions, turn, x)
    torch.cuda.synchronize()
    at = torch.tensor([[r % S] for r in rows])
    value, slack = hf.rotary(host, hf.table(at, turn.frequencies.cpu(), 1.0), "halves")
    ob.between(torch.stack([flat[r] for r in rows]), value, slack, "past one launch")
    del x, flat
    torch.cuda.empty_cache()
