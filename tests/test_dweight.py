"""The weight's gradient over many rows, against bounds that a missing row does
not pass."""
import pytest
import torch

from tests import dweight_bounds as db
from tests import operator_bounds as ob

# ranks, rows, columns: rows side by side in a wave and in a workgroup, more
# than one turn, one workgroup a rank, all widths' kernels
SHAPES = [(1, 70000, 8), (1, 3000, 64), (1, 2500, 1000), (8, 8 * 313, 1001), (64, 64 * 40, 100),
          (1, 20000, 3), (2, 1026, 4096), (16, 16 * 7, 2049), (1, 4099, 40), (5, 5 * 700, 520),
          (1, 1030, 9001), (4, 4 * 2, 9001), (3, 3 * 170, 20001), (1, 600, 33001)]


def _inputs(ranks, rows, cols, dtype, seed=1):
    g = torch.Generator().manual_seed(seed)
    x, dy = ((torch.randn((rows, cols), generator=g) * s).to(dtype) for s in (1.5, 1.0))
    rstd = 1 / torch.sqrt((x.float() ** 2).mean(1) + 1e-6)
    w = (1 + 0.2 * torch.randn(cols, generator=g)).to(dtype)
    return dy, x, w, rstd


def _caught(got, value, slack):
    try:
        ob.between(got, value, slack, "dweight")
    except AssertionError:
        return True
    return False


@pytest.mark.parametrize("dtype", (torch.float32, torch.bfloat16))
@pytest.mark.parametrize("ranks,rows,cols", [s for s in SHAPES if s[1] * s[2] <= 1 << 22])
def test_bound_catches_a_missing_row(ranks, rows, cols, dtype):
    """The float32 rounding of the value passes; without one row, or without
    the rows of one of the workgroups, it does not."""
    dy, x, _, rstd = _inputs(ranks, rows, cols, dtype)
    value, slack = db.dweight(dy, x, rstd, ranks)
    assert not _caught(value.float(), value, slack)
    n = rows // ranks
    blocks = min(n, max(1, db.WORKGROUPS // ranks))
    for lost in ([0], [n // 2], [n - 1], list(range(n // 3, min(n, n // 3 + -(-n // blocks))))):
        d = dy.clone()
        d[lost] = 0  # of the first rank
        assert _caught(db.dweight(d, x, rstd, ranks)[0].float(), value, slack), lost
    d = dy.clone()
    d[rows - n:rows - n + 1] *= 2  # a row of the last rank counted twice
    assert _caught(db.dweight(d, x, rstd, ranks)[0].float(), value, slack)


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", (torch.float32, torch.bfloat16))
@pytest.mark.parametrize("ranks,rows,cols", SHAPES)
def test_dweight(ranks, rows, cols, dtype):
    from collective_communication_ring_amd import api
    dev = torch.device("cuda:0")
    dy, x, w, rstd = _inputs(ranks, rows, cols, dtype)
    dx, dw = torch.empty((rows, cols), dtype=dtype, device=dev), torch.full((ranks, cols), 9.0, device=dev)
    api.rmsnorm_backward(dy.to(dev), x.to(dev), w.to(dev), rstd.to(dev), dx, dw)
    torch.cuda.synchronize()
    ob.between(dw, *db.dweight(dy, x, rstd, ranks), "dweight")
    ob.between(dx, *ob.norm_backward(dy, x, w, rstd)["dx"], "dx")
