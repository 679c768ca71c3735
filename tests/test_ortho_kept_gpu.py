"""How the orthogonalisation keeps a matrix: an element to 2^-23 of itself or 2^-37 of
the norm, for rows and columns of any sizes side by side.

A step of coefficients (1, 0, 0) gives X back as it was kept.  On the way an element is
rounded to float32 (2^-24 of it), to two halves (2^-23 of it, or half of float16's last
step, 2^-25 under an exponent that leaves the norm above 2^12: 2^-37 of it), and as
their sum (2^-24)."""
import pytest

pytestmark = pytest.mark.gpu

SIZES = [(40, 50), (96, 160), (257, 300), (256, 512), (700, 120), (1000, 1400)]


@pytest.mark.parametrize("m,n", SIZES)
@pytest.mark.parametrize("norm,eps", [(3.0, 1e-7), (1e-9, 1e-7), (1e-30, 1e-3)])
@pytest.mark.parametrize("by", ("rows", "columns", "both"))
def test_elements_of_any_size(m, n, norm, eps, by):
    import torch
    from collective_communication_ring_amd import api
    g = torch.Generator().manual_seed(m)
    x = torch.randn((m, n), generator=g, dtype=torch.float64)
    if by != "columns":
        x *= 10.0 ** (-8 * torch.rand((m, 1), generator=g, dtype=torch.float64))
    if by != "rows":
        x *= 10.0 ** (-8 * torch.rand((1, n), generator=g, dtype=torch.float64))
    x = (x * (norm / float(x.norm()))).float()
    want = x.double() / (x.double().norm() + eps)
    y = torch.empty((m, n), device="cuda")
    api.orthogonalize(x.cuda(), y, 1, (1.0, 0.0, 0.0), eps)
    torch.cuda.synchronize()
    off = (y.cpu().double() - want).abs()
    assert bool((off <= 2.0 ** -22 * want.abs() + 2.0 ** -37 * float(want.norm())).all())


def test_small_rows_after_five_steps():
    """256 x 512, a row in four 1e-6 of the others.  An element is kept to 2^-38 (half of
    2^-24 under 2^13), a small row of norm 7.2e-8 so to sqrt(512) 2^-38, 1.15e-3 of it; a
    step makes 3.4 times of the row and of that, and adds as much again: 1.4 times in all."""
    import torch
    from collective_communication_ring_amd import api
    from tests import ortho_forms as of
    x = torch.randn((256, 512), generator=torch.Generator().manual_seed(1))
    x[::4] *= 1e-6
    want = of.orthogonalize(x, 5, (3.4445, -4.7750, 2.0315), 1e-7)
    y = torch.empty((256, 512), device="cuda")
    api.orthogonalize(x.cuda(), y)
    torch.cuda.synchronize()
    off = y.cpu().double() - want
    assert float(off[::4].norm()) <= 1.4 * 1.15e-3 * float(want[::4].norm())
