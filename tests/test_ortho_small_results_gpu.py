"""Results of the orthogonalisation near the small end of float32's range, by a small
scale or a norm far below eps, are as exact as any others.

Two steps (a, b, c) = (1.9, -1.4, 0.5), whose polynomial is 1 at 1, of matrices of norm
3 or far below eps, against 64 bits in the 2-norm.  With s = 2^-22 + 2^-24 for keeping a
matrix, l(K) = 2^-22 + 3 K 2^-23 for a product of K columns (ortho_forms.py), and norms
of X, A and b A + c A A of at most 1, a step is off by
    A   3 s + l(n)                          (both operands, the sums, keeping it)
    B   |b| dA + |c| (2 dA + l(m)) + 2 s
    X   |a| s + dB + 2 s + l(m)
and two by 1 + 1.9 times that.  Far below eps only |a| X is left: (s + 2^-23) a step,
twice that for the rest.  An element in the subnormal range is rounded to 2^-150
besides, bfloat16 (eps 2^-7) to 2^-8 of itself or 2^-134.  (A factor of the products that is
subnormal itself loses its bits: 3e-5 of a result with a scale of 1e-33, 3% with 1e-36.)"""
import pytest

pytestmark = pytest.mark.gpu

K = (1.9, -1.4, 0.5)


def _two_steps(x, eps, scale):
    import torch
    y = x.double() / (x.double().norm() + eps)
    y = y.t() if y.shape[0] > y.shape[1] else y
    for _ in range(2):
        A = y @ y.t()
        y = K[0] * y + (K[1] * A + K[2] * A @ A) @ y
    y = y * float(torch.tensor(scale, dtype=torch.float32))
    return y.t() if x.shape[0] > x.shape[1] else y


@pytest.mark.parametrize("m,n", [(40, 60), (130, 200), (200, 130), (1000, 1400)])
@pytest.mark.parametrize("norm,eps,scale", [
    (3.0, 1e-7, 1e-33), (3.0, 1e-7, -1e-36), (1e-37, 1.0, 1.0), (1e-34, 1.0, 1.0), (1e-30, 1e-3, 1e-9),
    (1e-37, 1e10, 1e20), (1e-36, 1e30, 1e38), (1e-12, 1e-7, 1e-30), (3.0, 1e-7, 1e37)])
def test_small_results(m, n, norm, eps, scale):
    import torch
    from collective_communication_ring_amd import api
    # one large direction, so that an element is no smaller than the norm by much
    x = torch.outer(torch.linspace(0.5, 1.5, m, dtype=torch.float64), torch.ones(n, dtype=torch.float64))
    x = x + 0.01 * torch.randn((m, n), generator=torch.Generator().manual_seed(m), dtype=torch.float64)
    x = (x * (norm / float(x.norm()))).float()
    s, l = 2.0 ** -22 + 2.0 ** -24, lambda k: 2.0 ** -22 + 3 * k * 2.0 ** -23  # noqa: E731
    dA = 3 * s + l(max(m, n))
    dB = 1.4 * dA + 0.5 * (2 * dA + l(min(m, n))) + 2 * s
    lost = 2.9 * (1.9 * s + dB + 2 * s + l(min(m, n))) if norm > eps else 2 * 2 * (s + 2.0 ** -23)
    for z, half, least in ((x, 0.0, 2.0 ** -150), (x.bfloat16(), 2.0 ** -8, 2.0 ** -134)):
        want = _two_steps(z, eps, scale)
        y = torch.empty((m, n), device="cuda", dtype=z.dtype)
        api.orthogonalize(z.cuda(), y, 2, K, eps, scale)
        torch.cuda.synchronize()
        off, size = float((y.cpu().double() - want).norm()), float(want.norm())
        assert off <= 1.01 * (lost + half) * size + least * (m * n) ** 0.5, (z.dtype, off, size)


@pytest.mark.parametrize("m,n", [(40, 60), (130, 200)])
@pytest.mark.parametrize("small", (1e-30, 1e-33, 1e-36))
@pytest.mark.parametrize("scale", (1.0, 1e10, 1e-4))
def test_small_coefficients(m, n, small, scale):
    """The last step's coefficients make the result small.  It is at least half of |a|
    |X| here (0.9 and more), so the bound above, divided by 1.9 and doubled, is one
    relative to the result."""
    import torch
    from collective_communication_ring_amd import api
    x = torch.randn((m, n), generator=torch.Generator().manual_seed(m))
    k = [float(torch.tensor(v * small)) for v in K]
    y = torch.empty((m, n), device="cuda")
    for ks in ([k], [list(K), k]):
        want = x.double() / (x.double().norm() + 1e-7)
        for a, b, c in ks:
            A = want @ want.t()
            want = a * want + (b * A + c * A @ A) @ want
        want = want * float(torch.tensor(scale))
        api.orthogonalize(x.cuda(), y, len(ks), ks, 1e-7, scale)
        torch.cuda.synchronize()
        s, l = 2.0 ** -22 + 2.0 ** -24, lambda k: 2.0 ** -22 + 3 * k * 2.0 ** -23  # noqa: E731
        dA = 3 * s + l(n)
        dB = 1.4 * dA + 0.5 * (2 * dA + l(m)) + 2 * s
        lost = 2.9 * (1.9 * s + dB + 2 * s + l(m)) / 1.9 * 2
        off, size = float((y.cpu().double() - want).norm()), float(want.norm())
        assert off <= 1.01 * lost * size + 2.0 ** -150 * (m * n) ** 0.5, (ks, off / size, lost)
