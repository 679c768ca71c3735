"""The orthogonalisation of matrices whose norm is below eps, so that X = x / (norm(x)
+ eps) is far below 1: the result is as exact, measured by its own size, as that of
any other matrix.

A matrix is kept under a power of two of its own.  With t such that |X| lies in
(2^-(t + 1), 2^-t], singular values of the X of step i are at most 2^-t q_0 .. q_(i-1)
(q_j the largest |a + b s^2 + c s^4| over all that the step may meet), whose next
power of two is the exponent's: at most 4 |X| q_0 .. q_(i-1).  Half of float16's last
step, 2^-25 under 2^14, is so 2^-37 of |X| q_0 .. q_(i-1), which is what `halved` of
ortho_forms.py allows for a `top` of that; A's and B's bounds are squares, 16 and 32
times what they might be, and are given 9 times it (3 times the top), and 8 more.
"""
import pytest

from tests import operator_bounds as ob
from tests import ortho_forms as of

pytestmark = pytest.mark.gpu

COEFFICIENTS = (3.4445, -4.7750, 2.0315)
OTHERS = [(4.0, -6.0, 3.0), (3.0, -3.5, 1.5), (1.875, -1.25, 0.375), (1.5, -0.5, 0.0)]
EPS = 1e-7
SIZES = [(40, 50), (96, 160), (160, 96), (130, 200), (300, 257), (64, 1300)]


@pytest.fixture(scope="module")
def env():
    import torch
    from collective_communication_ring_amd import api
    assert torch.cuda.is_available(), "GPU tests need a GPU"
    api.lib()
    return dict(torch=torch, api=api, dev=torch.device("cuda:0"))


def _matrix(env, m, n, norm, seed):
    torch = env["torch"]
    x = torch.randn((m, n), generator=torch.Generator().manual_seed(seed), dtype=torch.float64)
    return (x * (norm / float(x.norm()))).float().bfloat16().float()


def _call(env, x, k, ks, eps, **more):
    torch, api, dev = env["torch"], env["api"], env["dev"]
    y = torch.empty_like(x, device=dev)
    api.orthogonalize(x.to(dev), y, k, ks[:k], eps, **more)
    torch.cuda.synchronize()
    return y.cpu()


def _own_tops(x, ks, eps):
    """Each step's largest singular value and |b s^2 + c s^4|, for this matrix."""
    grown = float(of.start(x, eps).norm())
    out = []
    for (top, mid), (a, b, c) in zip(of.tops(ks), ks):
        q = max(abs(a + b * s ** 2 + c * s ** 4) for s in (top * k / 2000 for k in range(2001)))
        out.append((min(top, 3 * grown), min(mid, 8 * 9 * grown ** 2 * max(abs(b), abs(b + c * top * top)))))
        grown *= q
    return out


@pytest.mark.parametrize("m,n", SIZES)
@pytest.mark.parametrize("small", (0.6, 0.03, 1e-2, 1e-4, 1e-6, 1e-9))
def test_step_by_step(env, m, n, small):
    """Each step against the form of a step from the one before, element by element."""
    for eps, ks in ((EPS, [COEFFICIENTS] * 5), (0.01, OTHERS)):
        x = _matrix(env, m, n, small * eps, m)
        tops, y = _own_tops(x, ks, eps), of.start(x, eps)
        y = y.t() if m > n else y
        for k in range(len(ks)):
            value, slack = of.step(y, 2.0 ** -24 * y.abs() if k else 0 * y, ks[k], *tops[k])
            if small <= 1e-4:  # then it is a few roundings; the sums' worst cases are left out
                assert float(slack.norm()) < 1e-6 * float(value.norm())
            got = _call(env, x, k + 1, ks, eps)
            got = got.t() if m > n else got
            ob.between(got, value, 1.001 * slack, (m, n, small, k))
            y = got.double()


@pytest.mark.parametrize("m,n", [(900, 1200), (1500, 1000)])
@pytest.mark.parametrize("small", (1e-2, 1e-4, 1e-6, 1e-9))
def test_by_groups(env, m, n, small):
    """Steps by groups: the 2-norm of all errors of each group after the one before."""
    ks = [COEFFICIENTS] * 5
    x = _matrix(env, m, n, small * EPS, 3)
    before, i = of.start(x, EPS), 0
    for group in of.groups_of(m, n, ks, 16.0):
        got = _call(env, x, i + group, ks, EPS).double()
        value = of.steps_of(before, ks[i:i + group])
        error, bound = float((got - value).norm()), of.group_error(before, ks[i:i + group])
        assert bound < 0.01 * float(value.norm())
        assert error <= bound, (error, bound, float(value.norm()))
        before, i = got, i + group


@pytest.mark.parametrize("m,n", [(40, 50), (130, 200), (1000, 1400)])
def test_direction_is_kept(env, m, n):
    """Five steps far below eps multiply by a^5: what the steps lose of it, a 2-norm
    of 5 (2^-22 + 2^-24 + 2^-23) of the result's by `halved` and a step's last
    operation, twice as much for a step's other products, for float32 and bfloat16."""
    torch = env["torch"]
    for small in (1e-4, 1e-6, 1e-9):
        x = _matrix(env, m, n, small * EPS, 7)
        value = of.orthogonalize(x, 5, COEFFICIENTS, EPS)
        got = _call(env, x, 5, [COEFFICIENTS] * 5, EPS)
        lost = 2 * 5 * (2.0 ** -22 + 2.0 ** -24 + 2.0 ** -23) * float(value.norm())
        assert float((got.double() - value).norm()) <= lost
        half = _call(env, x.bfloat16(), 5, [COEFFICIENTS] * 5, EPS)
        assert float((half.double() - value).norm()) <= lost + 2.0 ** -8 * float(value.norm())


@pytest.mark.parametrize("m,n", [(33, 70), (200, 140), (900, 1200)])
def test_matrices_of_other_sizes_beside(env, m, n):
    """Each matrix has a power of its own: those of one call as each by itself.  (The
    order of sums may depend on the number of matrices; here it does by groups, where
    each of the two is within the bound.)"""
    torch, api, dev = env["torch"], env["api"], env["dev"]
    x = torch.stack([_matrix(env, m, n, by, k) for k, by in enumerate((3.0, 1e-9, 1e-12, 0.0, 1e-16))]).to(dev)
    want = torch.empty_like(x)
    for a, b in zip(x, want):
        api.orthogonalize(a, b, 2)
    y = torch.empty_like(x)
    api.orthogonalize(x, y, 2)
    torch.cuda.synchronize()
    assert bool((y[3] == 0).all()) and all(bool((y[k] != 0).any()) for k in (1, 2, 4))
    if not of.by_groups(m, n):
        assert torch.equal(y, want)
    for a, b, c in zip(x, y, want):
        bound = of.group_error(of.start(a.cpu(), EPS), [COEFFICIENTS] * 2)
        assert float((b - c).norm()) <= 2 * bound


def test_steps_that_shrink(env):
    """Coefficients below 1, the last ones above: the bound's power falls and rises."""
    ks = [(0.25, 0.0, 0.0), (0.125, -0.1, 0.0), (2.0, -1.0, 0.5), (30.0, -3.0, 1.0)]
    for m, n in ((40, 50), (130, 200)):
        for small in (3e7, 1e-3, 1e-8):
            x = _matrix(env, m, n, small * EPS, 5)
            tops, y = _own_tops(x, ks, EPS), of.start(x, EPS)
            for k in range(4):
                value, slack = of.step(y, 2.0 ** -24 * y.abs() if k else 0 * y, ks[k], *tops[k])
                got = _call(env, x, k + 1, ks, EPS)
                ob.between(got, value, 1.001 * slack, (m, n, small, k))
                y = got.double()
