"""Plain 64-bit form of the Newton-Schulz orthogonalisation, with bounds.

A matrix in halves is off by 2^-22 of each element (two roundings by 2^-11),
2^-24 more (the float32 value that was halved), and 2^-38 of the largest value
its exponent allows for.  An element of a product of K columns drops the two
low halves' part, 2^-22 of the sum of |p q|, and makes 3 K additions, each off
by at most a float32 step of that sum (the matrix instructions' own rounding is
taken as either way): (2^-22 + 3 K 2^-23) |P| |Q|^T.

One step is bounded element by element so.  Errors of several steps grow (by
the polynomial's slopes, 3 and more a step), so those are taken one by one: each
step's result against the form of a step from the one before it.
"""
import torch

D = torch.float64
HALVES = 2.0 ** -22 + 2.0 ** -24


def tops(coefficients):
    """Largest singular values that the steps' start may have: 1, then by a
    fine walk over each interval; and the largest |b s^2 + c s^4|."""
    top, out = 1.0, []
    for a, b, c in coefficients:
        s = torch.linspace(0, top, 20001, dtype=D)
        mid = (b * s ** 2 + c * s ** 4).abs().max()
        out.append((top, float(mid)))
        top = float((a * s + b * s ** 3 + c * s ** 5).abs().max()) * 1.0001
    return out


def halved(x, most):
    return HALVES * x.abs() + 2.0 ** -37 * most


def product(p, q, dp, dq):
    """P Q^T and its slack."""
    lost = 2.0 ** -22 + 3 * p.shape[1] * 2.0 ** -23
    return p @ q.t(), p.abs() @ dq.t() + dp @ q.abs().t() + dp @ dq.t() + lost * (p.abs() @ q.abs().t())


def step(x, dx, coefficients, top, mid):
    """One step of X [m][n], m <= n, known to +- dx; its products' operands are
    halved."""
    a, b, c = coefficients
    dx = dx + halved(x, top)
    A, dA = product(x, x, dx, dx)
    dA = dA + halved(A, top * top)
    AA, dAA = product(A, A, dA, dA)
    B = b * A + c * AA
    dB = abs(b) * dA + abs(c) * dAA
    dB = dB + halved(B, mid) + 2.0 ** -23 * (abs(b) * A.abs() + abs(c) * AA.abs())
    BX, dBX = product(B, x.t().contiguous(), dB, dx.t().contiguous())
    y = a * x + BX
    return y, abs(a) * dx + dBX + 2.0 ** -23 * (abs(a) * x.abs() + BX.abs())


def start(x, eps):
    x = x.to(D)
    return x / (torch.sqrt((x * x).sum()) + eps)


def coefficient_list(coefficients, steps):
    return [coefficients] * steps if not hasattr(coefficients[0], "__len__") else list(coefficients)


def orthogonalize(x, steps, coefficients, eps, scale=1.0):
    tall = x.shape[0] > x.shape[1]
    y = start(x.t() if tall else x, eps)
    for a, b, c in coefficient_list(coefficients, steps):
        A = y @ y.t()
        y = a * y + (b * A + c * (A @ A)) @ y
    return scale * (y.t() if tall else y)


def one_step(x, coefficients, eps, scale=1.0):
    """(value, slack), element by element."""
    tall = x.shape[0] > x.shape[1]
    y = start(x.t() if tall else x, eps)
    y, dy = step(y, torch.zeros_like(y), coefficients, *tops([coefficients])[0])
    return scale * (y.t() if tall else y), abs(scale) * 1.001 * (dy.t() if tall else dy)


def next_step(y, k, coefficients):
    """(value, slack) of step k (from 0) from y, the float32 result of k steps."""
    ks = coefficient_list(coefficients, k + 1)
    tall = y.shape[0] > y.shape[1]
    y = (y.t() if tall else y).to(D)
    z, dz = step(y, 2.0 ** -24 * y.abs(), ks[k], *tops(ks)[k])
    return (z.t() if tall else z), 1.001 * (dz.t() if tall else dz)
