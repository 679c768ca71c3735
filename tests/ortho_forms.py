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


def by_groups(rows, cols):
    m, n = sorted((rows, cols))
    return 10 * n >= 13 * m and m * n >= 1 << 20


def groups_of(rows, cols, coefficients, most):
    """The groups in which steps of a large wide or tall matrix are taken: up to three,
    while what they make of an error of A stays below `most` times it."""
    m, n = sorted((rows, cols))
    steps, i, out = len(coefficients), 0, []
    top = [t for t, _ in tops(coefficients)]
    while i < steps:
        group, wide = 1, 1.0
        while by_groups(m, n) and group < 3 and i + group < steps:
            a, b, c = coefficients[i + group - 1]
            s = torch.linspace(0, top[i + group - 1], 257, dtype=D)
            wide *= float(((a + b * s ** 2 + c * s ** 4) * (a + 3 * b * s ** 2 + 5 * c * s ** 4)).abs().max())
            if wide > most:
                break
            group += 1
        out.append(group)
        i += group
    return out


def steps_of(X, part):
    """X after the steps of `part`."""
    for a, b, c in part:
        A = X @ X.t() if X.shape[0] <= X.shape[1] else X.t() @ X
        Q = b * A + c * A @ A
        X = a * X + (Q @ X if X.shape[0] <= X.shape[1] else X @ Q)
    return X


def group_error(X, part):
    """2-norm of all elements' errors (before the last rounding) of steps `part`
    taken from X as one group: A = X X^T and Q = a I + b A + c A A, then for the next
    step A = Q (Q A), its Q, and F = Q F, at last F X.

    To first order each loss goes through what follows by itself.  A loss E of a
    matrix reaches a polynomial of it as its elements (in the basis of the matrix's
    singular vectors) times the polynomial's divided differences, so its 2-norm
    grows by |p'|'s maximum over the singular values' range, with both signs for the
    odd polynomial that the steps make of X; a loss of a factor grows by the other
    factors' largest singular values."""
    X = X.to(D)
    X = X.t() if X.shape[0] > X.shape[1] else X
    size = lambda t: float(t.norm())  # noqa: E731

    def slopes_of(v, part):  # values and slopes of s -> s q(s^2), step by step, and of prod q by s^2
        f, df = v.clone(), torch.ones_like(v)
        for a, b, c in part:
            f, df = a * f + b * f ** 3 + c * f ** 5, df * (a + 3 * b * f ** 2 + 5 * c * f ** 4)
        return f, df

    def factor_of(u, part):  # prod q as a polynomial of A, and its slope
        g, dg, l, dl = torch.ones_like(u), torch.zeros_like(u), u.clone(), torch.ones_like(u)
        for a, b, c in part:
            q, dq = a + b * l + c * l * l, (b + 2 * c * l) * dl
            g, dg = g * q, dg * q + g * dq
            l, dl = l * q * q, dl * q * q + 2 * l * q * dq
        return float(g.abs().max()), float(dg.abs().max())

    def lost(P, Q):
        return (2.0 ** -22 + 3 * P.shape[1] * 2.0 ** -23) * size(P.abs() @ Q.abs())

    def kept(V):  # in halves, whose exponent is that of a bound up to 8 times the largest
        return size(halved(V, 8 * float(torch.linalg.matrix_norm(V, 2)))) + 2.0 ** -23 * size(V)
    top = float(torch.linalg.matrix_norm(X, 2))
    out = kept(X) * float(slopes_of(torch.linspace(0, top, 4097, dtype=D), part)[1].abs().max())
    A, F, eye = X @ X.t(), None, torch.eye(len(X), dtype=D, device=X.device)
    dA, above = lost(X, X.t()), top  # above: |F X|
    for j, (a, b, c) in enumerate(part):
        u = torch.linspace(0, float(torch.linalg.matrix_norm(A, 2)), 4097, dtype=D)
        out += (dA + kept(A)) * factor_of(u, part[j:])[1] * above
        Q = a * eye + b * A + c * A @ A
        dQ = abs(c) * lost(A, A) + 2.0 ** -22 * size(A) * (abs(b) + abs(c)) + kept(Q)
        T = Q @ A
        A2 = Q @ T
        after = torch.linspace(0, float(torch.linalg.matrix_norm(A2, 2)), 4097, dtype=D)
        g, dg = factor_of(after, part[j + 1:])
        dF = dQ * above
        if F is not None:
            dF += (lost(Q, F) + kept(Q @ F)) * top
        F = Q if F is None else Q @ F
        above = float(torch.linalg.matrix_norm(F @ X, 2))
        out += dF * g
        if j + 1 < len(part):
            out += dQ * 2 * float(torch.linalg.matrix_norm(T, 2)) * dg * above
            q = float(torch.linalg.matrix_norm(Q, 2))
            dA = q * (lost(Q, A) + kept(T)) + lost(Q, T)
            A = A2
    return 1.01 * (out + lost(F, X))
