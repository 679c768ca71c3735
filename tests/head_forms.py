"""Plain 64-bit forms of the operators on attention heads, with bounds.

(value, slack) pairs in float64, as operator_bounds.py's: a correct float32
computation lies within value +- slack before its last rounding.  U = 2^-24 is
half a float32 step.  Where the slacks come from:

  cosine and sine  the angle in 64 bits, off by 4 * 2^-53 of it; less whole
                   quarter turns it is at most pi / 4, and its rounding to
                   float32 moves a sine by at most 0.79 U and a cosine by 0.56
                   U; the series' first missing term is below 2e-9 (0.04 U);
                   its last addition rounds by U of at most 1, the square below
                   it by 0.31 U, the rest by 0.25 U: 2.2 U together
  the factor       one rounding
  a rotated value  c a - s b: one rounding of s b, one of the result
  sums of a head   16 values in a thread, up to 64 threads: 16 + 6 additions
"""
import torch

U = 2.0 ** -24
SLOP = 1.001  # the second-order terms
D = torch.float64
HEAD_SUM = 23


def table(positions, frequencies, factor):
    """cos and sin [batch, tokens, 1, pairs] times the factor, and their slack."""
    angle = positions.to(D)[:, :, None, None] * frequencies.to(D)
    c, s = torch.cos(angle) * factor, torch.sin(angle) * factor
    off = (2.2 * U + 4 * 2.0 ** -53 * angle.abs()) * abs(factor)
    return c, s, off + U * c.abs(), off + U * s.abs()


def turn(x, dx, t, layout, inverse=False):
    """The rotation (its transpose) of x [batch, tokens, heads, dim], known to
    +- dx."""
    c, s, dc, ds = t
    if inverse:
        s = -s
    r = 2 * c.shape[-1]
    if layout == "halves":
        first, second = slice(0, r // 2), slice(r // 2, r)
    else:
        first, second = slice(0, r, 2), slice(1, r, 2)
    y, dy = x.clone(), dx.clone()
    a, b, da, db = x[..., first], x[..., second], dx[..., first], dx[..., second]
    for to, p, q, dp, dq, sign in ((first, a, b, da, db, -1.0), (second, b, a, db, da, 1.0)):
        v = c * p + sign * s * q
        y[..., to] = v
        # either product may be the one that is rounded by itself
        dy[..., to] = (c.abs() * dp + s.abs() * dq + dc * p.abs() + ds * q.abs() +
                       U * torch.maximum((s * q).abs(), (c * p).abs()) + U * v.abs()) * SLOP
    return y, dy


def rotary(x, t, layout, inverse=False):
    x = x.to(D)
    return turn(x, torch.zeros_like(x), t, layout, inverse)


def rstd(x, eps):
    """1 / rms of heads, and its slack."""
    C = x.shape[-1]
    ss = (x * x).sum(-1, keepdim=True)
    r = 1 / torch.sqrt(ss / C + eps)
    dss = HEAD_SUM * U * ss
    return r, r * (0.5 * dss / (ss + C * eps).clamp_min(2.0 ** -1000) + 3.5 * U) * SLOP


def head_norm(x, weight, eps, t=None, layout="halves"):
    x, w = x.to(D), weight.to(D)
    r, dr = rstd(x, eps)
    v = x * r * w
    dv = (v.abs() * (dr / r) + 2 * U * v.abs()) * SLOP
    return (v, dv) if t is None else turn(v, dv, t, layout)


def additions(rows, dim):
    """How many a weight's gradient may pass through: rows of one rank and side
    go by 256 threads of 16 elements, in turns of at least 32 workgroups (as
    many as there are turns, if fewer), whose sums are then dealt to 8."""
    lanes = 1
    while lanes * 16 < dim:
        lanes *= 2
    turns = -(-rows * lanes // 256)
    return 20 + min(turns, 130 + turns // 32)


def head_norm_backward(dy, x, weight, eps, t=None, layout="halves", ranks=1):
    """dx, and dweight [ranks, dim]."""
    dy, x, w = dy.to(D), x.to(D), weight.to(D)
    C = x.shape[-1]
    r, dr = rstd(x, eps)
    u, du = (dy, torch.zeros_like(dy)) if t is None else rotary(dy, t, layout, True)
    n = x * r
    dn = (x.abs() * dr + U * n.abs()) * SLOP
    g = u * w
    dg = (w.abs() * du + U * g.abs()) * SLOP
    dot = (g * n).sum(-1, keepdim=True)
    ddot = (g.abs() * dn + n.abs() * dg + HEAD_SUM * U * (g * n).abs()).sum(-1, keepdim=True)
    m = dot / C
    dm = ddot / C + U * m.abs()
    inner = g - n * m
    dx = r * inner
    slack = r * (dg + n.abs() * dm + m.abs() * dn + U * (n * m).abs() + U * inner.abs()) + \
        dx.abs() * (dr / r + U)
    term = (u * n).reshape(ranks, -1, C)
    off = (u.abs() * dn + n.abs() * du).reshape(ranks, -1, C).sum(1)
    dw = term.sum(1)
    ddw = off + additions(term.shape[1], C) * U * term.abs().sum(1)
    return (dx, slack * SLOP), (dw, ddw * SLOP)
