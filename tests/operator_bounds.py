"""Plain 64-bit forms of the operators around the collectives, with bounds.

Each form returns (value, slack) pairs in float64: a correct float32
computation of that value lies within value +- slack before its last rounding,
whatever the order of its sums.  The slacks count roundings (U = 2^-24 each,
half a float32 step):

  a sum of n terms in any order, in chains of at most K additions: K U sum|terms|
  a product, quotient, root or addition: U of its result

`between` then rounds both ends to the output's type; as rounding keeps order,
the kernel's output lies between them, ends included.
"""
import torch

U = 2.0 ** -24
TINY = 2.0 ** -126
SLOP = 1.001  # the second-order terms of the bounds


def chain(n):
    """Additions one value may pass through: a wave's 64 lanes share n terms,
    then the lanes, and up to 16 waves, are joined."""
    return n / 64 + 8 + 6 + 16


def norm(x, weight, eps, residual=None, parts=None, divisor=1.0, group=None):
    """x [T, C] (or parts [R, T, C], in any order) -> dict of (value, slack)."""
    d = torch.float64
    w = weight.to(d)
    if parts is None:
        h = x.to(d)
        dh = torch.zeros_like(h)
    else:
        terms = parts.to(d)
        h = terms.sum(0) / divisor
        dh = parts.shape[0] * U * terms.abs().sum(0) / divisor
    if residual is not None:
        h = h + residual.to(d)
        dh = dh + U * h.abs()
    C = h.shape[1]
    ss = (h * h).sum(1)
    dss = 2 * (h.abs() * dh).sum(1) + chain(C) * U * ss
    r = 1 / torch.sqrt(ss / C + eps)
    # d(r)/r = d(mean)/(2 (mean + eps)); then the division, eps, root, reciprocal
    dr = r * (0.5 * dss / (ss + C * eps) + 3.5 * U) * SLOP
    v = h * r[:, None] * w
    dv = (v.abs() * (dr / r)[:, None] + 2 * U * v.abs() + dh * r[:, None] * w.abs()) * SLOP
    out = {"sum": (h, dh * SLOP), "rstd": (r, dr)}
    if group is None:
        out["y"] = (v, dv)
        return out
    group = group or C
    G = -(-C // group)
    pad = torch.nn.functional.pad
    va = pad(v.abs(), (0, G * group - C)).view(-1, G, group)
    da = pad(dv, (0, G * group - C)).view(-1, G, group)
    scale = torch.clamp(va.amax(2) / 448, min=TINY)
    dscale = (da.amax(2) / 448 + U * scale) * SLOP
    spread = lambda t: t[:, :, None].expand(-1, G, group).reshape(-1, G * group)[:, :C]  # noqa: E731
    s, ds = spread(scale), spread(dscale)
    q = v / s
    out["scale"] = (scale, dscale)
    out["y"] = (q, (dv / s + q.abs() * (ds / s + 3 * U)) * SLOP)
    return out


def norm_backward(dy, x, weight, rstd, dsum=None, ranks=1):
    d = torch.float64
    dy, x, w, r = dy.to(d), x.to(d), weight.to(d), rstd.to(d)[:, None]
    T, C = x.shape
    n, g = x * r, dy * w
    dot = (g * n).sum(1, keepdim=True)
    ddot = (chain(C) + 3) * U * (g * n).abs().sum(1, keepdim=True)
    m = dot / C
    dm = ddot / C + U * m.abs()
    dx = r * (g - n * m)
    slack = r * (2 * U * g.abs() + n.abs() * dm + 4 * U * (n * m).abs()) + 2 * U * dx.abs()
    if dsum is not None:
        dx = dx + dsum.to(d)
        slack = slack + U * dx.abs()
    t = (dy * n).view(ranks, -1, C) if T else dy.new_zeros((ranks, 0, C))
    dw = t.sum(1)
    # any order of a shard's rows: at most as many additions as rows, and two roundings a term
    ddw = (t.shape[1] + 4) * U * t.abs().sum(1)
    return {"dx": (dx, slack * SLOP), "dweight": (dw, ddw * SLOP)}


def between(got, value, slack, what):
    """Every element of `got` lies between the roundings of value -+ slack to
    its type (float32 first, as the kernels' values are; infinities and NaN
    must be equal)."""
    got, value, slack = got.detach().cpu(), value.cpu(), slack.cpu()
    assert got.shape == value.shape, (what, got.shape, value.shape)
    fine = torch.isfinite(value)
    g = got.to(torch.float64)
    assert torch.equal(torch.nan_to_num(g[~fine], nan=7.0), torch.nan_to_num(value[~fine], nan=7.0)), what
    lo = (value - slack)[fine].to(torch.float32).to(got.dtype).to(torch.float64)
    hi = (value + slack)[fine].to(torch.float32).to(got.dtype).to(torch.float64)
    g = g[fine]
    bad = ~((g >= lo) & (g <= hi))
    if bad.any():
        i = int(torch.nonzero(bad)[0])
        raise AssertionError("%s: %d of %d outside, first %r not in [%r, %r] (value %r)" % (
            what, int(bad.sum()), bad.numel(), float(g[i]), float(lo[i]), float(hi[i]),
            float(value[fine][i])))
