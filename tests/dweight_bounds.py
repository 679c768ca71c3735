"""How far the weight's gradient may be off: the additions that one term may
pass through, counted over the backward pass's launches.

A term dy n has one rounding (n = x r; the product is added by a fused
multiply-add), and each addition on its way rounds once more.  A thread adds
its own rows one after the other, the rows side by side in a workgroup are
added over lanes (halving) and then over waves (in a chain), and the
workgroups' partial rows in chains of every eighth, eight chains in the end.
"""
import torch

from tests import operator_bounds as ob

WAVES = 16        # of a workgroup
WORKGROUPS = 256  # partial rows of all ranks, at most
JOIN = 8          # chains of the join


def additions(ranks, rows, cols, bf16):
    """The longest way of a term; rows: all ranks'."""
    n = rows // ranks
    blocks = min(n, max(1, WORKGROUPS // ranks))
    vectors = -(-cols // (8 if bf16 else 4))
    join = -(-blocks // JOIN) + JOIN - 1
    if cols < (8 if bf16 else 4) or vectors > 4096:
        return -(-n // blocks) + join           # a row after the other
    if vectors > 1024:
        return n if n <= 2 else -(-n // blocks) + join
    lanes = -(-vectors // 64) * 64
    while lanes <= 64 and lanes > 1 and lanes // 2 >= vectors:
        lanes //= 2
    side = 64 * WAVES // lanes
    within = (64 // lanes - 1).bit_length() if lanes < 64 else 0
    if n <= 2 * side:
        return 2 + within + WAVES               # one workgroup, no join
    unit = max(1, 64 // lanes)
    side = min(side, -(-(-(-n // blocks)) // unit) * unit)
    blocks = min(blocks, -(-n // side))
    return -(-n // (blocks * side)) + within + WAVES + -(-blocks // JOIN) + JOIN - 1


def dweight(dy, x, rstd, ranks):
    """(value, slack) of the weight's gradient, [ranks, cols]."""
    d = torch.float64
    t = (dy.to(d) * (x.to(d) * rstd.to(d)[:, None])).view(ranks, -1, x.shape[1])
    steps = additions(ranks, x.shape[0], x.shape[1], x.dtype == torch.bfloat16) + 1
    return t.sum(1), steps * ob.U * t.abs().sum(1) * ob.SLOP
