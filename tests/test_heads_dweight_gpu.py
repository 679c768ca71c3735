"""The head norm's backward pass where its sums are longest and its values extreme.

A weight's gradient goes through so many additions, by the launch's own rules: a
thread's rounds of heads, the heads of a wave, four waves, the workgroups dealt to 32,
and those 32."""
import math

import pytest

from tests import head_forms as hf
from tests import operator_bounds as ob
from tests.test_heads_gpu import _host, _run, env  # noqa: F401

pytestmark = pytest.mark.gpu


def additions(ranks, batches, tokens, heads, side, dim):
    """At most, of a rank's `batches` of `tokens` with heads = (q, k) of each."""
    lanes = 1
    while lanes * 16 < dim:
        lanes *= 2
    group, waves, most = 64 // lanes, 4, 768 // ranks
    chunk = group
    while chunk > 1 and all(chunk // 2 * h % group == 0 for h in heads):
        chunk //= 2
    while chunk > 1 and batches * tokens < chunk * most * waves:
        chunk //= 2
    chunks = -(-tokens // chunk) * batches
    apart = all(heads) and 2 * chunks <= most * waves
    units = 2 * chunks if apart else chunks
    run = -(-units // (most * waves))
    blocks = -(-units // (run * waves))
    rounds = run * -(-chunk * heads[side] // group)
    return rounds + int(math.log2(group)) + 2 + -(-blocks // 32) + 5


@pytest.mark.parametrize("ranks,batches,tokens,heads,dim,dtype", [
    (64, 1, 12500, (8, 0), 128, "bf16"), (64, 3, 700, (5, 3), 64, "f32"), (1, 1, 30000, (16, 4), 128, "bf16"),
    (1, 2, 9001, (3, 3), 96, "f32"), (8, 1, 2048, (8, 2), 128, "bf16"), (1, 1, 1, (64, 8), 128, "f32"),
    (2, 1, 40000, (1, 1), 20, "f32")])
def test_sums(env, ranks, batches, tokens, heads, dim, dtype):  # noqa: F811
    torch, api, dev = env["torch"], env["api"], env["dev"]
    dt, D = env["types"][dtype], torch.float64
    g = torch.Generator(device=dev).manual_seed(dim)
    args, B = {}, ranks * batches
    for n, h in zip("qk", heads):
        if h:
            args[n], args["d%s_out" % n] = (torch.randn((B, tokens, h, dim), generator=g, device=dev).to(dt)
                                            for _ in range(2))
            args["d" + n] = torch.empty_like(args[n])
            args[n + "_weight"] = 1 + 0.2 * _host(env, (dim,), 3, torch.float32).to(dev)
            args[n + "_dweight"] = torch.full((ranks, dim), 9.0, device=dev)
    api.head_rmsnorm_backward(eps=1e-6, **args)
    torch.cuda.synchronize()
    for side, (n, h) in enumerate(zip("qk", heads)):
        K = additions(ranks, batches, tokens, heads, side, dim)
        for r in (range(ranks) if h else ()):
            x, dy = (args[v][r * batches:(r + 1) * batches].reshape(-1, dim).to(D) for v in (n, "d%s_out" % n))
            root, droot = hf.rstd(x, 1e-6)
            term = dy * x * root
            slack = K * hf.U * term.abs().sum(0) + (dy.abs() * (x.abs() * droot + hf.U * (x * root).abs())).sum(0)
            ob.between(args[n + "_dweight"][r], term.sum(0), hf.SLOP * slack, (n, r, K))


def test_extreme_values(env):  # noqa: F811
    """Heads whose squares leave float32's range, and zeros: r in 64 bits."""
    torch = env["torch"]
    x = _host(env, (1, 6, 2, 64), 3, torch.float32)
    for t, by in enumerate((1.0, 2.0 ** 66, 2.0 ** 100, 2.0 ** -80, 0.0, 2.0 ** -70)):
        x[0, t] *= by
    for dtype in ("f32", "bf16"):
        for rot in (0, 64):
            _run(env, "back", B=1, S=6, HQ=2, HK=0, D=64, rot=rot, dtype=dtype, values=[x])
    wide = torch.cat([x] * 9, 3)
    _run(env, "back", B=1, S=6, HQ=2, HK=0, D=576, rot=0, dtype="f32", values=[wide])


def test_no_eps(env):  # noqa: F811
    """No eps: tiny heads' r is taken again in 64 bits."""
    x = _host(env, (1, 3, 2, 64), 5, env["torch"].float32) * 2.0 ** -78
    _run(env, "back", B=1, S=3, HQ=2, HK=0, D=64, dtype="f32", values=[x], eps=0.0)
    _run(env, "back", B=1, S=3, HQ=2, HK=2, D=64, dtype="bf16", values=[x, x * 2.0 ** 40], eps=0.0)
