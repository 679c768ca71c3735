"""The operators on attention heads on the GPU, against their 64-bit forms
(head_forms.py): every output lies between the roundings of the form's value
minus and plus the float32 computation's slack."""
import itertools

import pytest

from tests import head_forms as hf
from tests import operator_bounds as ob

pytestmark = pytest.mark.gpu

EPS = 1e-6


@pytest.fixture(scope="module")
def env():
    import torch
    from collective_communication_ring_amd import api
    assert torch.cuda.is_available(), "GPU tests need a GPU"
    api.lib()
    return dict(torch=torch, api=api, dev=torch.device("cuda:0"),
                types={"f32": torch.float32, "bf16": torch.bfloat16})


def _host(env, shape, seed, dtype, scale=1.0):
    torch = env["torch"]
    return (torch.randn(shape, generator=torch.Generator().manual_seed(seed)) * scale).to(dtype)


def _place(env, x, how):
    """x [batch, tokens, heads, dim] on the GPU in a memory order of `how`; its
    surroundings hold 55."""
    torch = env["torch"]
    B, S, H, D = x.shape
    if how == "tokens":
        y = torch.empty((B, S, H, D), dtype=x.dtype, device=env["dev"])
    elif how == "heads":  # [batch, heads, tokens, dim]
        y = torch.empty((B, H, S, D), dtype=x.dtype, device=env["dev"]).transpose(1, 2)
    elif how == "odd":  # distances that are no multiples of anything, an odd start
        flat = torch.full((3 + B * (S * (H * (D + 3) + 5) + 7),), 55.0, device=env["dev"]).to(x.dtype)
        y = flat[3:].as_strided((B, S, H, D), (S * (H * (D + 3) + 5) + 7, H * (D + 3) + 5, D + 3, 1),
                                flat.storage_offset() + 3)
    else:  # a part of wider rows
        y = torch.full((B, S, 3, H, D), 55.0, device=env["dev"]).to(x.dtype)[:, :, 1]
    y.copy_(x)
    return y


def _rotation(env, rot, layout, seed=0, **scaling):
    r = env["api"].Rotation(rot, 10000.0, layout, device=env["dev"], **scaling)
    return r, r.frequencies.cpu(), float(env["torch"].tensor(r.factor, dtype=env["torch"].float32))


def _positions(env, B, S, seed, far=70000, dtype=None):
    torch = env["torch"]
    g = torch.Generator().manual_seed(seed + 77)
    p = torch.randint(-5, far, (B, 1), generator=g) + torch.randint(0, 9, (B, S), generator=g).cumsum(1)
    return p.to(dtype or torch.int64)


def _run(env, kind, B=2, S=3, HQ=4, HK=2, D=64, rot=None, layout="halves", dtype="bf16", how="tokens",
         wtype=None, ranks=1, inverse=False, in_place=False, seed=0, scaling={}, values=None,
         shared=False, pdtype=None, eps=EPS, far=70000):
    """One call, all outputs checked."""
    torch, api, dev = env["torch"], env["api"], env["dev"]
    dt = env["types"][dtype]
    rot = D // 2 * 2 if rot is None else rot
    sides = [("q", HQ), ("k", HK)] if HK else [("q", HQ)]
    pos = _positions(env, 1 if shared else B, S, seed, far, pdtype)
    turn, t = {}, None
    if rot:
        rotation, freq, factor = _rotation(env, rot, layout, **scaling)
        t = hf.table(pos.expand(B, S), freq, factor)
        turn = dict(positions=(pos[0] if shared else pos).to(dev), rotation=rotation)
    args, out, want = {}, {}, {}
    for i, (n, H) in enumerate(sides):
        x = _host(env, (B, S, H, D), 10 * seed + i, dt, 1.5) if values is None else values[i].to(dt)
        w = (1 + 0.2 * _host(env, (D,), 10 * seed + 4 + i, torch.float32)).to(
            env["types"][wtype or dtype])
        args[n] = _place(env, x, how)
        if kind == "rotary":
            want[n + "_out"] = hf.rotary(x, t, layout, inverse)
        elif kind == "norm":
            args[n + "_weight"] = w.to(dev)
            want[n + "_out"] = hf.head_norm(x, w, eps, t, layout)
        else:
            dy = _host(env, (B, S, H, D), 10 * seed + 2 + i, dt, 0.1)
            args[n + "_weight"] = w.to(dev)
            args["d" + n + "_out"] = _place(env, dy, how)
            args[n + "_dweight"] = torch.full((ranks, D), 9.0, device=dev)
            want["d" + n], want[n + "_dweight"] = hf.head_norm_backward(dy, x, w, eps, t, layout, ranks)
        name = "d" + n if kind == "back" else n + "_out"
        args[name] = args["d" + n + "_out" if in_place == "dy" else n] if in_place else \
            _place(env, torch.full_like(x, -3.0), how)
        out[name] = args[name]
        if kind == "back":
            out[n + "_dweight"] = args[n + "_dweight"]
    f = dict(rotary=api.rotary, norm=api.head_rmsnorm, back=api.head_rmsnorm_backward)[kind]
    if kind == "rotary":
        args["inverse"] = inverse
    else:
        args["eps"] = eps
    f(**args, **turn)
    torch.cuda.synchronize()
    for n, (value, slack) in want.items():
        ob.between(out[n], value, slack, (kind, n, B, S, HQ, HK, D, rot, layout, dtype, how))
    if how in ("odd", "wide"):  # nothing beside the outputs is written
        for n in out:
            if out[n].dim() == 4:
                base = out[n]._base
                mask = torch.ones(base.numel(), dtype=torch.bool, device=dev)
                mask.as_strided(out[n].shape, out[n].stride(),
                                out[n].storage_offset() - base.storage_offset()).fill_(False)
                assert bool((base.reshape(-1)[mask] == 55).all()), n


KINDS = ("rotary", "norm", "back")
# heads of a vector and less, of odd lengths, with a half that cuts a vector, up to the longest
DIMS = (2, 3, 8, 17, 34, 40, 64, 80, 96, 100, 127, 128, 192, 250, 256, 511, 576, 1000, 1024)


@pytest.mark.parametrize("D", DIMS)
@pytest.mark.parametrize("kind", KINDS)
def test_dims(env, kind, D):
    for k, (dtype, layout) in enumerate(itertools.product(("f32", "bf16"), ("halves", "pairs"))):
        _run(env, kind, D=D, dtype=dtype, layout=layout, seed=k)


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("D,rot", [(64, 32), (64, 2), (80, 20), (96, 36), (128, 64), (100, 26), (33, 10),
                                   (256, 128), (576, 64), (1024, 6)])
def test_part_of_a_head(env, kind, D, rot):
    for k, (dtype, layout) in enumerate(itertools.product(("f32", "bf16"), ("halves", "pairs"))):
        _run(env, kind, D=D, rot=rot, dtype=dtype, layout=layout, seed=k)


@pytest.mark.parametrize("kind", ("norm", "back"))
@pytest.mark.parametrize("D", (64, 90, 128, 1024))
def test_norm_alone(env, kind, D):
    _run(env, kind, D=D, rot=0, dtype="bf16")
    _run(env, kind, D=D, rot=0, dtype="f32", S=5, HQ=7, HK=0)


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("how", ("heads", "odd", "wide"))
@pytest.mark.parametrize("D", (48, 63, 128))
def test_memory_orders(env, kind, how, D):
    _run(env, kind, D=D, how=how, dtype="bf16", layout="pairs", B=3, S=5)
    _run(env, kind, D=D, how=how, dtype="f32", B=1, S=4, HQ=3, HK=3)


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("B,S,HQ,HK", [(1, 1, 1, 0), (1, 1, 1, 1), (1, 1, 32, 8), (5, 1, 3, 1), (1, 257, 1, 0),
                                       (2, 130, 1, 1), (1, 33, 40, 1), (4, 1, 64, 64), (1, 1000, 5, 2)])
def test_counts(env, kind, B, S, HQ, HK):
    _run(env, kind, B=B, S=S, HQ=HQ, HK=HK, D=128, dtype="bf16", ranks=1)
    _run(env, kind, B=B, S=S, HQ=HQ, HK=HK, D=24, dtype="f32", ranks=B)


@pytest.mark.parametrize("kind", KINDS)
def test_many_heads(env, kind):
    """Several turns of a workgroup, stores past the caches, many partial rows."""
    _run(env, kind, B=2, S=2100, HQ=17, HK=3, D=128, dtype="bf16", ranks=2)
    _run(env, kind, B=1, S=4099, HQ=6, HK=6, D=80, rot=40, dtype="f32", layout="pairs")
    _run(env, kind, B=8, S=1500, HQ=3, HK=1, D=64, dtype="bf16", how="heads", ranks=8)


@pytest.mark.parametrize("ranks", (1, 3, 6))
def test_ranks(env, ranks):
    _run(env, "back", B=6, S=70, HQ=3, HK=2, D=128, ranks=ranks)


@pytest.mark.parametrize("scaling", ("linear", "base", "bands", "ramp"))
@pytest.mark.parametrize("inverse", (False, True))
def test_scaled_and_inverse(env, scaling, inverse):
    how = dict(scaling=scaling, scale=4.0, original=4096)
    _run(env, "rotary", D=128, dtype="f32", scaling=how, inverse=inverse)
    _run(env, "rotary", D=96, rot=64, dtype="bf16", layout="pairs", scaling=how, inverse=inverse)


@pytest.mark.parametrize("kind", KINDS)
def test_weights_and_positions(env, kind):
    torch = env["torch"]
    _run(env, kind, D=64, dtype="bf16", wtype="f32", pdtype=torch.int32)
    _run(env, kind, D=64, dtype="bf16", shared=True)
    _run(env, kind, D=64, dtype="f32", shared=True, pdtype=torch.int32)
    _run(env, kind, D=64, dtype="f32", far=2_000_000_000)


@pytest.mark.parametrize("D", (64, 70, 128))
def test_in_place(env, D):
    for dtype, how in (("bf16", "tokens"), ("f32", "odd")):
        _run(env, "rotary", D=D, S=50, dtype=dtype, how=how, in_place=True)
        _run(env, "norm", D=D, S=50, dtype=dtype, how=how, in_place=True)
        _run(env, "back", D=D, S=50, dtype=dtype, how=how, in_place=True)
        _run(env, "back", D=D, S=50, dtype=dtype, how=how, in_place="dy")


def test_inverse_undoes(env):
    """A rotation and its transpose: each rounds once."""
    torch, api, dev = env["torch"], env["api"], env["dev"]
    x = _host(env, (5, 4, 64), 1, torch.float32).to(dev)
    r = api.Rotation(64, device=dev)
    p = torch.tensor([0, 1, 1000, 10 ** 6, 3], device=dev)
    y, z = torch.empty_like(x), torch.empty_like(x)
    api.rotary(x, p, r, y)
    api.rotary(y, p, r, z, inverse=True)
    # twice: c and s off by 2.2 U each against a pair's length, two roundings
    length = torch.sqrt(x[..., :32] ** 2 + x[..., 32:] ** 2).repeat(1, 1, 2)
    assert bool(((z - x).abs() <= 2 * (2 * 2.2 + 2) * hf.U * 1.5 * length).all())
    assert torch.equal(y[0], x[0])


def test_extreme_values(env):
    """Heads whose squares leave float32's range; zeros; infinities beside what
    is not rotated."""
    torch, api, dev = env["torch"], env["api"], env["dev"]
    x = _host(env, (1, 6, 2, 64), 3, torch.float32)
    for t, by in enumerate((1.0, 2.0 ** 66, 2.0 ** 100, 2.0 ** -80, 0.0, 2.0 ** -70)):
        x[0, t] *= by
    for dtype in ("f32", "bf16"):
        _run(env, "norm", B=1, S=6, HQ=2, HK=0, D=64, dtype=dtype, values=[x])
    x = torch.randn(1, 1, 7, device=dev)
    for bad in (float("inf"), float("nan")):
        x[..., 3] = bad
        y = torch.empty_like(x)
        api.rotary(x, torch.tensor([5], device=dev), api.Rotation(2, layout="pairs", device=dev), y)
        got, was = y[0, 0].cpu(), x[0, 0].cpu()
        assert torch.equal(got[[2, 4, 5, 6]], was[[2, 4, 5, 6]]) and bool(torch.isfinite(got[:2]).all())
        assert torch.equal(torch.isnan(got), torch.isnan(was))


def test_no_eps(env):
    """No eps: tiny heads are taken again in 64 bits, a head of zeros is 0 / 0."""
    torch, api, dev = env["torch"], env["api"], env["dev"]
    x = _host(env, (1, 3, 2, 64), 5, torch.float32) * 2.0 ** -78
    _run(env, "norm", B=1, S=3, HQ=2, HK=0, D=64, dtype="f32", values=[x], eps=0.0)
    z = torch.zeros(2, 1, 64, device=dev)
    api.head_rmsnorm(z, torch.ones(64, device=dev), z, 0.0)
    assert bool(torch.isnan(z).all())


def test_nothing(env):
    torch, api, dev = env["torch"], env["api"], env["dev"]
    r = api.Rotation(8, device=dev)
    e = torch.empty(0, 3, 8, device=dev)
    p = torch.empty(0, dtype=torch.int64, device=dev)
    api.rotary(e, p, r, e.clone())
    w, dw = torch.ones(8, device=dev), torch.full((1, 8), 3.0, device=dev)
    api.head_rmsnorm(e, w, e.clone(), positions=p, rotation=r)
    api.head_rmsnorm_backward(e.clone(), e, w, e.clone(), dw, positions=p, rotation=r)
    torch.cuda.synchronize()
    assert bool((dw == 0).all())


def test_past_32_bits(env):
    """Heads whose addresses are more than 2^32 elements into their arrays."""
    torch, api, dev = env["torch"], env["api"], env["dev"]
    S, D = 3, 64
    far = (1 << 31) + 64
    flat = torch.empty(2 * far + S * D, dtype=torch.bfloat16, device=dev)
    x = flat.as_strided((3, S, 1, D), (far, D, D, 1))
    host = _host(env, (3, S, 1, D), 1, torch.bfloat16)
    x.copy_(host)
    pos = _positions(env, 3, S, 0)
    r, freq, factor = _rotation(env, D, "halves")
    api.rotary(x, pos.to(dev), r, x)
    torch.cuda.synchronize()
    value, slack = hf.rotary(host, hf.table(pos, freq, factor), "halves")
    ob.between(x, value, slack, "far")


def test_repeats_and_streams(env):
    """The same bits every time, on two streams with a workspace each, and from
    a graph replayed between eager calls on the same data."""
    torch, api, dev = env["torch"], env["api"], env["dev"]
    B, S, H, D = 2, 300, 6, 128
    q, dy = (_host(env, (B, S, H, D), k, torch.bfloat16).to(dev) for k in (1, 2))
    w = torch.ones(D, device=dev, dtype=torch.bfloat16)
    r = api.Rotation(D, device=dev)
    pos = torch.arange(S, device=dev)

    def make():
        return torch.empty_like(q), torch.empty_like(q), torch.empty(2, D, device=dev), \
            api.head_rmsnorm_backward_workspace(2, D)

    def call(y, dq, dw, ws):
        api.head_rmsnorm(q, w, y, positions=pos, rotation=r)
        api.head_rmsnorm_backward(dy, q, w, dq, dw, positions=pos, rotation=r, workspace=ws)
    first = make()
    call(*first)
    torch.cuda.synchronize()
    want = [t.clone() for t in first[:3]]
    streams = [torch.cuda.Stream() for _ in range(2)]
    sets = [make() for _ in streams]
    for s, m in zip(streams, sets):
        with torch.cuda.stream(s):
            for _ in range(5):
                call(*m)
    torch.cuda.synchronize()
    for m in sets:
        assert all(torch.equal(a, b) for a, b in zip(m, want))
    m = make()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        call(*m)
    for k in range(4):
        q.mul_(1.25 if k == 2 else 1.0)
        for t in m[:3]:
            t.zero_()
        g.replay()
        call(*first)
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(m[:3], first[:3])), k


def test_wrappers_refuse(env):
    torch, api, dev = env["torch"], env["api"], env["dev"]
    q = torch.zeros(2, 3, 4, 8, device=dev)
    k = torch.zeros(2, 3, 2, 8, device=dev)
    w, dw = torch.ones(8, device=dev), torch.zeros(2, 8, device=dev)
    p, r = torch.zeros(2, 3, dtype=torch.int64, device=dev), api.Rotation(8, device=dev)
    host = api.Rotation(8, device="cpu")
    ws = api.head_rmsnorm_backward_workspace(2, 8)
    o = lambda t=q: torch.empty_like(t)  # noqa: E731
    for call in (
            lambda: api.rotary(q, p, r, o(k)), lambda: api.rotary(q, p, r, o().bfloat16()),
            lambda: api.rotary(q, p, r, o().cpu()), lambda: api.rotary(q, p[:, :2], r, o()),
            lambda: api.rotary(q, p.float(), r, o()), lambda: api.rotary(q, p.cpu(), r, o()),
            lambda: api.rotary(q, p, host, o()), lambda: api.rotary(q, p, r, o(), k=k),
            lambda: api.rotary(q, None, r, o()),
            lambda: api.rotary(q, p, r, o(), k=k, k_out=o()),
            lambda: api.rotary(q[0, 0], p, r, o()), lambda: api.rotary(q.double(), p, r, o()),
            lambda: api.rotary(q.transpose(2, 3), p, r, o().transpose(2, 3)),
            lambda: api.rotary(q, p.t().contiguous().t(), r, o()),
            lambda: api.head_rmsnorm(q, w[:7], o()), lambda: api.head_rmsnorm(q, w.bfloat16(), o()),
            lambda: api.head_rmsnorm(q, w, o(), positions=p),
            lambda: api.head_rmsnorm(q, w, o(), k=k, k_out=o(k)),
            lambda: api.head_rmsnorm(q.bfloat16(), w, o().bfloat16(), k=k.bfloat16(),
                                     k_weight=w.bfloat16(), k_out=o(k).bfloat16()),
            lambda: api.head_rmsnorm_backward(q, q, w, o(), dw[:, :4], workspace=ws),
            lambda: api.head_rmsnorm_backward(q, q, w, o(), torch.zeros(3, 8, device=dev), workspace=ws),
            lambda: api.head_rmsnorm_backward(q, q, w, o(), dw, k=k, dk=o(k), workspace=ws),
            lambda: api.head_rmsnorm_backward(q, q, w, o(), dw, workspace=ws.cpu())):
        with pytest.raises(ValueError):
            call()
    for call in (lambda: api.rotary(q, p, r, q[:1].expand(2, 3, 4, 8)),
                 lambda: api.head_rmsnorm_backward(o(), q, w, o(), dw, workspace=ws[:256]),
                 lambda: api.head_rmsnorm(q, w, o(), eps=-1.0)):
        with pytest.raises(api.ArError):
            call()
