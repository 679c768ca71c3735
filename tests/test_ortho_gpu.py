"""The orthogonalisation on the GPU, against its 64-bit form (ortho_forms.py):
element by element, each step from the one before."""
import pytest

from tests import operator_bounds as ob
from tests import ortho_forms as of

pytestmark = pytest.mark.gpu

COEFFICIENTS = (3.4445, -4.7750, 2.0315)
EPS = 1e-7


@pytest.fixture(scope="module")
def env():
    import torch
    from collective_communication_ring_amd import api
    assert torch.cuda.is_available(), "GPU tests need a GPU"
    api.lib()
    return dict(torch=torch, api=api, dev=torch.device("cuda:0"),
                types={"f32": torch.float32, "bf16": torch.bfloat16})


def _host(env, shape, seed, dtype="f32", scale=1.0):
    torch = env["torch"]
    g = torch.Generator().manual_seed(seed)
    return (torch.randn(shape, generator=g) * scale).to(env["types"][dtype])


def _rows_apart(env, x, pad, offset=0):
    torch = env["torch"]
    m, n = x.shape
    flat = torch.full((offset + m * (n + pad),), 55.0, device=env["dev"]).to(x.dtype)
    view = flat[offset:].view(m, n + pad)[:, :n]
    view.copy_(x)
    return view, flat


def _one_step(env, m, n, dtype="f32", coefficients=COEFFICIENTS, scale=1.0, pad=0, offset=0, x=None,
              eps=EPS, seed=0):
    torch, api = env["torch"], env["api"]
    x = _host(env, (m, n), seed, dtype, 0.02) if x is None else x
    gx, _ = _rows_apart(env, x, pad, offset)
    y, flat = _rows_apart(env, torch.zeros_like(x), 2 * pad, offset)
    api.orthogonalize(gx, y, 1, coefficients, eps, scale)
    torch.cuda.synchronize()
    value, slack = of.one_step(x, coefficients, eps, scale)
    ob.between(y, value, slack, (m, n, dtype))
    if pad:
        wide = flat[offset:].view(m, n + 2 * pad)
        assert bool((wide[:, n:] == 55).all()) and bool((flat[:offset] == 55).all())


def _steps(env, m, n, steps=5, coefficients=COEFFICIENTS, x=None, seed=0):
    """Steps one by one: each one's float32 result against a step from the one
    before, and bfloat16 is the same with one more rounding.  Steps by groups: the
    2-norm of all errors of each group after the one before, and of bfloat16's first."""
    torch, api, dev = env["torch"], env["api"], env["dev"]
    x = _host(env, (m, n), seed, "bf16", 0.02).float() if x is None else x
    ks = of.coefficient_list(coefficients, steps)

    def call(x, k):
        y = torch.empty_like(x, device=dev)
        api.orthogonalize(x.to(dev), y, k, ks[:k], EPS)
        torch.cuda.synchronize()
        return y.cpu()
    if not of.by_groups(m, n):
        before = None
        for k in range(steps):
            y = call(x, k + 1)
            value, slack = of.next_step(before, k, ks) if k else of.one_step(x, ks[0], EPS)
            ob.between(y, value, slack, (m, n, k))
            before = y
        if torch.equal(x.bfloat16().float(), x):
            assert torch.equal(call(x.bfloat16(), steps), y.bfloat16()), (m, n)
        return
    before, i = of.start(x, EPS), 0
    for group in of.groups_of(m, n, ks, 16.0):
        y = call(x, i + group)
        value = of.steps_of(before, ks[i:i + group])
        error, bound = float((y.double() - value).norm()), of.group_error(before, ks[i:i + group])
        print(m, n, "steps", i, "to", i + group, "error", error, "bound", bound, "of", float(value.norm()))
        assert error <= bound
        before, i = y.double(), i + group
    z = x.bfloat16()
    first = of.groups_of(m, n, ks, 256.0)[0]
    before = of.start(z, EPS)
    value = of.steps_of(before, ks[:first])
    error = float((call(z, first).double() - value).norm())
    bound = of.group_error(before, ks[:first])
    assert error <= bound + 2.0 ** -8 * (float(value.norm()) + bound)


SIDES = [(1, 1), (1, 7), (2, 2), (5, 3), (31, 33), (32, 32), (33, 64), (64, 128), (65, 40), (100, 260),
         (127, 129), (128, 128), (129, 300), (257, 255), (300, 40), (8, 700), (700, 3),
         (32, 512), (480, 20), (64, 256), (65, 128), (96, 128), (97, 128), (127, 90)]  # about LDS's room


@pytest.mark.parametrize("m,n", SIDES)
@pytest.mark.parametrize("dtype", ("f32", "bf16"))
def test_one_step(env, m, n, dtype):
    _one_step(env, m, n, dtype)


@pytest.mark.parametrize("m,n", [(40, 50), (70, 33), (130, 140)])
@pytest.mark.parametrize("dtype", ("f32", "bf16"))
def test_strides_scale_and_coefficients(env, m, n, dtype):
    _one_step(env, m, n, dtype, pad=3, offset=1)
    _one_step(env, m, n, dtype, scale=-0.2)
    _one_step(env, m, n, dtype, coefficients=(1.5, -0.5, 0.0))
    _one_step(env, m, n, dtype, coefficients=(0.0, 0.0, 1.0))
    _one_step(env, m, n, dtype, coefficients=(1.0, 0.0, 0.0))


@pytest.mark.parametrize("m,n", [(5, 9), (64, 64), (100, 70), (130, 200), (257, 300)])
def test_steps(env, m, n):
    _steps(env, m, n)


def test_steps_of_their_own(env):
    ks = [(4.0, -6.0, 3.0), (3.0, -3.5, 1.5), (1.875, -1.25, 0.375), (1.5, -0.5, 0.0)]
    _steps(env, 50, 90, 4, ks)
    _steps(env, 90, 50, 4, ks)


@pytest.mark.parametrize("m,n", [(520, 1000), (1100, 513)])
def test_larger(env, m, n):
    _one_step(env, m, n, "f32")
    _one_step(env, m, n, "bf16")
    _steps(env, m, n)


@pytest.mark.parametrize("m,n", [(900, 1200), (1500, 1000)])
def test_steps_by_groups(env, m, n):
    """Also three at once, whose sums are split otherwise."""
    torch, api, dev = env["torch"], env["api"], env["dev"]
    _steps(env, m, n)
    x = _host(env, (3, m, n), 8)
    y = torch.empty_like(x, device=dev)
    api.orthogonalize(x.to(dev), y, 2, COEFFICIENTS, EPS)
    torch.cuda.synchronize()
    for i in range(3):
        before = of.start(x[i], EPS)
        value = of.steps_of(before, [COEFFICIENTS] * 2)
        assert float((y[i].cpu().double() - value).norm()) <= of.group_error(before, [COEFFICIENTS] * 2)


@pytest.mark.parametrize("m,n", [(900, 1170), (1170, 900), (64, 16390), (10500, 100), (201, 5301), (1001, 2500)])
@pytest.mark.parametrize("steps", (2, 3, 5, 7))
def test_groups_of_steps(env, m, n, steps):
    """Steps by groups, on a matrix with one element in each row and column (of the
    shorter side): each element goes by the polynomials alone, and an element of a
    product has one term, so that nothing but halves' and float32's roundings is
    lost: three steps widen an error 2^-20 of A by up to 141, and what is off by
    more than 2^-12 is in the wrong place, or is not that polynomial."""
    torch, api, dev = env["torch"], env["api"], env["dev"]
    g = torch.Generator().manual_seed(m + n + steps)
    k = min(m, n)
    x = torch.zeros(m, n)
    at = torch.randperm(m, generator=g)[:k], torch.randperm(n, generator=g)[:k]
    x[at] = torch.exp(torch.rand(k, generator=g) * 4 - 2) * torch.sign(torch.rand(k, generator=g) - 0.5)
    x = x.bfloat16().float()
    y, b = torch.empty(m, n, device=dev), torch.empty(m, n, device=dev, dtype=torch.bfloat16)
    api.orthogonalize(x.to(dev), y, steps, COEFFICIENTS, EPS)
    api.orthogonalize(x.to(dev).bfloat16(), b, steps, COEFFICIENTS, EPS)
    s = x.double() / (x.double().norm() + EPS)
    for _ in range(steps):
        s = 3.4445 * s - 4.7750 * s ** 3 + 2.0315 * s ** 5
    torch.cuda.synchronize()
    assert bool(((y.cpu().double() - s).abs() <= 2.0 ** -12).all())
    assert bool(((b.cpu().double() - s).abs() <= 2.0 ** -12 + 2.0 ** -8 * s.abs()).all())
    assert bool((y.cpu()[x == 0] == 0).all()) and bool((b.cpu()[x == 0] == 0).all())


@pytest.mark.parametrize("count,m,n,steps", [(1, 100, 2500, 2), (1, 2300, 70, 2), (1, 2900, 2900, 1),
                                             (1, 4096, 4100, 1), (1, 4400, 4096, 1), (9, 1030, 1000, 2),
                                             (1, 2048, 2048, 2), (1, 4096, 4096, 1)])
def test_every_tile(env, count, m, n, steps):
    """Sizes at which each tile is taken for each product (64 to 256 wide, whole
    and by parts), against the form computed on the GPU; with two steps, the
    second from the first's result."""
    torch, api, dev = env["torch"], env["api"], env["dev"]
    g = torch.Generator(device=dev).manual_seed(m)
    x = torch.randn(count, m, n, generator=g, device=dev) * 0.02
    y, z = torch.empty_like(x), torch.empty_like(x)
    api.orthogonalize(x, y, 1, COEFFICIENTS, EPS)
    if steps > 1:
        api.orthogonalize(x, z, 2, COEFFICIENTS, EPS)
    torch.cuda.synchronize()
    for i in {0, count - 1}:
        value, slack = of.one_step(x[i], COEFFICIENTS, EPS)
        ob.between(y[i], value, slack, (m, n))
        if steps > 1:
            value, slack = of.next_step(y[i], 1, COEFFICIENTS)
            ob.between(z[i], value, slack, (m, n, "second"))


def test_values(env):
    """Few directions, wide ranges of values, the smallest and largest floats."""
    torch = env["torch"]
    low = _host(env, (60, 4), 1) @ _host(env, (4, 80), 2)
    _one_step(env, 60, 80, x=low)
    _steps(env, 60, 80, x=low)
    _steps(env, 60, 80, x=low.bfloat16().float())
    wide = _host(env, (50, 70), 3) * torch.exp(torch.arange(50.0) * 0.5)[:, None]
    _one_step(env, 50, 70, x=wide)
    for by in (2.0 ** 120, 2.0 ** -100):
        _one_step(env, 40, 30, x=_host(env, (40, 30), 4) * by, eps=0.0)


def test_special_values(env):
    torch, api, dev = env["torch"], env["api"], env["dev"]
    for dt in env["types"].values():
        x = torch.zeros(40, 50, dtype=dt, device=dev)
        y = torch.full_like(x, 3.0)
        api.orthogonalize(x, y)
        assert bool((y == 0).all())
        for bad in (float("inf"), float("nan")):
            x = torch.randn(40, 50, device=dev).to(dt)
            x[3, 4] = bad
            api.orthogonalize(x, y)
            assert bool(torch.isnan(y).all())


@pytest.mark.parametrize("m,n", [(130, 300), (1200, 900)])
def test_special_values_of_larger(env, m, n):
    torch, api, dev = env["torch"], env["api"], env["dev"]
    for dt in env["types"].values():
        x = torch.zeros(m, n, dtype=dt, device=dev)
        y = torch.full_like(x, 3.0)
        api.orthogonalize(x, y)
        assert bool((y == 0).all())
        for bad in (float("inf"), float("nan")):
            x = torch.randn(m, n, device=dev).to(dt)
            x[77, 101] = bad
            api.orthogonalize(x, y)
            assert bool(torch.isnan(y).all())


def _same(env, got, want):
    assert all(env["torch"].equal(a, b) for a, b in zip(got, want))


@pytest.mark.parametrize("m,n", [(33, 70), (200, 140)])
def test_many_matrices(env, m, n):
    """Matrices do not touch each other: each as by itself, in any form of the
    arguments, in place, and with a workspace of a few."""
    torch, api, dev = env["torch"], env["api"], env["dev"]
    count = 150
    x = _host(env, (count, m, n), 5).to(dev)
    x[7] *= 100
    want = torch.empty_like(x)
    for i in range(count):
        api.orthogonalize(x[i], want[i], 2)
    y = torch.empty_like(x)
    api.orthogonalize(x, y, 2)
    _same(env, y, want)
    apart = [torch.empty(m, n, device=dev) for _ in range(count)]
    api.orthogonalize(list(x), apart, 2, workspace=api.orthogonalize_workspace(7, m, n))
    _same(env, apart, want)
    api.orthogonalize(x, x, 2)
    _same(env, x, want)


def test_repeats_and_graph(env):
    """The same bits every time, on two streams, and from a graph replayed
    between eager calls on changing data."""
    torch, api, dev = env["torch"], env["api"], env["dev"]
    x = _host(env, (3, 150, 220), 6, "bf16").to(dev)
    y, ws = torch.empty_like(x), api.orthogonalize_workspace(3, 150, 220)
    api.orthogonalize(x, y, workspace=ws)
    torch.cuda.synchronize()
    want = y.clone()
    streams = [torch.cuda.Stream() for _ in range(2)]
    outs = [torch.empty_like(x) for _ in streams]
    for s, o in zip(streams, outs):
        for _ in range(3):
            api.orthogonalize(x, o, stream=s)
    torch.cuda.synchronize()
    for o in outs:
        assert torch.equal(o, want)
    g = torch.cuda.CUDAGraph()
    z, ws2 = torch.empty_like(x), api.orthogonalize_workspace(3, 150, 220)
    with torch.cuda.graph(g):
        api.orthogonalize(x, z, workspace=ws2)
    for k in range(4):
        if k == 2:
            x.add_(0.5)
        z.zero_()
        g.replay()
        api.orthogonalize(x, y, workspace=ws)
        torch.cuda.synchronize()
        assert torch.equal(y, z), k


@pytest.mark.parametrize("shape", [(3, 40, 50), (2, 1150, 920)])
def test_forms_of_the_arguments(env, shape):
    """Matrices that lie in turn in rows of one array, one of them by itself, a
    list for a tensor, on another stream, in place, and from a graph replayed
    between eager calls: the same bits."""
    torch, api, dev = env["torch"], env["api"], env["dev"]
    count, m, n = shape
    x = _host(env, shape, 9).to(dev)
    want = torch.empty_like(x)
    api.orthogonalize(x, want)
    room = torch.full((m, count, n + 5), 7.0, device=dev)
    turn = room.permute(1, 0, 2)[:, :, :n]
    turn.copy_(x)
    y = torch.empty_like(x)
    api.orthogonalize(turn, list(y))
    assert torch.equal(y, want)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    api.orthogonalize(list(turn), turn, stream=side)
    torch.cuda.synchronize()
    assert torch.equal(turn, want) and bool((room[:, :, n:] == 7.0).all())
    ws, z = api.orthogonalize_workspace(*shape), torch.empty_like(x)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        api.orthogonalize(x, z, workspace=ws)
    for k in range(4):
        if k == 2:
            x.add_(0.01)
        z.zero_()
        g.replay()
        api.orthogonalize(x, y)
        torch.cuda.synchronize()
        assert torch.equal(y, z), k
    assert api.orthogonalize([], []) == []
    assert api.orthogonalize(x[:0], y[:0]).shape[0] == 0


def test_wrapper_refuses(env):
    torch, api, dev = env["torch"], env["api"], env["dev"]
    x, y = (torch.zeros(2, 30, 40, device=dev) for _ in range(2))
    ws = api.orthogonalize_workspace(2, 30, 40)
    for call in (lambda: api.orthogonalize(x, y[:1], workspace=ws),
                 lambda: api.orthogonalize(x, []), lambda: api.orthogonalize([], y),
                 lambda: api.orthogonalize(x[None], y[None]), lambda: api.orthogonalize(x[0, 0], y[0, 0]),
                 lambda: api.orthogonalize([x], [y], workspace=ws),
                 lambda: api.orthogonalize(x, list(y)[:1], workspace=ws),
                 lambda: api.orthogonalize(x, y[:, :, :20], workspace=ws),
                 lambda: api.orthogonalize(x, y.bfloat16(), workspace=ws),
                 lambda: api.orthogonalize(x, y.cpu(), workspace=ws),
                 lambda: api.orthogonalize(x.double(), y.double(), workspace=ws),
                 lambda: api.orthogonalize(x, y.transpose(1, 2), workspace=ws),
                 lambda: api.orthogonalize(x.transpose(1, 2), y.transpose(1, 2), workspace=ws),
                 lambda: api.orthogonalize(x, y, workspace=ws.cpu()),
                 lambda: api.orthogonalize([x[0], torch.zeros(30, 80, device=dev)[:, :40]], y, workspace=ws),
                 lambda: api.orthogonalize(x, y, coefficients=(1.0, 2.0), workspace=ws)):
        with pytest.raises(ValueError):
            call()
    for call in (lambda: api.orthogonalize(x, y, workspace=ws[:1024]),
                 lambda: api.orthogonalize(x, y, steps=0, coefficients=[], workspace=ws),
                 lambda: api.orthogonalize(x, y, coefficients=(50.0, 50.0, 50.0), workspace=ws),
                 lambda: api.orthogonalize(x[:, 1:], x[:, :-1], workspace=ws)):
        with pytest.raises(api.ArError):
            call()
