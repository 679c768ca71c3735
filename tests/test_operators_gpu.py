"""The operators around the collectives on the GPU, against their 64-bit forms
(operator_bounds.py): every output lies between the roundings of the form's
value minus and plus the float32 computation's slack."""
import itertools
import math

import pytest

from tests import operator_bounds as ob

pytestmark = pytest.mark.gpu

EPS = 1e-6


@pytest.fixture(scope="module")
def env():
    import torch
    from collective_communication_ring_amd import api
    assert torch.cuda.is_available(), "GPU tests need a GPU"
    api.lib()
    return dict(torch=torch, api=api, dev=torch.device("cuda:0"))


def _types(torch):
    return {"f32": torch.float32, "bf16": torch.bfloat16, "e4m3": torch.float8_e4m3fn}


def _rand(env, shape, seed, dtype, scale=1.0):
    torch = env["torch"]
    g = torch.Generator().manual_seed(seed)
    return (torch.randn(shape, generator=g) * scale).to(dtype)


def _strided(env, host, pad=0, offset=0):
    """`host` on the GPU as rows of a wider array, `offset` elements into it."""
    torch = env["torch"]
    rows, cols = host.shape
    flat = torch.empty(offset + rows * (cols + pad), dtype=host.dtype, device=env["dev"])
    view = flat[offset:].view(rows, cols + pad)[:, :cols]
    view.copy_(host)
    return view


def _check_norm(env, got, form):
    for k, t in got.items():
        value, slack = form[k]
        ob.between(t.float() if k == "scale" else t, value.reshape(t.shape), slack.reshape(t.shape), k)


def _run_norm(env, rows, cols, dtype, out, group, wtype, residual, pad=0, offset=0, seed=0,
              x=None, eps=EPS):
    """Runs one norm and checks all its outputs."""
    torch, api, dev = env["torch"], env["api"], env["dev"]
    T = _types(torch)
    dt, ydt = T[dtype], T[dtype if out == "same" else out]
    hx = _rand(env, (rows, cols), 10 * seed + 1, dt) if x is None else x
    hr = _rand(env, (rows, cols), 10 * seed + 2, dt, 2.0) if residual else None
    hw = (1 + 0.2 * _rand(env, (cols,), 10 * seed + 3, torch.float32)).to(T[wtype])
    x = _strided(env, hx, pad, offset)
    r = _strided(env, hr, 2 * pad, offset) if residual else None
    w = hw.to(dev)
    y = _strided(env, torch.full((rows, cols), 3.0).to(ydt), pad, offset)
    got = {"y": y, "rstd": torch.full((rows,), -1.0, device=dev)}
    if residual:
        got["sum"] = _strided(env, torch.zeros((rows, cols), dtype=dt), pad, 2 * offset)
    if out == "e4m3":
        got["scale"] = torch.full((rows, -(-cols // group) if group else 1), -1.0, device=dev)
    api.rmsnorm(x, w, y, eps, residual=r, sum=got.get("sum"), scale=got.get("scale"), group=group,
                rstd=got["rstd"])
    torch.cuda.synchronize()
    _check_norm(env, got, ob.norm(hx, hw, eps, residual=hr, group=group if out == "e4m3" else None))


COLS = (1, 2, 7, 8, 31, 64, 100, 512, 1001, 2048, 4096, 5120, 8195, 16384)


@pytest.mark.parametrize("cols", COLS)
@pytest.mark.parametrize("dtype", ("f32", "bf16"))
def test_norm(env, dtype, cols):
    for k, (rows, residual) in enumerate(itertools.product((1, 3, 70), (False, True))):
        _run_norm(env, rows, cols, dtype, "same", 0, dtype, residual, seed=k)


@pytest.mark.parametrize("cols", COLS)
@pytest.mark.parametrize("dtype", ("f32", "bf16"))
@pytest.mark.parametrize("group", (0, 32, 64, 128, 256))
def test_norm_e4m3(env, dtype, cols, group):
    for k, rows in enumerate((1, 5)):
        _run_norm(env, rows, cols, dtype, "e4m3", group, dtype, k == 1, seed=k)


@pytest.mark.parametrize("dtype,out,cols,pad,offset", [
    ("bf16", "same", 1000, 24, 0), ("bf16", "same", 1000, 1, 0), ("bf16", "same", 1024, 0, 1),
    ("bf16", "e4m3", 1024, 7, 3), ("f32", "same", 1000, 5, 1), ("f32", "e4m3", 129, 2, 1),
    ("bf16", "same", 8200, 3, 1), ("f32", "same", 4100, 3, 1), ("bf16", "e4m3", 70, 3, 5),
    ("bf16", "same", 3, 1, 1), ("f32", "same", 40000, 1, 1),
])
def test_norm_strides_and_alignment(env, dtype, out, cols, pad, offset):
    _run_norm(env, 9, cols, dtype, out, 64 if out == "e4m3" else 0, "f32", True, pad, offset)


@pytest.mark.parametrize("dtype", ("f32", "bf16"))
@pytest.mark.parametrize("cols", (20000, 32768, 33000, 70001))
def test_norm_long_rows(env, dtype, cols):
    _run_norm(env, 3, cols, dtype, "same", 0, dtype, True)
    _run_norm(env, 2, cols, dtype, "e4m3", 0, dtype, False)
    _run_norm(env, 2, cols, dtype, "e4m3", 128, "f32", True)


@pytest.mark.parametrize("rows,cols", [(1000, 64), (257, 1001), (4099, 200), (300, 8192), (70000, 8)])
def test_norm_many_rows(env, rows, cols):
    _run_norm(env, rows, cols, "bf16", "same", 0, "bf16", True)
    _run_norm(env, rows, cols, "f32", "e4m3", 32, "f32", False)


@pytest.mark.parametrize("cols", (5, 1000, 9000, 40000))
def test_norm_extreme_values(env, cols):
    """Rows of zeros; rows whose squares leave float32's range on both sides
    (they are held in 64 bits then, and below it eps decides); a scale at its
    floor."""
    torch = env["torch"]
    for dtype, out in (("f32", "same"), ("bf16", "same"), ("f32", "e4m3")):
        x = _rand(env, (6, cols), 4, torch.float32)
        x[0] = 0
        x[1] *= 2.0 ** 66   # squares pass 2^128
        x[2] *= 2.0 ** 100
        x[3] *= 2.0 ** -80  # squares below 2^-149
        x[4] = 0
        x[4, cols // 2] = 2.0 ** -133  # its v / 448 is below the smallest scale
        x = x.to(_types(torch)[dtype])
        _run_norm(env, 6, cols, dtype, out, 32 if out == "e4m3" else 0, dtype, False, x=x)


@pytest.mark.parametrize("cols", (5, 100, 1000, 9000, 40000))
@pytest.mark.parametrize("eps", (0.0, 1e-30))
def test_norm_without_eps(env, cols, eps):
    """No eps, or hardly any: rows whose squares float32 cannot hold, below
    and above, and a row of zeros, 0 / 0 without eps."""
    torch, api, dev = env["torch"], env["api"], env["dev"]
    x = _rand(env, (5, cols), 14, torch.float32)
    x[1] *= 2.0 ** -70   # squares about 2^-140
    x[2] *= 2.0 ** -100  # squares are 0 in float32
    x[3] *= 2.0 ** 80
    _run_norm(env, 5, cols, "f32", "same", 0, "f32", False, x=x, eps=eps)
    y, rstd = torch.ones((1, cols), device=dev), torch.zeros(1, device=dev)
    api.rmsnorm(torch.zeros((1, cols), device=dev), torch.ones(cols, device=dev), y, eps, rstd=rstd)
    torch.cuda.synchronize()
    if eps:
        assert (y == 0).all() and abs(float(rstd) * eps ** 0.5 - 1) < 4 * ob.U
    else:
        assert torch.isnan(y).all() and float(rstd) == math.inf


@pytest.mark.parametrize("cols", (40, 1024, 8192, 40000))
def test_norm_infinities_and_nan(env, cols):
    """An infinity makes its row's rstd 0: it becomes NaN (and its group's
    scale), the rest 0.  A NaN makes its row NaN.  Other rows are as without."""
    torch, api, dev = env["torch"], env["api"], env["dev"]
    x = _rand(env, (4, cols), 9, torch.float32)
    x[1, 3] = math.inf
    x[2, 5] = math.nan
    w = torch.ones(cols, device=dev)
    y = torch.empty((4, cols), device=dev)
    rstd = torch.empty(4, device=dev)
    q = torch.empty((4, cols), device=dev, dtype=torch.float8_e4m3fn)
    groups = -(-cols // 32)
    scale = torch.empty((4, groups), device=dev)
    api.rmsnorm(x.to(dev), w, y, EPS, rstd=rstd)
    api.rmsnorm(x.to(dev), w, q, EPS, scale=scale, group=32)
    torch.cuda.synchronize()
    form = ob.norm(x[[0, 3]], w.cpu(), EPS, group=32)
    for got, k in ((rstd, "rstd"), (scale, "scale"), (q, "y")):
        ob.between(got.cpu()[[0, 3]], *form[k], k)
    y, rstd, q, scale = y.cpu(), rstd.cpu(), q.cpu().float(), scale.cpu()
    assert rstd[1] == 0 and torch.isnan(rstd[2])
    assert torch.isnan(y[2]).all() and torch.isnan(q[2]).all() and torch.isnan(scale[2]).all()
    assert torch.isnan(y[1, 3]) and (y[1, :3] == 0).all() and (y[1, 4:] == 0).all()
    assert torch.isnan(q[1, :32]).all() and (q[1, 32:] == 0).all()
    assert torch.isnan(scale[1, 0]) and (scale[1, 1:] == ob.TINY).all()


@pytest.mark.parametrize("dtype", ("f32", "bf16"))
@pytest.mark.parametrize("cols", (33, 4096, 40000))
def test_norm_in_place(env, dtype, cols):
    """sum over the residual's or x's array, y over x's: the same bits as
    apart from them."""
    torch, api, dev = env["torch"], env["api"], env["dev"]
    dt = _types(torch)[dtype]
    x, r = (_rand(env, (65, cols), s, dt).to(dev) for s in (1, 2))
    w = _rand(env, (cols,), 3, dt).to(dev)
    y, h = torch.empty_like(x), torch.empty_like(x)
    api.rmsnorm(x, w, y, EPS, residual=r, sum=h)
    for how in ("sum=residual", "sum=x", "y=x,sum=residual"):
        a, b = x.clone(), r.clone()
        out = a if how.startswith("y") else torch.empty_like(x)
        s = a if how == "sum=x" else b
        api.rmsnorm(a, w, out, EPS, residual=b, sum=s)
        torch.cuda.synchronize()
        assert torch.equal(out, y) and torch.equal(s, h), how


@pytest.mark.parametrize("cols", (70, 4096, 40000))
def test_e4m3_of_a_product_that_overflows(env, cols):
    """v = h r w past float32's range: its group's scale is infinite, it
    becomes NaN and the rest of the group 0; the other groups are as without."""
    torch, api, dev = env["torch"], env["api"], env["dev"]
    x = _rand(env, (3, cols), 2, torch.float32)
    x[:, 40] = 3.0
    w = torch.ones(cols)
    w[40] = 3e38
    groups = -(-cols // 32)
    q = torch.empty((3, cols), device=dev, dtype=torch.float8_e4m3fn)
    scale = torch.empty((3, groups), device=dev)
    api.rmsnorm(x.to(dev), w.to(dev), q, EPS, scale=scale, group=32)
    torch.cuda.synchronize()
    w[40] = 1.0  # for the other groups
    form = ob.norm(x, w, EPS, group=32)
    keep = torch.ones(cols, dtype=torch.bool)
    keep[32:64] = False
    ob.between(q[:, keep.to(dev)], *(t[:, keep] for t in form["y"]), "y")
    q, scale = q.cpu().float(), scale.cpu()
    assert (scale[:, 1] == math.inf).all() and torch.isnan(q[:, 40]).all()
    assert (q[:, 32:40] == 0).all() and (q[:, 41:64] == 0).all()


def _guarded(env, rows, cols, dtype, pad, offset):
    """Rows of a wider array whose other elements hold a mark, the array, and a
    check that these still do."""
    torch = env["torch"]
    flat = torch.full((offset + rows * (cols + pad) + 40,), 3.0, device=env["dev"]).to(dtype)
    view = flat[offset:offset + rows * (cols + pad)].view(rows, cols + pad)[:, :cols]

    def untouched():
        rest = flat.clone()
        rest[offset:offset + rows * (cols + pad)].view(rows, cols + pad)[:, :cols] = 3.0
        assert (rest.float() == 3.0).all()
    return view, untouched


@pytest.mark.parametrize("cols,pad,offset", [
    (1, 3, 1), (5, 2, 0), (8, 1, 3), (63, 1, 2), (64, 8, 8), (500, 7, 1), (1001, 3, 5), (2057, 1, 1),
    (4099, 5, 0), (8192, 16, 0), (9001, 2, 1), (17003, 1, 1), (33001, 3, 1),
])
@pytest.mark.parametrize("dtype", ("f32", "bf16"))
def test_nothing_beside_the_outputs_is_written(env, dtype, cols, pad, offset):
    torch, api, dev = env["torch"], env["api"], env["dev"]
    dt = _types(torch)[dtype]
    rows, e4m3, f32 = 5, torch.float8_e4m3fn, torch.float32
    x, res, dy = (_rand(env, (rows, cols), s, dt).to(dev) for s in (1, 2, 3))
    w = torch.ones(cols, device=dev, dtype=dt)
    for group in (None, 0, 32):
        groups = -(-cols // group) if group else 1
        outs = {"y": _guarded(env, rows, cols, dt if group is None else e4m3, pad, offset),
                "sum": _guarded(env, rows, cols, dt, pad, 2 * offset),
                "rstd": _guarded(env, 1, rows, f32, pad, offset)}
        if group is not None:
            outs["scale"] = _guarded(env, 1, rows * groups, f32, pad, offset)
        o = {k: v[0] for k, v in outs.items()}
        api.rmsnorm(x, w, o["y"], EPS, residual=res, sum=o["sum"], rstd=o["rstd"][0], group=group or 0,
                    scale=o["scale"].view(rows, groups) if group is not None else None)
        torch.cuda.synchronize()
        for _, untouched in outs.values():
            untouched()
    r = torch.ones(rows, device=dev)
    dx, untouched_dx = _guarded(env, rows, cols, dt, pad, offset)
    dw, untouched_dw = _guarded(env, 1, cols, f32, pad, offset)
    ws, untouched_ws = _guarded(env, 1, max(64, api.ar_rmsnorm_backward_workspace(1, rows, cols) // 4),
                                f32, 0, 64)
    api.rmsnorm_backward(dy, x, w, r, dx, dw, dsum=res, workspace=ws[0])
    torch.cuda.synchronize()
    untouched_dx(), untouched_dw(), untouched_ws()


def test_norm_interleaved_rows(env):
    """x and y as the halves of one array's rows: no overlap."""
    torch, api, dev = env["torch"], env["api"], env["dev"]
    buf = torch.zeros((50, 600), device=dev)
    hx = _rand(env, (50, 300), 1, torch.float32)
    buf[:, :300] = hx.to(dev)
    w = torch.ones(300, device=dev)
    api.rmsnorm(buf[:, :300], w, buf[:, 300:], EPS)
    torch.cuda.synchronize()
    ob.between(buf[:, 300:], *ob.norm(hx, w.cpu(), EPS)["y"], "y")
    assert torch.equal(buf[:, :300].cpu(), hx)
    with pytest.raises(api.ArError):
        api.rmsnorm(buf[:, :300], w, buf[:, 299:599], EPS)


def test_norm_rows_past_32_bits(env):
    """Rows 2^32 + 8 elements apart, in every array."""
    torch, api, dev = env["torch"], env["api"], env["dev"]
    cols, stride = 520, (1 << 32) + 8
    hx, hr = (_rand(env, (2, cols), s, torch.bfloat16) for s in (1, 2))
    big = torch.empty(stride + cols, dtype=torch.bfloat16, device=dev)
    x = big.as_strided((2, cols), (stride, 1))
    x.copy_(hx)
    y = torch.empty(stride + cols, dtype=torch.bfloat16, device=dev).as_strided((2, cols), (stride, 1))
    w = torch.ones(cols, device=dev)
    r = hr.to(dev)
    api.rmsnorm(x, w, y, EPS, residual=r, sum=x)
    torch.cuda.synchronize()
    form = ob.norm(hx, w.cpu(), EPS, residual=hr)
    ob.between(y, *form["y"], "y")
    ob.between(x, *form["sum"], "sum")


def test_norm_of_more_rows_than_a_launch_holds(env):
    """2^26 + 5 rows of 64 lanes each are past 2^32 threads: 35 GB of rows, by
    three launches; rows on both sides of their borders are checked."""
    torch, api, dev = env["torch"], env["api"], env["dev"]
    rows, cols = (1 << 26) + 5, 264
    at = sorted({0, 1, (1 << 25) - 1, 1 << 25, (1 << 25) + 3, (1 << 26) - 1, 1 << 26, rows - 1})
    hx = _rand(env, (len(at), cols), 1, torch.bfloat16)
    x = torch.ones((rows, cols), dtype=torch.bfloat16, device=dev)
    x[at] = hx.to(dev)
    w = torch.ones(cols, device=dev)
    y = torch.zeros_like(x)
    api.rmsnorm(x, w, y, EPS)
    torch.cuda.synchronize()
    ob.between(y[at], *ob.norm(hx, w.cpu(), EPS)["y"], "y")
    some = torch.arange(7, rows, 65537, device=dev)  # the rows of ones: 1 / sqrt(1 + eps) is 1
    some = some[~torch.isin(some, torch.tensor(at, device=dev))]
    assert (y[some] == 1).all()


# ---- behind a reduce-scatter --------------------------------------------------

@pytest.mark.parametrize("R,tokens,cols,dtype,out,group,residual,redop", [
    (2, 1, 1, "f32", "same", 0, False, "sum"),
    (8, 1, 4096, "bf16", "same", 0, True, "sum"),
    (8, 5, 1000, "f32", "same", 0, True, "avg"),
    (3, 7, 1001, "bf16", "e4m3", 64, True, "sum"),
    (16, 2, 513, "f32", "e4m3", 0, False, "sum"),
    (5, 33, 100, "bf16", "same", 0, True, "avg"),
    (64, 1, 8200, "bf16", "e4m3", 128, False, "sum"),
    (4, 3, 40000, "f32", "same", 0, True, "sum"),
    (8, 64, 8192, "bf16", "e4m3", 128, True, "sum"),
    (7, 9, 16384, "f32", "same", 0, True, "sum"),
])
def test_reduce_scatter_norm(env, R, tokens, cols, dtype, out, group, residual, redop):
    torch, api, dev = env["torch"], env["api"], env["dev"]
    T = _types(torch)
    dt = T[dtype]
    hs = _rand(env, (R, R * tokens * cols), 1, dt)
    hr = _rand(env, (R, tokens * cols), 2, dt) if residual else None
    hw = (1 + 0.2 * _rand(env, (cols,), 3, torch.float32)).to(dt)
    comm = api.Comm(R, R * tokens * cols, "bf16" if dtype == "bf16" else "float32", device=dev,
                    redop=redop)
    send = hs.to(dev)
    got = {"y": torch.empty((R, tokens * cols), dtype=T[dtype if out == "same" else out], device=dev),
           "rstd": torch.empty((R, tokens), device=dev),
           "sum": torch.empty((R, tokens * cols), dtype=dt, device=dev)}
    if out == "e4m3":
        got["scale"] = torch.empty((R, tokens * (-(-cols // group) if group else 1)), device=dev)
    comm.reduce_scatter_rmsnorm(send, hw.to(dev), got["y"], EPS,
                                residual=hr.to(dev) if residual else None, sum=got["sum"],
                                scale=got.get("scale"), group=group, rstd=got["rstd"])
    torch.cuda.synchronize()
    form = ob.norm(None, hw, EPS, residual=hr.view(-1, cols) if residual else None,
                   parts=hs.view(R, R * tokens, cols), divisor=R if redop == "avg" else 1.0,
                   group=group if out == "e4m3" else None)
    _check_norm(env, got, form)
    if dtype == "f32":  # the fold's order is the reduce-scatter's own: the same bits
        shard = torch.empty((R, tokens * cols), device=dev)
        comm.reduce_scatter(send, shard)
        if residual:
            shard += hr.to(dev)
        torch.cuda.synchronize()
        assert torch.equal(shard, got["sum"])
    assert comm.check() == api.AR_SUCCESS
    comm.close()


# ---- backward -----------------------------------------------------------------

def _run_back(env, ranks, rows, cols, dtype, wtype, dsum, pad=0, offset=0, dx_over=None):
    torch, api, dev = env["torch"], env["api"], env["dev"]
    T = _types(torch)
    dt = T[dtype]
    hx, hd = _rand(env, (rows, cols), 1, dt, 1.5), _rand(env, (rows, cols), 2, dt)
    hs = _rand(env, (rows, cols), 3, dt) if dsum else None
    hw = (1 + 0.2 * _rand(env, (cols,), 4, torch.float32)).to(T[wtype])
    hr = ob.norm(hx, hw, EPS)["rstd"][0].float()
    x, dy = _strided(env, hx, pad, offset), _strided(env, hd, 3 * pad, 2 * offset)
    ds = _strided(env, hs, pad, offset) if dsum else None
    dx = {None: None, "dy": dy, "x": x, "dsum": ds}[dx_over]
    if dx is None:
        dx = _strided(env, torch.zeros((rows, cols), dtype=dt), pad, offset)
    dw = torch.full((ranks, cols), 5.0, device=dev)
    api.rmsnorm_backward(dy, x, hw.to(dev), hr.to(dev), dx, dw, dsum=ds)
    torch.cuda.synchronize()
    form = ob.norm_backward(hd, hx, hw, hr, dsum=hs, ranks=ranks)
    ob.between(dx, *form["dx"], "dx")
    ob.between(dw, *form["dweight"], "dweight")
    return dx.clone(), dw


@pytest.mark.parametrize("cols", COLS + (20000, 33000, 70001))
@pytest.mark.parametrize("dtype", ("f32", "bf16"))
def test_backward(env, dtype, cols):
    for ranks, rows, dsum in ((1, 1, False), (1, 70, True), (4, 12, False), (8, 8, True)):
        _run_back(env, ranks, rows, cols, dtype, dtype, dsum)


@pytest.mark.parametrize("ranks,rows,cols,dtype,wtype,pad,offset", [
    (1, 3000, 64, "bf16", "bf16", 0, 0), (1, 2500, 1000, "f32", "f32", 24, 0),
    (8, 8 * 313, 1001, "bf16", "f32", 1, 1), (64, 64, 100, "f32", "f32", 0, 1),
    (3, 9, 8193, "bf16", "f32", 5, 3), (1, 70000, 8, "f32", "f32", 0, 0),
    (2, 1026, 4096, "bf16", "bf16", 8, 8),
])
def test_backward_shapes(env, ranks, rows, cols, dtype, wtype, pad, offset):
    _run_back(env, ranks, rows, cols, dtype, wtype, True, pad, offset)


@pytest.mark.parametrize("dtype", ("f32", "bf16"))
@pytest.mark.parametrize("cols", (31, 2048, 40000))
def test_backward_in_place(env, dtype, cols):
    """dx over each of its inputs gives the bits it gives apart from them."""
    want = _run_back(env, 2, 66, cols, dtype, dtype, True)
    for over in ("dy", "x", "dsum"):
        got = _run_back(env, 2, 66, cols, dtype, dtype, True, dx_over=over)
        assert env["torch"].equal(got[0], want[0]) and env["torch"].equal(got[1], want[1]), over


def test_backward_of_nothing(env):
    """No rows: the weight's gradient is zero, not what was there."""
    torch, api, dev = env["torch"], env["api"], env["dev"]
    e = torch.empty((0, 40), device=dev)
    dw = torch.full((3, 40), 9.0, device=dev)
    api.rmsnorm_backward(e, e, torch.ones(40, device=dev), torch.empty(0, device=dev), e.clone(), dw)
    torch.cuda.synchronize()
    assert (dw == 0).all()
    api.rmsnorm(e, torch.ones(40, device=dev), e.clone(), rstd=torch.empty(0, device=dev))


def test_backward_against_differences(env):
    """dx and dweight against central differences of the 64-bit forward form.
    The differences are off by about step^2 = 1e-10; the kernel by the form's
    slack."""
    torch, api, dev = env["torch"], env["api"], env["dev"]
    T, C, step = 3, 17, 1e-5
    hx, hd, hw = (_rand(env, s, k, torch.float32) for k, s in enumerate(((T, C), (T, C), (C,))))
    f = ob.norm(hx, hw, 1e-3)
    dx = torch.empty((T, C), device=dev)
    dw = torch.empty((1, C), device=dev)
    rstd = torch.empty(T, device=dev)
    y = torch.empty((T, C), device=dev)
    api.rmsnorm(hx.to(dev), hw.to(dev), y, 1e-3, rstd=rstd)
    api.rmsnorm_backward(hd.to(dev), hx.to(dev), hw.to(dev), rstd, dx, dw)
    torch.cuda.synchronize()
    form = ob.norm_backward(hd, hx, hw, f["rstd"][0])
    x, w, dy = hx.double(), hw.double(), hd.double()
    for at, got, slack in ((x, dx, form["dx"][1]), (w, dw, form["dweight"][1])):
        flat = at.view(-1)
        # rstd itself is float32: its relative error, about 4 U, passes into the gradient
        room = slack.view(-1) + 8 * ob.U * float(got.abs().max()) + 1e-8
        for i in range(flat.numel()):
            old = float(flat[i])
            loss = []
            for v in (old + step, old - step):
                flat[i] = v
                loss.append(float((ob.norm(x, w, 1e-3)["y"][0] * dy).sum()))
            flat[i] = old
            assert abs((loss[0] - loss[1]) / (2 * step) - float(got.view(-1)[i])) <= float(room[i])


# ---- gradient norm and clipping -------------------------------------------------

def _check_clip(env, tensors, max_norm, inplace, given=None):
    """The norm is within half a float32 step (64-bit sums leave nothing else),
    and each product within three float32 roundings before its own."""
    torch, api, dev = env["torch"], env["api"], env["dev"]
    comm = api.Comm(2, 4, "float32", device=dev)
    host = [t.detach().cpu() for t in tensors]
    norm = torch.full((1,), -1.0, device=dev)
    comm.grad_norm(given if given is not None else tensors, norm)
    total = sum(float((h.double() ** 2).sum()) for h in host)
    want = math.sqrt(total)
    torch.cuda.synchronize()
    n = float(norm)
    assert abs(n - want) <= 1.0001 * ob.U * want, (n, want)
    out = None if inplace else [torch.empty_like(t) for t in tensors]
    comm.grad_clip(tensors, norm, max_norm, out=out)
    torch.cuda.synchronize()
    c = min(1.0, max_norm / (n + 1e-6))
    for h, t, o in zip(host, tensors, tensors if inplace else out):
        v = h.double() * c
        if c == 1.0:
            assert torch.equal(o.cpu(), h)
        else:
            ob.between(o, v, 3.001 * ob.U * v.abs(), "clipped")
        if not inplace:
            assert torch.equal(t.cpu(), h)
    assert comm.check() == api.AR_SUCCESS
    comm.close()


def _many(env, sizes, seed=1, types=("f32", "bf16"), offsets=False):
    """Tensors of these sizes in turn of each type, cut from one array per type
    so that most begin off a 16-byte boundary."""
    torch = env["torch"]
    T = _types(torch)
    got = []
    for i, n in enumerate(sizes):
        dt = T[types[i % len(types)]]
        lead = (i * 3) % 9 if offsets else 0
        t = torch.empty(n + lead, dtype=dt, device=env["dev"])[lead:]
        t.copy_(_rand(env, (n,), seed + i, torch.float32, 0.02))
        got.append(t)
    return got


@pytest.mark.parametrize("sizes", [
    (1,), (7,), (8,), (1000,), (16384, 16385, 1), (4096 * 4 + 3,), (300001, 5, 70000),
    (0, 3, 0, 10, 0), (1 << 22,),
])
@pytest.mark.parametrize("inplace", (False, True))
def test_clip(env, sizes, inplace):
    for offsets in (False, True):
        norm = 0.02 * math.sqrt(sum(sizes))
        _check_clip(env, _many(env, sizes, offsets=offsets), norm / 3, inplace)
        _check_clip(env, _many(env, sizes, types=("bf16",), offsets=offsets), norm * 100, inplace)


@pytest.mark.parametrize("count", (128, 129, 700))
def test_clip_many_tensors(env, count):
    """More tensors than one launch's table holds, empty ones among them."""
    sizes = [(i * i * 37) % 5003 for i in range(count)]
    _check_clip(env, _many(env, sizes, offsets=True), 0.1, True)
    _check_clip(env, _many(env, sizes, offsets=True), 0.1, False)


@pytest.mark.parametrize("count", (3, 190, 400))
@pytest.mark.parametrize("buffers", (1, 4, 5, 97))
def test_clip_into_buffers(env, count, buffers):
    """Outputs cut from a number of buffers in turn: at up to four distances
    from their inputs a table holds no addresses of outputs."""
    torch, dev = env["torch"], env["dev"]
    sizes = [(i * 911) % 3001 + 1 for i in range(count)]
    total = sum(sizes) + 8
    src = _rand(env, (total,), 3, torch.float32, 0.02).bfloat16().to(dev)
    dst = [torch.full((total,), 7.0, device=dev).bfloat16() for _ in range(buffers)]
    comm = env["api"].Comm(2, 4, "float32", device=dev)
    norm = torch.full((1,), 3.0, device=dev)
    grads, out, lo = [], [], 3
    for i, n in enumerate(sizes):
        grads.append(src[lo:lo + n])
        out.append(dst[i % buffers][lo:lo + n])
        lo += n
    comm.grad_clip(grads, norm, 0.75, out=out)
    torch.cuda.synchronize()
    c = 0.75 / (3.0 + 1e-6)
    for g, o in zip(grads, out):
        v = g.cpu().double() * c
        ob.between(o, v, 3.001 * ob.U * v.abs(), "clipped")
    for k, d in enumerate(dst):  # and nothing beside them
        want, lo = torch.full_like(d, 7.0), 3
        for i, n in enumerate(sizes):
            if i % buffers == k:
                want[lo:lo + n] = out[i]
            lo += n
        assert torch.equal(d, want)
    comm.close()


def test_clip_tensor_list(env):
    """A TensorList kept over calls, dense tensors of any dimension order, and
    an address that changes under it."""
    torch, api = env["torch"], env["api"]
    ts = [t.view(40, 25).t() for t in _many(env, (1000, 1000))] + _many(env, (77,))
    kept = api.TensorList(ts)
    _check_clip(env, ts, 0.2, False, given=kept)
    ts[0].data = ts[0].detach().clone() * 3
    _check_clip(env, ts, 0.2, False, given=kept)
    with pytest.raises(ValueError):
        api.TensorList([ts[0][:, :3][:, ::2]])
    comm = api.Comm(2, 4, "float32")
    norm = torch.zeros(1, device=env["dev"])
    with pytest.raises(ValueError):
        comm.grad_clip(ts, norm, 1.0, out=[t.contiguous() for t in ts])  # other strides
    with pytest.raises(ValueError):
        comm.grad_norm(ts, torch.zeros(2, device=env["dev"]))
    with pytest.raises(api.ArError):
        comm.grad_norm(ts[2:], ts[2][:1])  # the norm inside a gradient
    comm.close()


def test_grad_norm_of_nothing(env):
    torch, api, dev = env["torch"], env["api"], env["dev"]
    comm = api.Comm(2, 4, "float32", device=dev)
    for ts in ([], [torch.empty(0, device=dev)] * 3):
        norm = torch.full((1,), 4.0, device=dev)
        comm.grad_norm(ts, norm)
        torch.cuda.synchronize()
        assert float(norm) == 0.0
        comm.grad_clip(ts, norm, 1.0)
    comm.close()


def test_grad_norm_range(env):
    """Squares outside float32's range: large, denormal, and both at once;
    infinities and NaN; and what clipping makes of them."""
    torch, api, dev = env["torch"], env["api"], env["dev"]
    comm = api.Comm(2, 4, "float32", device=dev)
    norm = torch.empty(1, device=dev)

    def of(*values):
        t = torch.tensor(values, device=dev)
        comm.grad_norm([t[:1], t[1:]], norm)
        clipped = torch.empty_like(t)
        comm.grad_clip([t], norm, 1.0, out=[clipped])
        torch.cuda.synchronize()
        return float(norm), clipped.cpu()
    for scale in (2.0 ** 120, 2.0 ** -140):
        n, c = of(3 * scale, 4 * scale)
        assert n == 5 * scale
    n, c = of(3e38, 3e38, 3e38)
    assert n == math.inf and (c == 0).all()
    n, c = of(1.0, math.inf)
    assert n == math.inf and c[0] == 0 and torch.isnan(c[1])
    n, c = of(1.0, -math.inf, math.nan)
    assert math.isnan(n) and torch.isnan(c).all()
    n, c = of(-0.0, 0.0)
    assert n == 0 and (c == 0).all()
    comm.close()


def test_grad_norm_long_tensor(env):
    """A tensor past 2^32 elements, its only values other than zero beyond
    them; clipped in place."""
    torch, api, dev = env["torch"], env["api"], env["dev"]
    n = (1 << 32) + 4099
    t = torch.zeros(n, dtype=torch.bfloat16, device=dev)
    t[-4000:] = 2.0
    t[5] = 3.0
    comm = api.Comm(2, 4, "float32", device=dev)
    norm = torch.empty(1, device=dev)
    comm.grad_norm([t], norm)
    comm.grad_clip([t], norm, 1.0)
    torch.cuda.synchronize()
    want = math.sqrt(4000 * 4.0 + 9.0)
    assert abs(float(norm) - want) <= 1.0001 * ob.U * want
    v = torch.full((4000,), 2.0, dtype=torch.float64) / (float(norm) + 1e-6)
    ob.between(t[-4000:], v, 3.001 * ob.U * v, "clipped")
    assert float(t[6:-4000].abs().max()) == 0.0
    comm.close()


# ---- streams, graphs, repeats -----------------------------------------------------

def _step(env, s):
    """A norm, its backward pass, and the clipping of both gradients."""
    api = env["api"]
    s["comm"].reduce_scatter_rmsnorm(s["send"], s["w"], s["y"], EPS, residual=s["res"], sum=s["h"],
                                     rstd=s["rstd"])
    h = s["h"].view(-1, s["w"].numel())
    api.rmsnorm_backward(s["dy"], h, s["w"], s["rstd"].view(-1), s["dx"], s["dw"],
                         workspace=s["ws"])
    s["comm"].grad_norm([s["dx"], s["dw"]], s["norm"])
    s["comm"].grad_clip([s["dx"], s["dw"]], s["norm"], 1.0, out=[s["cx"], s["cw"]])


def _state(env, R=4, tokens=65, cols=1000):
    torch, api, dev = env["torch"], env["api"], env["dev"]
    n = R * tokens
    e = lambda *shape: torch.empty(shape, device=dev)  # noqa: E731
    return dict(comm=api.Comm(R, n * cols, "float32", device=dev), send=e(R, n * cols),
                res=e(R, tokens * cols), w=e(cols), y=e(R, tokens * cols), h=e(R, tokens * cols),
                rstd=e(R, tokens), dy=e(n, cols), dx=e(n, cols), dw=e(R, cols), norm=e(1),
                cx=e(n, cols), cw=e(R, cols), ws=api.rmsnorm_backward_workspace(R, n, cols, dev))


def _fill(env, s, seed):
    g = env["torch"].Generator(device=env["dev"])
    g.manual_seed(seed)
    for k in ("send", "res", "w", "dy"):
        s[k].normal_(generator=g)


OUT = ("y", "h", "rstd", "dx", "dw", "norm", "cx", "cw")


def test_step_in_a_graph(env):
    """Captured once, replayed on other inputs with eager calls of the same
    buffers and allocations in between: each replay has the eager call's
    bits."""
    torch = env["torch"]
    s, e = _state(env), _state(env)
    _fill(env, s, 0)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        _step(env, s)
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        _step(env, s)
    for seed in range(1, 5):
        _fill(env, e, seed)
        _step(env, e)
        _fill(env, s, seed)
        for k in OUT:
            s[k].fill_(-2.0)
        torch.randn(1000, device=env["dev"]).sum().item()
        graph.replay()
        torch.cuda.synchronize()
        for k in OUT:
            assert torch.equal(s[k], e[k]), (seed, k)
        _step(env, s)  # eager, on the graph's own buffers and workspace
        torch.cuda.synchronize()
        for k in OUT:
            assert torch.equal(s[k], e[k]), (seed, k)


def test_step_on_another_stream_and_twice(env):
    """The same bits on a stream given by the caller, and again."""
    torch, api, dev = env["torch"], env["api"], env["dev"]
    a, b = _state(env), _state(env)
    _fill(env, a, 7)
    _fill(env, b, 7)
    _step(env, a)
    torch.cuda.synchronize()
    st = torch.cuda.Stream()
    with torch.cuda.stream(st):
        _step(env, b)
        _step(env, b)
    st.synchronize()
    for k in OUT:
        assert torch.equal(a[k], b[k]), k
    y = torch.empty_like(a["dx"])
    api.rmsnorm(a["dy"], a["w"], y, EPS, stream=st)
    dx, dw = torch.empty_like(a["dx"]), torch.empty_like(a["dw"])
    api.rmsnorm_backward(a["dy"], a["h"].view(-1, 1000), a["w"], a["rstd"].view(-1), dx, dw, stream=st)
    a["comm"].grad_norm([dx, dw], a["norm"], stream=st)
    st.synchronize()
    assert torch.equal(dx, b["dx"]) and torch.equal(dw, b["dw"]) and torch.equal(a["norm"], b["norm"])


def test_grad_norm_between_collectives(env):
    """The norm's ticket and sums lie in the comm's workspace: collectives of
    every form before and after it, on one stream, are not disturbed."""
    torch, api, dev = env["torch"], env["api"], env["dev"]
    for algo, proto, launch in (("ring", "simple", "pipelined"), ("tree", "ll", None),
                                ("ring", "ll", None), ("ring", "simple", "step")):
        comm = api.Comm(4, 5000, "float32", algo, proto, device=dev, launch=launch)
        x = _rand(env, (4, 5000), 3, torch.float32).to(dev)
        want, got = torch.empty_like(x), torch.empty_like(x)
        comm.allreduce(x, want)
        norm = torch.empty(1, device=dev)
        for _ in range(3):
            comm.grad_norm([want[0]], norm)
            comm.allreduce(x, got)
            comm.grad_clip([got[q] for q in range(4)], norm, 1e9)
        torch.cuda.synchronize()
        assert comm.check() == api.AR_SUCCESS and torch.equal(got, want)
        ref = math.sqrt(float((want[0].double() ** 2).sum()))
        assert abs(float(norm) - ref) <= 1.0001 * ob.U * ref
        comm.close()


def test_refused_tensors(env):
    torch, api, dev = env["torch"], env["api"], env["dev"]
    x, w = torch.zeros((3, 8), device=dev), torch.zeros(8, device=dev)
    y = torch.zeros_like(x)
    for kw in (dict(residual=x[:2]), dict(residual=x.cpu()), dict(sum=x.double()), dict(rstd=w),
               dict(residual=x.t().contiguous().t()), dict(rstd=torch.zeros(6, device=dev)[::2])):
        with pytest.raises(ValueError):
            api.rmsnorm(x, w, y, **kw)
    with pytest.raises(api.ArError):
        api.rmsnorm(x, w, y, eps=-1.0)
    with pytest.raises(api.ArError):
        api.rmsnorm(x[:1].expand(3, 8), w, y)  # rows on top of each other
    with pytest.raises(api.ArError):
        api.rmsnorm(x, w, x.view(-1)[:24].view(3, 8), residual=y, sum=x)  # two outputs in one array
    comm = api.Comm(2, 96, "float32", device=dev)
    send, y2 = torch.zeros((2, 96), device=dev), torch.zeros((2, 48), device=dev)
    comm.reduce_scatter_rmsnorm(send, w, y2)
    for bad in (lambda: comm.reduce_scatter_rmsnorm(send[:, :80].contiguous(), w, y2),
                lambda: comm.reduce_scatter_rmsnorm(send, w, y2[:, :47].contiguous()),
                lambda: comm.reduce_scatter_rmsnorm(send, w, y2, residual=send),
                lambda: comm.reduce_scatter_rmsnorm(send.bfloat16(), w, y2)):
        with pytest.raises(ValueError):
            bad()
    with pytest.raises(ValueError):
        comm.grad_clip([x], torch.zeros(1), 1.0)
    with pytest.raises(api.ArError):
        comm.grad_clip([x], torch.zeros(1, device=dev), -1.0)
    torch.cuda.synchronize()
    comm.close()
