"""Host side of the operators around the collectives: what they refuse, before
anything touches a device, and the 64-bit forms the GPU tests compare with."""
import ctypes
import os

import pytest
import torch

from tests import operator_bounds as ob


@pytest.fixture(scope="module")
def api():
    from collective_communication_ring_amd import api
    if not os.path.exists(api.LIB_PATH) or not os.path.exists(os.path.join(api.HERE, "_binding.so")):
        import __graft_entry__
        __graft_entry__.build()
    api.lib()
    return api


# device addresses that no refused call touches
X, RES, W, SUM, Y, SCALE, RSTD = (0x10000000 * k for k in range(1, 8))


def _norm(api, **change):
    f = dict(dtype=api.AR_BF16, out_dtype=api.AR_BF16, weight_dtype=api.AR_BF16, eps=1e-6, rows=4,
             cols=100, group=0, x=X, x_stride=100, residual=RES, residual_stride=100, weight=W,
             sum=SUM, sum_stride=100, y=Y, y_stride=100, scale=None, rstd=RSTD)
    f.update(change)
    a = api.ar_rmsnorm_t()
    for k, v in f.items():
        setattr(a, k, v)
    return a


@pytest.mark.parametrize("change", [
    dict(dtype=0, out_dtype=0), dict(dtype=3, out_dtype=3), dict(dtype=9), dict(out_dtype=1),
    dict(weight_dtype=0), dict(weight_dtype=3),
    dict(eps=-1.0), dict(eps=float("nan")), dict(eps=float("inf")),
    dict(x=None), dict(weight=None), dict(y=None),
    dict(x_stride=99), dict(residual_stride=3), dict(sum_stride=0), dict(y_stride=99),
    dict(x=X + 1), dict(residual=RES + 1), dict(sum=SUM + 1), dict(y=Y + 1), dict(weight=W + 1),
    dict(rstd=RSTD + 2), dict(cols=(1 << 28) + 1, x_stride=1 << 31), dict(x_stride=1 << 45),
    dict(rows=1 << 60), dict(rows=(1 << 64) - 1),
    dict(out_dtype=3), dict(out_dtype=3, scale=SCALE + 2),
    dict(out_dtype=3, scale=SCALE, group=16), dict(out_dtype=3, scale=SCALE, group=100),
    dict(out_dtype=3, scale=SCALE, group=512),
])
def test_norm_refuses_bad_arguments(api, change):
    a = _norm(api, **change)
    assert api.lib().ar_rmsnorm(ctypes.byref(a), None) == api.AR_ERR_INVALID_ARG


@pytest.mark.parametrize("change", [
    dict(y=SUM), dict(y=X + 2), dict(y=X, y_stride=101), dict(sum=RES + 50), dict(sum=W),
    dict(y=W - 100), dict(rstd=Y + 4), dict(rstd=SUM), dict(sum=X, y=X),
    dict(out_dtype=3, scale=SCALE, y=X), dict(out_dtype=3, scale=X),
    # rows between another's rows: 100 columns of 180 leave 80, not enough for another 100
    dict(x_stride=180, y=X + 2 * 100, y_stride=180),
    # one row across a gap
    dict(weight=Y + 2 * 99),
])
def test_norm_refuses_overlaps(api, change):
    a = _norm(api, **change)
    assert api.lib().ar_rmsnorm(ctypes.byref(a), None) == api.AR_ERR_INVALID_USAGE


def test_norm_of_nothing(api):
    L = api.lib()
    for empty in (dict(rows=0), dict(cols=0), dict(rows=0, x=None, weight=None, y=None)):
        assert L.ar_rmsnorm(ctypes.byref(_norm(api, **empty)), None) == api.AR_SUCCESS
    assert L.ar_rmsnorm(None, None) == api.AR_ERR_INVALID_ARG


def test_reduce_scatter_norm_refusals(api):
    L = api.lib()
    c = api.ar_init(4, 4 * 300, api.AR_BF16)
    try:
        def call(send=X, **change):
            a = _norm(api, **{**dict(rows=3), **change})
            return L.ar_reduce_scatter_rmsnorm(c, send, ctypes.byref(a), None)
        assert call(rows=4) == api.AR_ERR_INVALID_ARG             # 4 * 4 * 100 > 1200
        assert call(rows=1 << 62) == api.AR_ERR_INVALID_ARG       # R * rows wraps around
        assert call(send=None) == api.AR_ERR_INVALID_ARG
        assert call(weight_dtype=7) == api.AR_ERR_INVALID_ARG
        assert call(y=X) == api.AR_ERR_INVALID_USAGE              # send cannot be overwritten
        assert call(sum=X + 2 * 4700) == api.AR_ERR_INVALID_USAGE
        assert call(y=SUM) == api.AR_ERR_INVALID_USAGE
        assert call(rows=0) == api.AR_SUCCESS
        assert L.ar_reduce_scatter_rmsnorm(None, X, ctypes.byref(_norm(api)), None) == api.AR_ERR_INVALID_ARG
        assert L.ar_reduce_scatter_rmsnorm(c, X, None, None) == api.AR_ERR_INVALID_ARG
        api.ar_set_option(c, api.AR_OPT_REDOP, api.AR_MAX)
        assert call() == api.AR_ERR_UNSUPPORTED
        api.ar_set_option(c, api.AR_OPT_REDOP, api.AR_SUM)
        api.ar_set_option(c, api.AR_OPT_ALGO, api.AR_TREE)
        assert call() == api.AR_ERR_UNSUPPORTED
    finally:
        api.ar_destroy(c)
    c = api.ar_init(4, 1200, api.AR_INT32)
    try:
        assert L.ar_reduce_scatter_rmsnorm(c, X, ctypes.byref(_norm(api)), None) == api.AR_ERR_UNSUPPORTED
    finally:
        api.ar_destroy(c)


def test_e4m3_is_no_comm_type(api):
    h = ctypes.c_void_p()
    for algo in (api.AR_RING, api.AR_TREE, api.AR_AUTO):
        assert api.lib().ar_init(ctypes.byref(h), 4, 64, api.AR_E4M3, algo, api.AR_SIMPLE) == \
            api.AR_ERR_INVALID_ARG


DY, BX, BW, BR, DS, DX, DW, WS = (0x20000000 * k for k in range(1, 9))


def _back(api, **change):
    f = dict(dtype=api.AR_FLOAT32, weight_dtype=api.AR_FLOAT32, ranks=2, rows=6, cols=50, dy=DY,
             dy_stride=50, x=BX, x_stride=50, weight=BW, rstd=BR, dsum=DS, dsum_stride=50, dx=DX,
             dx_stride=50, dweight=DW, workspace=WS,
             workspace_bytes=api.ar_rmsnorm_backward_workspace(2, 6, 50))
    f.update(change)
    a = api.ar_rmsnorm_backward_t()
    for k, v in f.items():
        setattr(a, k, v)
    return a


@pytest.mark.parametrize("change", [
    dict(dtype=0), dict(dtype=3), dict(weight_dtype=2), dict(ranks=0), dict(ranks=65), dict(ranks=4),
    dict(dy=None), dict(x=None), dict(weight=None), dict(rstd=None), dict(dx=None),
    dict(dweight=None), dict(workspace=None), dict(workspace=WS + 64), dict(workspace_bytes=255),
    dict(dy_stride=49), dict(x_stride=49), dict(dsum_stride=49), dict(dx_stride=49),
    dict(dx=DX + 2), dict(rstd=BR + 1), dict(dweight=DW + 2), dict(cols=(1 << 28) + 1),
    dict(rows=(1 << 63)), dict(dx_stride=1 << 60),
])
def test_backward_refuses_bad_arguments(api, change):
    a = _back(api, **change)
    assert api.lib().ar_rmsnorm_backward(ctypes.byref(a), None) == api.AR_ERR_INVALID_ARG


@pytest.mark.parametrize("change", [
    dict(dx=DY + 4), dict(dx=DY, dx_stride=60), dict(dweight=BW), dict(dx=BW), dict(dweight=DX + 40),
    dict(workspace=BX & ~255), dict(dweight=WS), dict(dx=BR),
])
def test_backward_refuses_overlaps(api, change):
    a = _back(api, **change)
    assert api.lib().ar_rmsnorm_backward(ctypes.byref(a), None) == api.AR_ERR_INVALID_USAGE


def test_backward_workspace_sizes(api):
    f = api.ar_rmsnorm_backward_workspace
    assert f(1, 0, 50) == 0 and f(1, 10, 0) == 0
    assert f(3, 10, 50) == 0 and f(0, 10, 50) == 0 and f(65, 65, 50) == 0   # refused sizes
    for ranks, rows, cols in ((1, 1, 1), (1, 100_000, 8192), (64, 64, 7), (8, 8 * 1000, 1001)):
        n = f(ranks, rows, cols)
        assert n % 256 == 0 and n >= ranks * cols * 4
        assert n <= ranks * min(rows // ranks, 512) * cols * 4 + 255
    assert api.lib().ar_rmsnorm_backward(None, None) == api.AR_ERR_INVALID_ARG


def _spans(api, *triples):
    a = (api.ar_span_t * len(triples))()
    for i, (p, n, dt) in enumerate(triples):
        a[i] = api.ar_span_t(p, n, dt)
    return a


def test_grad_norm_refusals(api):
    L = api.lib()
    F, B = api.AR_FLOAT32, api.AR_BF16
    c = api.ar_init(2, 16, F)
    try:
        ok = _spans(api, (X, 10, F))
        assert L.ar_grad_norm(None, ok, 1, Y, None) == api.AR_ERR_INVALID_ARG
        assert L.ar_grad_norm(c, ok, 1, Y, None) == api.AR_ERR_INVALID_USAGE  # no workspace yet
    finally:
        api.ar_destroy(c)


def test_grad_clip_refusals(api):
    L = api.lib()
    F, B = api.AR_FLOAT32, api.AR_BF16
    one = _spans(api, (X, 10, F))

    def call(a, b, n, norm=Y, most=1.0):
        return L.ar_grad_clip(a, b, n, norm, most, None)
    bad, usage = api.AR_ERR_INVALID_ARG, api.AR_ERR_INVALID_USAGE
    assert call(one, one, 1, norm=None) == bad
    assert call(one, one, 1, norm=Y + 2) == bad
    assert call(one, one, 1, most=-1.0) == bad
    assert call(one, one, 1, most=float("nan")) == bad
    assert call(None, one, 1) == bad and call(one, None, 1) == bad
    assert call(None, None, 0) == api.AR_SUCCESS
    empty = _spans(api, (None, 0, F), (None, 0, B))
    assert call(empty, empty, 2) == api.AR_SUCCESS
    for s in ((X, 10, 0), (X, 10, 3), (None, 10, F), (X + 2, 10, F), (X + 1, 10, B),
              (X, (1 << 36) + 1, B), (X, (1 << 64) - 1, F)):
        s = _spans(api, s)
        assert call(s, s, 1) == bad
    assert call(one, _spans(api, (Y, 11, F)), 1) == bad
    assert call(one, _spans(api, (Y, 10, B)), 1) == bad
    # overlaps: partly its own input, another tensor's input or output, the norm
    assert call(one, _spans(api, (X + 4, 10, F)), 1) == usage
    two = _spans(api, (X, 10, F), (X + 40, 10, F))
    assert call(two, _spans(api, (X + 40, 10, F), (X, 10, F)), 2) == usage
    assert call(two, _spans(api, (SUM, 10, F), (SUM + 36, 10, F)), 2) == usage
    assert call(two, _spans(api, (SUM, 10, F), (X, 10, F)), 2) == usage
    twice = _spans(api, (X, 10, F), (X, 10, F))
    assert call(twice, twice, 2) == usage
    assert call(one, one, 1, norm=X + 8) == usage


def test_struct_fields_match_the_header(api):
    """The ctypes structs list the header's fields, in order."""
    import re
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    src = re.sub(r"/\*.*?\*/", "", open(os.path.join(root, "include", "ar.h")).read(), flags=re.S)
    for cls in (api.ar_rmsnorm_t, api.ar_rmsnorm_backward_t, api.ar_span_t):
        body = re.search(r"typedef struct \{([^{}]*)\} %s;" % cls.__name__, src).group(1)
        names = [n.strip().lstrip("* ") for decl in body.split(";") if decl.strip()
                 for n in re.sub(r"^\s*(const\s+)?\w+\s*", "", decl.strip()).split(",")]
        assert names == [n for n, _ in cls._fields_], cls.__name__


def test_tensor_list_checks(api):
    with pytest.raises(ValueError):
        api.TensorList([torch.zeros(3)])                    # not on a GPU
    with pytest.raises(ValueError):
        api.TensorList([torch.zeros(3, dtype=torch.float16)])
    assert len(api.TensorList([])) == 0
    dense = api.binding().dense
    assert dense(torch.zeros(4, 5).t()) and dense(torch.zeros(2, 3, 4).permute(2, 0, 1))
    assert not dense(torch.zeros(4, 5)[:, :4]) and not dense(torch.zeros(3, 1).expand(3, 4))
    assert dense(torch.zeros(())) and dense(torch.zeros(3, 0)) and dense(torch.zeros(5, 1, 3)[:, :, :])
    with pytest.raises(ValueError):
        api.TensorList([None])


def test_python_norm_checks(api):
    x, w = torch.zeros(3, 8), torch.zeros(8)
    for kw in (dict(x=torch.zeros(24)), dict(x=x.double()), dict(weight=w.double()),
               dict(weight=w.to(torch.bfloat16)), dict(y=x.double()), dict(group=32),
               dict(scale=torch.zeros(3, 1)), dict(y=torch.zeros(3, 8, dtype=torch.float8_e4m3fn)),
               dict(y=torch.zeros(3, 8, dtype=torch.float8_e4m3fn), scale=torch.zeros(3, 1), group=7),
               dict()):  # the last: not on a GPU
        f = {**dict(x=x, weight=w, y=x.clone()), **kw}
        with pytest.raises(ValueError):
            api.rmsnorm(f.pop("x"), f.pop("weight"), f.pop("y"), **f)
    with pytest.raises(ValueError):
        api.rmsnorm_backward(x, x, w, torch.zeros(3), x.clone(), torch.zeros(8))


# ---- the 64-bit forms themselves -------------------------------------------------

def test_backward_form_against_differences():
    """The gradient's formula against central differences of the forward
    form, in 64 bits: the differences' own error is about step^2."""
    g = torch.Generator().manual_seed(3)
    T, C, eps, step = 3, 7, 1e-3, 1e-5
    draw = lambda *s: torch.randn(*s, generator=g, dtype=torch.float64)  # noqa: E731
    x, w, dy, ds = draw(T, C), draw(C), draw(T, C), draw(T, C)

    def loss(x, w):
        f = ob.norm(x, w, eps)
        return (f["y"][0] * dy).sum() + (x * ds).sum()
    f = ob.norm_backward(dy, x, w, ob.norm(x, w, eps)["rstd"][0], dsum=ds)
    for at, grad in ((x, f["dx"][0]), (w, f["dweight"][0][0])):
        flat = at.view(-1)
        for i in range(flat.numel()):
            old = float(flat[i])
            flat[i] = old + step
            up = float(loss(x, w))
            flat[i] = old - step
            down = float(loss(x, w))
            flat[i] = old
            assert abs((up - down) / (2 * step) - float(grad.view(-1)[i])) < 1e-7


def test_bounds_catch_a_planted_mistake():
    """A float32 evaluation passes its bounds; the same with a mistake of a
    few roundings in one element does not."""
    g = torch.Generator().manual_seed(5)
    x = torch.randn(5, 300, generator=g)
    w = torch.randn(300, generator=g)
    f = ob.norm(x, w, 1e-6)
    r = 1 / torch.sqrt((x * x).mean(1) + 1e-6)
    y = x * r[:, None] * w
    ob.between(y, *f["y"], "y")
    y[2, 7] *= 1 + 2.0 ** -18
    with pytest.raises(AssertionError):
        ob.between(y, *f["y"], "y")
    q = ob.norm(x, w, 1e-6, group=128)
    s = q["scale"][0].float()
    e = (q["y"][0]).float().to(torch.float8_e4m3fn)
    ob.between(e, *q["y"], "y")
    ob.between(s, *q["scale"], "scale")
    e.view(torch.uint8)[0, 0] ^= 1
    with pytest.raises(AssertionError):
        ob.between(e, *q["y"], "y")
