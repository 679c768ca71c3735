"""Host side of the orthogonalisation: what it refuses, its workspace, and the
64-bit form the GPU tests compare with."""
import ctypes
import os

import pytest
import torch

from tests import ortho_forms as of

COEFFICIENTS = (3.4445, -4.7750, 2.0315)
X, OUT, WS = 0x10000000, 0x20000000, 0x40000000


@pytest.fixture(scope="module")
def api():
    from collective_communication_ring_amd import api
    if not os.path.exists(api.LIB_PATH) or not os.path.exists(os.path.join(api.HERE, "_binding.so")):
        import __graft_entry__
        __graft_entry__.build()
    api.lib()
    return api


def _call(api, x=(X, X + 40000), out=(OUT, OUT + 40000), k=COEFFICIENTS, **change):
    f = dict(dtype=api.AR_FLOAT32, steps=1, eps=1e-7, scale=1.0, count=2, rows=50, cols=60, x_stride=60,
             out_stride=60, workspace=WS, workspace_bytes=1 << 26)
    f.update(change)
    n = max(1, f["count"] if f["count"] < 100 else 1)
    xs = (ctypes.c_void_p * n)(*(list(x) + [X] * n)[:n]) if x is not None else None
    outs = (ctypes.c_void_p * n)(*(list(out) + [OUT] * n)[:n]) if out is not None else None
    steps = max(1, min(f["steps"], 100))
    ks = (ctypes.c_float * (3 * steps))(*(list(k) * steps)) if k is not None else None
    a = api.ar_orthogonalize_t(x=xs, out=outs, coefficients=ks, **f)
    return api.lib().ar_orthogonalize(ctypes.byref(a), None)


def test_refuses_bad_arguments(api):
    nan, inf = float("nan"), float("inf")
    one = api.ar_orthogonalize_workspace(1, 50, 60)
    for change in (dict(dtype=0), dict(dtype=3), dict(steps=0), dict(steps=65), dict(eps=-1.0), dict(eps=nan),
                   dict(eps=inf), dict(scale=nan), dict(scale=inf), dict(rows=65537), dict(cols=65537),
                   dict(count=1 << 25), dict(k=None), dict(k=(nan, 1.0, 1.0)), dict(k=(1.0, inf, 1.0)),
                   dict(x=None), dict(out=None), dict(x=(X, 0)), dict(out=(0, OUT)), dict(x=(X + 2, X + 40000)),
                   dict(out=(OUT, OUT + 1)), dict(x_stride=59), dict(out_stride=59), dict(x_stride=1 << 45),
                   dict(workspace=None), dict(workspace=WS + 64), dict(workspace_bytes=one - 1)):
        assert _call(api, **change) == api.AR_ERR_INVALID_ARG, change
    assert api.lib().ar_orthogonalize(None, None) == api.AR_ERR_INVALID_ARG


def test_refuses_overlaps(api):
    size = 4 * 50 * 60
    for change in (dict(out=(X + 4, OUT)), dict(out=(OUT, OUT + size - 4)), dict(out=(OUT, OUT)),
                   dict(out=(X + 40000, OUT)), dict(out=(X, X + 40000), out_stride=61),
                   dict(x=(WS + 100, X)), dict(out=(OUT, WS - size + 4)),
                   # rows in turn: 60 columns of 100 leave room for 40
                   dict(x_stride=100, out_stride=100, out=(X + 4 * 50, OUT))):
        assert _call(api, **change) == api.AR_ERR_INVALID_USAGE, change


def test_refuses_steps_that_grow(api):
    for k in ((20.0, 20.0, 20.0), (3.4445, -4.7750, 200.0), (-30.0, 0.0, 0.0)):
        assert _call(api, k=k, steps=8) == api.AR_ERR_UNSUPPORTED
    assert _call(api, k=(70000.0, 0.0, 0.0)) == api.AR_ERR_UNSUPPORTED


def test_accepts(api):
    """What passes the checks ends in an error of the device: there is none."""
    if torch.cuda.is_available():
        pytest.skip("the addresses are not real")
    for change in (dict(), dict(out=(X, X + 40000)), dict(k=COEFFICIENTS, steps=64),
                   dict(x_stride=120, out_stride=120, out=(X + 240, OUT), x=(X, OUT + 240)),
                   dict(rows=1, x_stride=0), dict(k=(0.0, 0.0, 0.0), steps=3), dict(x=(X, X)),
                   dict(workspace_bytes=api.ar_orthogonalize_workspace(1, 50, 60))):
        assert _call(api, **change) == api.AR_ERR_HIP, change


def test_of_nothing(api):
    for empty in (dict(count=0), dict(rows=0), dict(cols=0), dict(count=0, x=None, out=None, workspace=None)):
        assert _call(api, **empty) == api.AR_SUCCESS, empty


def test_workspace(api):
    f = api.ar_orthogonalize_workspace
    assert f(0, 5, 5) == f(1, 0, 5) == f(1, 5, 0) == f(1, 65537, 5) == 0
    assert f(1, 100, 300) == f(1, 300, 100)
    one = f(2, 100, 300) - f(1, 100, 300)
    assert f(3, 100, 300) == f(1, 100, 300) + 2 * one and f(1, 1, 1) % 256 == 0
    assert f(500, 100, 300) == f(128, 100, 300)  # more go by parts


def test_wrapper_refuses(api):
    x = torch.zeros(3, 4, 5)
    with pytest.raises(ValueError):
        api.orthogonalize(x, x, steps=2, coefficients=[(1.0, 0.0, 0.0)] * 3, workspace=x)
    with pytest.raises(ValueError):
        api.orthogonalize(x, x, workspace=x)  # not on the GPU
    assert api.orthogonalize([], []) == []


# ---- the form ---------------------------------------------------------------------

def _matrix(m, n, seed):
    return torch.randn(m, n, generator=torch.Generator().manual_seed(seed), dtype=torch.float64)


@pytest.mark.parametrize("m,n", [(5, 9), (9, 5), (7, 7)])
def test_form_works_on_singular_values(m, n):
    """U p(p(..s..)) V^T of the matrix's U s V^T."""
    x = _matrix(m, n, 1)
    got = of.orthogonalize(x, 3, COEFFICIENTS, 1e-7, 2.0)
    u, s, v = torch.linalg.svd(x, full_matrices=False)
    s = s / (torch.sqrt((x * x).sum()) + 1e-7)
    for _ in range(3):
        a, b, c = COEFFICIENTS
        s = a * s + b * s ** 3 + c * s ** 5
    assert torch.allclose(got, 2.0 * (u * s) @ v, atol=1e-12)


def test_bounds_hold_for_a_plain_computation():
    """float32 products lie well within the bounds of the halves' products, and
    operands of one half, 11 bits, do not."""
    x = _matrix(24, 40, 2)
    value, slack = of.one_step(x, COEFFICIENTS, 1e-7)
    a, b, c = COEFFICIENTS

    def step(cut):
        y = (x / x.norm()).float()
        A = cut(y) @ cut(y).t()
        B = b * A + c * (cut(A) @ cut(A))
        return (a * y + cut(B) @ cut(y)).double()
    assert bool(((step(lambda t: t) - value).abs() <= slack).all())
    assert bool(((step(lambda t: (t * 4096).half().float() / 4096) - value).abs() > slack).any())
    y = (x / x.norm()).float()
    for k in range(5):
        value, slack = of.next_step(y, k, COEFFICIENTS)
        A = y @ y.t()
        y = a * y + (b * A + c * A @ A) @ y
        assert bool(((y.double() - value).abs() <= slack).all())
    assert float(slack.norm()) < 0.003 * float(value.norm())


def test_groups_of_steps_form():
    """A float32 computation by groups is the same polynomial, and within the
    bound, which a step left out is not."""
    x = _matrix(20, 60, 5)
    ks = [COEFFICIENTS] * 5
    assert of.groups_of(1000, 2000, ks, 16.0) == [2, 2, 1] and of.groups_of(2000, 1000, ks, 256.0) == [3, 2]
    assert of.groups_of(20, 60, ks, 256.0) == of.groups_of(2000, 2500, ks, 256.0) == [1] * 5
    for group, tight in ((1, 2.0 ** -12), (2, 2.0 ** -10), (3, 2.0 ** -5)):
        before = x / (x.norm() + 1e-7)
        value, y = of.steps_of(before, ks[:group]), before.float()
        A, F = y @ y.t(), None
        for a, b, c in ks[:group]:
            Q = a * torch.eye(20) + b * A + c * A @ A
            F = Q if F is None else Q @ F
            A = Q @ (Q @ A)
        bound = of.group_error(before, ks[:group])
        assert float(((F @ y).double() - value).norm()) <= bound < tight * float(value.norm())
    assert torch.allclose(of.steps_of(x.t() / (x.norm() + 1e-7), ks).t(), of.orthogonalize(x, 5, ks, 1e-7))
