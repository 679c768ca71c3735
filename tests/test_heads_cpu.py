"""Host side of the operators on attention heads: what they refuse, the
frequencies, and the 64-bit forms the GPU tests compare with."""
import ctypes
import math
import os

import pytest
import torch

from tests import head_forms as hf


@pytest.fixture(scope="module")
def api():
    from collective_communication_ring_amd import api
    if not os.path.exists(api.LIB_PATH) or not os.path.exists(os.path.join(api.HERE, "_binding.so")):
        import __graft_entry__
        __graft_entry__.build()
    api.lib()
    return api


# device addresses that no refused call touches: 2 batches of 3 tokens, 4 and 2 heads of 8
Q, K, QO, KO, QW, KW, FREQ, POS, DQO, DKO, DQ, DK, QDW, KDW, WS = (0x10000000 * k for k in range(1, 16))
B, S, HQ, HK, DIM = 2, 3, 4, 2, 8


def _heads(api, at, heads):
    return api.ar_heads_t(at, S * heads * DIM, heads * DIM, DIM)


def _rotation(api, **change):
    f = dict(rot_dim=8, layout=0, factor=1.0, frequencies=FREQ, positions=POS, position_bytes=8,
             position_stride=S)
    f.update(change)
    return api.ar_rotation_t(**f)


def _call(api, kind, rotation=None, **change):
    f = dict(dtype=api.AR_BF16, batch=B, tokens=S, q_heads=HQ, k_heads=HK, dim=DIM,
             rotation=_rotation(api, **(rotation or {})), q=_heads(api, Q, HQ), k=_heads(api, K, HK))
    if kind != "back":
        f.update(q_out=_heads(api, QO, HQ), k_out=_heads(api, KO, HK))
    if kind != "rotary":
        f.update(weight_dtype=api.AR_BF16, eps=1e-6, q_weight=QW, k_weight=KW)
    if kind == "back":
        f.update(ranks=2, dq_out=_heads(api, DQO, HQ), dk_out=_heads(api, DKO, HK),
                 dq=_heads(api, DQ, HQ), dk=_heads(api, DK, HK), q_dweight=QDW, k_dweight=KDW,
                 workspace=WS, workspace_bytes=1 << 26)
    f.update(change)
    L = api.lib()
    if kind == "rotary":
        return L.ar_rotary(ctypes.byref(api.ar_rotary_t(**f)), None)
    if kind == "norm":
        return L.ar_head_rmsnorm(ctypes.byref(api.ar_head_rmsnorm_t(**f)), None)
    return L.ar_head_rmsnorm_backward(ctypes.byref(api.ar_head_rmsnorm_backward_t(**f)), None)


KINDS = ("rotary", "norm", "back")


@pytest.mark.parametrize("kind", KINDS)
def test_refuses_bad_arguments(api, kind):
    h = lambda *a: api.ar_heads_t(*a)  # noqa: E731
    full = (S * HQ * DIM, HQ * DIM, DIM)
    out = "dq" if kind == "back" else "q_out"
    bad = [dict(dtype=0), dict(dtype=3), dict(dim=0), dict(dim=1025), dict(q=h(0, *full)),
           dict(q=h(Q + 1, *full)), dict(batch=1 << 31), dict(tokens=1 << 31), dict(q_heads=1 << 31),
           dict(batch=1 << 16, tokens=1 << 16, q_heads=1), dict(q=h(Q, (1 << 46) + 1, HQ * DIM, DIM)),
           dict(k=h(0, *full)), {out: h(0, *full)}, {out: h(QO + 1, *full)},
           # an output's element twice: heads, tokens, batches in each other's way
           {out: h(QO, S * HQ * DIM, HQ * DIM, DIM - 1)}, {out: h(QO, S * HQ * DIM, 0, DIM)},
           {out: h(QO, HQ * DIM, HQ * DIM, DIM)}, {out: h(QO, S * HQ * DIM, HQ * DIM - 1, DIM)},
           dict(rotation=dict(rot_dim=7)), dict(rotation=dict(rot_dim=10)), dict(rotation=dict(layout=2)),
           dict(rotation=dict(layout=-1)), dict(rotation=dict(factor=float("nan"))),
           dict(rotation=dict(factor=float("inf"))), dict(rotation=dict(frequencies=None)),
           dict(rotation=dict(positions=None)), dict(rotation=dict(position_bytes=2)),
           dict(rotation=dict(frequencies=FREQ + 4)), dict(rotation=dict(positions=POS + 4)),
           dict(rotation=dict(position_stride=1 << 47))]
    if kind == "rotary":
        bad += [dict(rotation=dict(rot_dim=0))]
    else:
        bad += [dict(weight_dtype=0), dict(weight_dtype=3), dict(eps=-1.0), dict(eps=float("nan")),
                dict(eps=float("inf")), dict(q_weight=None), dict(k_weight=None),
                dict(q_weight=QW + 1), dict(weight_dtype=1, k_weight=KW + 2)]
    if kind == "back":
        bad += [dict(ranks=0), dict(ranks=65), dict(ranks=3), dict(workspace=None),
                dict(workspace=WS + 128), dict(q_dweight=None), dict(k_dweight=KDW + 2),
                dict(workspace_bytes=api.ar_head_rmsnorm_backward_workspace(2, DIM) - 1)]
    for change in bad:
        assert _call(api, kind, **change) == api.AR_ERR_INVALID_ARG, change


@pytest.mark.parametrize("kind", KINDS)
def test_refuses_overlaps(api, kind):
    h = lambda at, heads=HQ: _heads(api, at, heads)  # noqa: E731
    q_out, k_out = ("dq", "dk") if kind == "back" else ("q_out", "k_out")
    bad = [{q_out: h(Q + 2)}, {q_out: h(K)}, {k_out: h(Q, HK)},
           {k_out: h(QO if kind != "back" else DQ, HK)}, {q_out: h(POS)}, {q_out: h(FREQ)},
           {k_out: h(POS + 8 * 5, HK)},
           # q's address, but tokens ahead of heads in memory
           {q_out: api.ar_heads_t(Q, S * HQ * DIM, DIM, S * DIM)}]
    if kind != "rotary":
        bad += [{q_out: h(QW)}, {k_out: h(KW, HK)}]
    if kind == "back":
        bad += [dict(dq=h(WS)), dict(q_dweight=Q), dict(q_dweight=WS), dict(k_dweight=QDW), dict(dq=h(DKO)),
                dict(workspace=DQO), dict(dk=h(DQO, HK))]
    for change in bad:
        assert _call(api, kind, **change) == api.AR_ERR_INVALID_USAGE, change


def test_parts_of_one_product_do_not_overlap(api):
    """Queries, keys and values side by side in each token's row, or token by
    head, rotated in place: refused only where they do meet.  (A call that
    passes the checks ends in an error of the device: there is none here.)"""
    if torch.cuda.is_available():
        pytest.skip("the addresses are not real")
    wide = (HQ + 2 * HK) * DIM
    part = lambda at: api.ar_heads_t(Q + 2 * at, S * wide, wide, DIM)  # noqa: E731
    place = dict(q=part(0), k=part(HQ * DIM))
    ok = dict(q_out=part(0), k_out=part(HQ * DIM))
    assert _call(api, "rotary", **place, **ok) == api.AR_ERR_HIP
    assert _call(api, "rotary", **place, **{**ok, "k_out": part(HQ * DIM + HK * DIM)}) == api.AR_ERR_HIP
    assert _call(api, "rotary", **place, **{**ok, "k_out": part(HQ * DIM - 1)}) == api.AR_ERR_INVALID_USAGE
    assert _call(api, "rotary", **place, **{**ok, "k_out": part(wide - HK * DIM + 1)}) == \
        api.AR_ERR_INVALID_USAGE  # the last head reaches the next token's queries
    # [tokens, heads, 3, dim]
    turn = lambda i: api.ar_heads_t(Q + 2 * i * DIM, S * HQ * 3 * DIM, HQ * 3 * DIM, 3 * DIM)  # noqa: E731
    same = dict(k_heads=HQ, q=turn(0), k=turn(1))
    assert _call(api, "rotary", **same, q_out=turn(0), k_out=turn(1)) == api.AR_ERR_HIP
    assert _call(api, "rotary", **same, q_out=turn(2), k_out=turn(1)) == api.AR_ERR_HIP
    assert _call(api, "rotary", **same, q_out=turn(1), k_out=turn(0)) == api.AR_ERR_INVALID_USAGE
    # heads ahead of tokens, and a shared (broadcast) input
    first = lambda at, n: api.ar_heads_t(at, S * n * DIM, DIM, S * DIM)  # noqa: E731
    assert _call(api, "rotary", q=first(Q, HQ), q_out=first(Q, HQ)) == api.AR_ERR_HIP
    assert _call(api, "rotary", q=api.ar_heads_t(Q, 0, 0, DIM)) == api.AR_ERR_HIP
    assert _call(api, "rotary", q=api.ar_heads_t(Q, 0, 0, 0), q_out=_heads(api, Q, HQ)) == \
        api.AR_ERR_INVALID_USAGE


@pytest.mark.parametrize("kind", KINDS)
def test_of_nothing(api, kind):
    for empty in (dict(batch=0), dict(tokens=0), dict(q_heads=0, k_heads=0)):
        if kind == "back" and "q_heads" not in empty:
            continue  # writes zeros
        assert _call(api, kind, **empty) == api.AR_SUCCESS
    L = api.lib()
    for f in (L.ar_rotary, L.ar_head_rmsnorm, L.ar_head_rmsnorm_backward):
        assert f(None, None) == api.AR_ERR_INVALID_ARG


def test_backward_workspace(api):
    f = api.ar_head_rmsnorm_backward_workspace
    assert f(0, 64) == f(65, 64) == f(1, 0) == f(1, 1025) == 0
    for ranks in (1, 3, 64):
        assert f(ranks, 128) % 256 == 0 and f(ranks, 128) >= ranks * 2 * 128 * 4


# ---- frequencies -----------------------------------------------------------------

def _scheme(api, **change):
    f = dict(rot_dim=64, scaling=0, base=10000.0, scale=8.0, original=4096.0, low=1.0, high=4.0,
             fast=32.0, slow=1.0)
    f.update(change)
    return api.ar_rotary_scheme_t(**f)


@pytest.mark.parametrize("scaling", (None, "linear", "base", "bands", "ramp"))
@pytest.mark.parametrize("rot,base", [(4, 10000.0), (64, 10000.0), (96, 500000.0), (128, 1e6)])
def test_frequencies(api, scaling, rot, base):
    got, factor = api.ar_rotary_frequencies(_scheme(api, rot_dim=rot, base=base,
                                                    scaling=api.SCALINGS[scaling]))
    assert len(got) == rot // 2 and got[0] <= 1.0
    for i, f in enumerate(got):
        want = base ** (-2 * i / rot)
        if scaling == "linear":
            want /= 8
        elif scaling == "base":
            want = (base * 8 ** (rot / (rot - 2))) ** (-2 * i / rot)
        elif scaling == "bands":
            turns = 4096 * want / (2 * math.pi)
            share = (turns - 1) / 3
            want = want if turns >= 4 else want / 8 if turns <= 1 else \
                share * want + (1 - share) * want / 8
        elif scaling == "ramp":
            lo = max(0, math.floor(rot * math.log(4096 / (32 * 2 * math.pi)) / (2 * math.log(base))))
            hi = min(rot - 1, math.ceil(rot * math.log(4096 / (2 * math.pi)) / (2 * math.log(base))))
            share = 1 - min(1, max(0, (i - lo) / max(hi - lo, 0.001)))
            want = share * want + (1 - share) * want / 8
        assert abs(f - want) <= 1e-14 * want
    assert factor == (0.1 * math.log(8.0) + 1.0 if scaling == "ramp" else 1.0)
    if scaling == "base":  # the fastest pair stays, the slowest is divided by the scale
        assert got[0] == 1.0 and abs(got[-1] * 8 / base ** (-(rot - 2) / rot) - 1) < 1e-12


def test_frequencies_refuse(api):
    nan, inf = float("nan"), float("inf")
    for change in (dict(rot_dim=0), dict(rot_dim=3), dict(rot_dim=1026), dict(scaling=5),
                   dict(scaling=-1), dict(base=1.0), dict(base=nan), dict(base=inf),
                   dict(scaling=1, scale=0.5), dict(scaling=1, scale=nan), dict(scaling=2, rot_dim=2),
                   dict(scaling=3, original=0.0), dict(scaling=3, low=0.0), dict(scaling=3, high=1.0),
                   dict(scaling=4, original=inf), dict(scaling=4, slow=0.0), dict(scaling=4, fast=1.0)):
        with pytest.raises(api.ArError) as e:
            api.ar_rotary_frequencies(_scheme(api, **change))
        assert e.value.status == api.AR_ERR_INVALID_ARG, change
    # what a scaling does not use is not looked at
    api.ar_rotary_frequencies(_scheme(api, scale=nan, original=nan, low=nan, fast=nan))
    for bad in (dict(scaling="sideways"), dict(layout="thirds")):
        with pytest.raises(ValueError):
            api.Rotation(64, device="cpu", **bad)


# ---- the wrappers' refusals --------------------------------------------------------

def test_wrappers_refuse(api):
    x = torch.zeros(2, 3, 4, 8)
    r = api.Rotation(8, device="cpu")
    p = torch.arange(3)
    for call in (lambda: api.rotary(x, p, r, x), lambda: api.rotary(x.int(), p, r, x),
                 lambda: api.rotary(None, p, r, x), lambda: api.head_rmsnorm(x, torch.ones(8), x),
                 lambda: api.head_rmsnorm_backward(x, x, torch.ones(8), x, torch.ones(1, 8),
                                                   workspace=x),
                 lambda: api.orthogonalize(torch.zeros(3, 3), torch.zeros(3, 3), workspace=x)):
        with pytest.raises((ValueError, AttributeError)):
            call()


# ---- the forms -----------------------------------------------------------------------

@pytest.mark.parametrize("layout", ("halves", "pairs"))
@pytest.mark.parametrize("rot", (0, 6, 10))
def test_backward_form(layout, rot):
    """Against automatic differentiation, and against differences."""
    g = torch.Generator().manual_seed(rot)
    rand = lambda *s: torch.randn(s, generator=g, dtype=torch.float64)  # noqa: E731
    x, dy, w = rand(2, 3, 2, 10), rand(2, 3, 2, 10), rand(10)
    t = hf.table(torch.randint(-50, 50, (2, 3), generator=g), rand(rot // 2), 1.3) if rot else None
    f = lambda x, w: hf.head_norm(x, w, 1e-3, t, layout)[0]  # noqa: E731
    (dx, _), (dw, _) = hf.head_norm_backward(dy, x, w, 1e-3, t, layout, ranks=2)
    xa, wa = x.clone().requires_grad_(), w.clone().requires_grad_()
    f(xa, wa).backward(dy)
    assert torch.allclose(dx, xa.grad, rtol=1e-12, atol=1e-12)
    assert torch.allclose(dw.sum(0), wa.grad, rtol=1e-12, atol=1e-12)
    h = 1e-6
    for at in ((0, 0, 0, 0), (1, 2, 1, 9), (0, 1, 1, 5)):
        step = torch.zeros_like(x)
        step[at] = h
        slope = ((f(x + step, w) - f(x - step, w)) * dy).sum() / (2 * h)
        assert abs(slope - dx[at]) < 1e-7
    one = (f(x[:1], w + h * torch.eye(10, dtype=torch.float64)[3]) - f(x[:1], w)) if t is None else None
    if one is not None:
        assert abs((one * dy[:1]).sum() / h - dw[0, 3]) < 1e-7


def test_rotation_form():
    """A rotation keeps a pair's length and adds its angle."""
    t = hf.table(torch.tensor([[0, 5]]), torch.tensor([0.1, 0.02]), 1.0)
    x = torch.zeros(1, 2, 1, 5, dtype=torch.float64)
    x[..., 0] = 1.0
    x[..., 4] = 7.0
    y, _ = hf.rotary(x, t, "halves")
    assert torch.allclose(y[0, 1, 0], torch.tensor([math.cos(.5), 0, math.sin(.5), 0, 7.0],
                                                   dtype=torch.float64))
    y, _ = hf.rotary(x, t, "pairs")
    assert torch.allclose(y[0, 1, 0], torch.tensor([math.cos(.5), math.sin(.5), 0, 0, 7.0],
                                                   dtype=torch.float64))
    assert torch.equal(y[0, 0], x[0, 0])
    back, _ = hf.rotary(y, t, "pairs", inverse=True)
    assert torch.allclose(back, x)
