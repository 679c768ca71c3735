"""The operators' kernels that the widths of the other tests do not reach: the
backward pass in place over rows past one vector a thread, and several ranks'
rows with a float32 weight beside a bfloat16 stream."""
import pytest

from tests import operator_bounds as ob
from tests.test_operators_gpu import EPS, _check_norm, _rand, _run_back, _types, env  # noqa: F401

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dtype,wtype", [("f32", "f32"), ("bf16", "bf16"), ("bf16", "f32")])
@pytest.mark.parametrize("cols", (4104, 8200, 9001, 16390, 20001))
@pytest.mark.parametrize("ranks,rows", [(2, 66), (2, 520)])
def test_backward_in_place_of_long_rows(env, dtype, wtype, cols, ranks, rows):  # noqa: F811
    """dx over each of its inputs gives the bits it gives apart from them: rows
    held in registers and rows read again, one and several a workgroup."""
    torch = env["torch"]
    want = _run_back(env, ranks, rows, cols, dtype, wtype, True)
    for over in ("dy", "x", "dsum"):
        got = _run_back(env, ranks, rows, cols, dtype, wtype, True, dx_over=over)
        assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1]), over


@pytest.mark.parametrize("dtype,wtype", [("f32", "f32"), ("bf16", "bf16"), ("bf16", "f32")])
@pytest.mark.parametrize("cols,pad,offset", [(4100, 3, 1), (8200, 1, 1), (16385, 5, 3), (20001, 1, 0)])
def test_backward_of_long_rows_at_any_alignment(env, dtype, wtype, cols, pad, offset):  # noqa: F811
    _run_back(env, 1, 300, cols, dtype, wtype, True, pad, offset)
    _run_back(env, 3, 6, cols, dtype, wtype, False, pad, offset, dx_over="x")


@pytest.mark.parametrize("cols", (5, 100, 1000, 8192, 8200, 16392, 20000, 33000))
@pytest.mark.parametrize("out,group", [("same", 0), ("e4m3", 0), ("e4m3", 128)])
@pytest.mark.parametrize("dtype,wtype", [("bf16", "f32"), ("bf16", "bf16"), ("f32", "f32")])
def test_reduce_scatter_norm_over_the_residual(env, cols, out, group, dtype, wtype):  # noqa: F811
    """1, 2 and 4 vectors a thread and an element at a time, the new stream
    over the residual's array, 2 and 5 ranks."""
    torch, api, dev = env["torch"], env["api"], env["dev"]
    T = _types(torch)
    dt = T[dtype]
    for R, tokens, redop in ((2, 3, "sum"), (5, 1, "avg")):
        hs = _rand(env, (R, R * tokens * cols), 1, dt)
        hr = _rand(env, (R, tokens * cols), 2, dt)
        hw = (1 + 0.2 * _rand(env, (cols,), 3, torch.float32)).to(T[wtype])
        comm = api.Comm(R, R * tokens * cols, "bf16" if dtype == "bf16" else "float32", device=dev,
                        redop=redop)
        stream = hr.to(dev)
        got = {"y": torch.empty((R, tokens * cols), dtype=T[dtype if out == "same" else out], device=dev),
               "rstd": torch.empty((R, tokens), device=dev), "sum": stream}
        if out == "e4m3":
            got["scale"] = torch.empty((R, tokens * (-(-cols // group) if group else 1)), device=dev)
        comm.reduce_scatter_rmsnorm(hs.to(dev), hw.to(dev), got["y"], EPS, residual=stream, sum=stream,
                                    scale=got.get("scale"), group=group, rstd=got["rstd"])
        torch.cuda.synchronize()
        form = ob.norm(None, hw, EPS, residual=hr.view(-1, cols), parts=hs.view(R, R * tokens, cols),
                       divisor=R if redop == "avg" else 1.0, group=group if out == "e4m3" else None)
        _check_norm(env, got, form)
        assert comm.check() == api.AR_SUCCESS
        comm.close()


def test_low_level_calls(env):  # noqa: F811
    """The functions with the C names, of plain integers: the bits of the torch
    wrappers."""
    torch, api, dev = env["torch"], env["api"], env["dev"]
    R, tokens, cols = 2, 3, 200
    n = R * tokens
    send, x, dy = (_rand(env, s, k, torch.float32).to(dev) for k, s in
                   enumerate(((R, n * cols), (n, cols), (n, cols))))
    w = _rand(env, (cols,), 5, torch.float32).to(dev)
    comm = api.Comm(R, n * cols, "float32", device=dev)
    want, got = ([torch.zeros((n, cols), device=dev), torch.zeros((R, tokens * cols), device=dev),
                  torch.zeros((n, cols), device=dev), torch.zeros((R, cols), device=dev),
                  torch.zeros(n, device=dev)] for _ in range(2))
    ws = api.rmsnorm_backward_workspace(R, n, cols, dev)
    api.rmsnorm(x, w, want[0], EPS, rstd=want[4])
    comm.reduce_scatter_rmsnorm(send, w, want[1], EPS)
    api.rmsnorm_backward(dy, x, w, want[4], want[2], want[3], workspace=ws)
    torch.cuda.synchronize()
    s = torch.cuda.current_stream().cuda_stream
    a = api.ar_rmsnorm_t(dtype=api.AR_FLOAT32, out_dtype=api.AR_FLOAT32, weight_dtype=api.AR_FLOAT32,
                         eps=EPS, rows=n, cols=cols, x=x.data_ptr(), x_stride=cols, weight=w.data_ptr(),
                         y=got[0].data_ptr(), y_stride=cols, rstd=got[4].data_ptr())
    api.ar_rmsnorm(a, s)
    a.rows, a.y, a.rstd = tokens, got[1].data_ptr(), None
    api.ar_reduce_scatter_rmsnorm(comm.handle, send.data_ptr(), a, s)
    b = api.ar_rmsnorm_backward_t(dtype=api.AR_FLOAT32, weight_dtype=api.AR_FLOAT32, ranks=R, rows=n,
                                  cols=cols, dy=dy.data_ptr(), dy_stride=cols, x=x.data_ptr(),
                                  x_stride=cols, weight=w.data_ptr(), rstd=got[4].data_ptr(),
                                  dx=got[2].data_ptr(), dx_stride=cols, dweight=got[3].data_ptr(),
                                  workspace=ws.data_ptr(), workspace_bytes=ws.numel())
    api.ar_rmsnorm_backward(b, s)
    torch.cuda.synchronize()
    for g, t in zip(got, want):
        assert torch.equal(g, t)
    with pytest.raises(api.ArError):
        a.eps = -1.0
        api.ar_rmsnorm(a, s)
    comm.close()
