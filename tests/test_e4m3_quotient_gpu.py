"""The e4m3 output is the float32 quotient v / scale, rounded to nearest even:
equal to the bits of the same division on the host, at values where a product
with a rounded reciprocal of the scale would land on the other side of a
border of e4m3."""
import pytest
import torch

pytestmark = pytest.mark.gpu

E4M3 = torch.float8_e4m3fn


def _bits(q):
    return q.to(E4M3).view(torch.uint8)


def _group_of_borders(n, g):
    """n float32 weights whose largest is known, the others next to the values
    half way between two of e4m3, times the scale; and the scale.  Of the
    candidates (three for each border and each largest value tried) those come
    first that the division and the reciprocal's product round apart."""
    grid = torch.arange(0, 0x7f, dtype=torch.uint8).view(E4M3).float()  # 0 .. 448
    middle = (grid[1:] + grid[:-1]) / 2
    best = None
    for _ in range(64):
        top = 1 + torch.rand(1, generator=g)
        scale = top / 448
        near = middle * scale
        w = torch.cat([near, torch.nextafter(near, torch.zeros(1)), torch.nextafter(near, top * 2)])
        w = w[w < top]
        apart = _bits(w / scale) != _bits(w * (1 / scale))
        if best is None or int(apart.sum()) > best[2]:
            order = torch.argsort((~apart).to(torch.uint8), stable=True)
            w = w[order][torch.arange(n - 1) % len(w)]
            best = torch.cat([w, top]), scale, int(apart.sum())
    w, scale, apart = best
    assert n == 1 or apart, "no candidate tells the two forms apart"
    return w[torch.randperm(n, generator=g)], scale


@pytest.mark.parametrize("cols,group,power", [
    (3, 0, 0), (70, 32, 0), (1000, 0, 0), (8192, 128, 0), (9000, 64, 0), (16384, 256, 0),
    (40000, 0, 0), (40000, 32, 0), (1000, 32, -110), (1000, 32, -71), (1000, 32, 88), (1000, 0, 110),
])
@pytest.mark.parametrize("dtype", ("f32", "bf16"))
@pytest.mark.parametrize("ranks", (1, 2))
def test_quotients_at_borders(cols, group, power, dtype, ranks):
    """Rows of +-1 without eps: sums of squares and rstd are exact, and v = +-w,
    with weights of about 2^power."""
    from collective_communication_ring_amd import api
    dev = torch.device("cuda:0")
    dt = {"f32": torch.float32, "bf16": torch.bfloat16}[dtype]
    g = torch.Generator().manual_seed(cols + group)
    step = group or cols
    parts = [_group_of_borders(min(step, cols - lo), g) for lo in range(0, cols, step)]
    w = torch.cat([p[0] for p in parts]) * 2.0 ** power
    scales = torch.cat([p[1] for p in parts]) * 2.0 ** power
    rows = 4
    sign = torch.where(torch.rand((rows, cols), generator=g) < 0.5, -1.0, 1.0)
    wide = scales.repeat_interleave(step)[:cols]
    want = _bits(sign * w / wide)
    assert (_bits(sign * w / wide) != _bits(sign * w * (1 / wide))).any()
    y = torch.empty((rows, cols), dtype=E4M3, device=dev)
    scale = torch.empty((rows, len(parts)), device=dev)
    if ranks == 1:
        api.rmsnorm(sign.to(dt).to(dev), w.to(dev), y, 0.0, scale=scale, group=group)
    else:  # two ranks' halves of every row
        comm = api.Comm(2, rows * cols, "bf16" if dtype == "bf16" else "float32", device=dev)
        send = (sign / 2).to(dt).to(dev).view(1, -1).repeat(2, 1)
        comm.reduce_scatter_rmsnorm(send, w.to(dev), y.view(2, -1), 0.0, scale=scale.view(2, -1),
                                    group=group)
    torch.cuda.synchronize()
    assert torch.equal(scale.cpu(), scales.expand(rows, -1))
    assert torch.equal(y.view(torch.uint8).cpu(), want)
    if ranks == 2:
        comm.close()
