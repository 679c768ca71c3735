"""examples/attention_step.py: its gradients against automatic differentiation
of the same network in 64 bits on the host and against differences, its update
against the update's formula, and its single-token steps against the whole
sequence: the head operators and the orthogonalisation together, among the
collectives and norms."""
import importlib.util
import os

import pytest

pytestmark = pytest.mark.gpu

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.fixture(scope="module")
def example():
    spec = importlib.util.spec_from_file_location(
        "attention_step", os.path.join(ROOT, "examples", "attention_step.py"))
    m = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(m)
    return m


SHAPES = [(2, 3, 64, 2, 1, 16), (4, 9, 96, 3, 3, 24), (2, 32, 128, 4, 2, 32)]


def _network(example, block, stream, params):
    """out [tokens, H] in 64 bits on the host."""
    import torch
    Wqkv, Wo, w1, w2, wq, wk = params
    H, D, h, kv = block.H, block.D, block.heads, block.kv_heads

    def norm(x, w):
        return x * torch.rsqrt((x * x).mean(-1, keepdim=True) + example.EPS) * w
    s = stream.view(-1, H)
    n = norm(s, w1)
    T = s.shape[0]
    angle = torch.arange(T, dtype=torch.float64)[:, None] * \
        10000.0 ** (-torch.arange(0, D, 2, dtype=torch.float64) / D)
    c, sn = angle.cos()[:, None], angle.sin()[:, None]

    def turn(x):  # [T, heads, D]
        if block.rotation.layout == 0:
            a, b = x[..., :D // 2], x[..., D // 2:]
            return torch.cat([a * c - b * sn, b * c + a * sn], -1)
        a, b = x[..., ::2], x[..., 1::2]
        return torch.stack([a * c - b * sn, b * c + a * sn], -1).flatten(-2)
    mask = torch.ones(T, T, dtype=torch.bool).triu(1)
    s2 = s
    for r in range(block.R):
        qkv = (n @ Wqkv[r]).view(T, h + 2 * kv, D)
        q, k, v = qkv[:, :h], qkv[:, h:h + kv], qkv[:, h + kv:]
        if block.head_norms:
            q, k = norm(q, wq), norm(k, wk)
        q, k = turn(q), turn(k)
        o = []
        for i in range(h):
            j = i // (h // kv)
            p = torch.softmax((q[:, i] @ k[:, j].t() * D ** -0.5).masked_fill(mask, -torch.inf), 1)
            o.append(p @ v[:, j])
        s2 = s2 + torch.cat(o, 1) @ Wo[r]
    return norm(s2, w2)


def _params(block):
    import torch
    return [p.detach().cpu().to(torch.float64).requires_grad_() for p in
            (block.Wqkv, block.Wo, block.w1, block.w2, block.wq, block.wk)]


@pytest.mark.parametrize("layout,head_norms", [("halves", True), ("pairs", True), ("halves", False),
                                               ("pairs", False)])
@pytest.mark.parametrize("R,tokens,hidden,heads,kv_heads,dim", SHAPES)
def test_gradients(example, R, tokens, hidden, heads, kv_heads, dim, layout, head_norms):
    """Float32 sums of at most 256 terms through six products, four norms and a
    softmax: off by at most about 11 * 256 * 2^-24 of the terms' sizes, 1.7e-4;
    the norms of whole tensors are compared to 5e-4."""
    import torch
    block = example.Attention(R, tokens, hidden, heads, kv_heads, dim, layout, head_norms, seed=3)
    g = torch.Generator().manual_seed(4)
    stream, d_out = (torch.randn((R, tokens * hidden), generator=g) for _ in range(2))
    out = block.forward(stream.cuda()).clone()
    d_stream = block.backward(stream.cuda(), d_out.cuda())
    torch.cuda.synchronize()
    params = _params(block)
    s = stream.double().requires_grad_()
    want = _network(example, block, s, params)
    want.backward(d_out.double().view(-1, hidden))

    def near(got, ref, what):
        got, ref = got.detach().cpu().double().reshape(ref.shape), ref.detach()
        assert float((got - ref).norm()) < 5e-4 * float(ref.norm()), what
    near(out, want, "out")
    near(d_stream, s.grad, "d_stream")
    near(block.d_matrices[0], params[0].grad, "Wqkv")
    near(block.d_matrices[1], params[1].grad, "Wo")
    names = ("w1", "w2", "wq", "wk")[:4 if head_norms else 2]
    for rows, p, what in zip(block.dw_all, params[2:], names):
        near(rows[0], p.grad, what)
        assert all(torch.equal(rows[q], rows[0]) for q in range(R))
    assert block.comm.check() == 0


def test_gradients_by_differences(example):
    """The gradient along a random direction of each parameter against the 64-bit
    network's central difference: h = 1e-5 leaves h^2 of the third derivative and
    2^-52 / h of the value, both under 1e-8."""
    import torch
    block = example.Attention(2, 5, 64, 2, 1, 16, seed=7)
    g = torch.Generator().manual_seed(8)
    stream, d_out = (torch.randn((2, 5 * 64), generator=g) for _ in range(2))
    block.forward(stream.cuda())
    block.backward(stream.cuda(), d_out.cuda())
    torch.cuda.synchronize()
    params = [p.detach() for p in _params(block)]
    grads = block.d_matrices + [rows[0] for rows in block.dw_all]
    for i, grad in enumerate(grads):
        way = torch.randn(params[i].shape, generator=g, dtype=torch.float64)
        way /= way.norm()
        values = []
        for step in (1e-5, -1e-5):
            moved = list(params)
            moved[i] = params[i] + step * way
            values.append(float((_network(example, block, stream.double(), moved)
                                 * d_out.double().view(-1, 64)).sum()))
        slope = (values[0] - values[1]) / 2e-5
        got = float((grad.cpu().double() * way).sum())
        assert abs(got - slope) < 5e-4 * float(grad.double().norm()), i


def test_update(example):
    """Two updates move the matrices by the steps' polynomial of their momentum:
    its float32 form is off by the sums of five steps of three products."""
    import torch
    block = example.Attention(2, 8, 96, 2, 2, 16, seed=5)
    stream, seen = example.train(block, steps=2, rate=0.0)
    assert seen[0] == seen[1]
    before = [w.clone() for w in block.matrices]
    block.update(0.5)
    for w, b, m in zip(block.matrices, before, block.momenta):
        for r in range(2):
            x = m[r].cpu().double()
            scale = max(1.0, x.shape[0] / x.shape[1]) ** 0.5
            x = x / (x.norm() + 1e-7)
            for _ in range(5):
                A = x @ x.t()
                x = 3.4445 * x + (-4.7750 * A + 2.0315 * A @ A) @ x
            moved = (b[r] - w[r]).cpu().double()
            # a step's slope is at most 3.4445, so 2^-21 a step grows to 2^-21 * 485
            assert float((moved - 0.5 * scale * x).norm()) < 2.0 ** -11 * float(x.norm())


@pytest.mark.parametrize("head_norms", (True, False))
def test_training_and_single_tokens(example, head_norms):
    """Runs; a sequence token by token is the same as whole, to float32's sums of
    up to 256 terms through the five products and four norms."""
    import torch
    block = example.Attention(4, 8, 128, 4, 2, 16, head_norms=head_norms, seed=6)
    stream, seen = example.train(block, steps=4)
    assert len(seen) == 4 and all(torch.isfinite(torch.tensor(v)) for v in seen)
    want = block.forward(stream).view(-1, block.H).clone()
    block.start(block.n + 3)
    got = torch.stack([block.next_token(x) for x in stream.view(-1, block.H)])
    torch.cuda.synchronize()
    assert float((got - want).norm()) < 5e-4 * float(want.norm())
    assert bool((block.cache[:, :, block.n:] == 0).all())
    assert block.comm.check() == 0
