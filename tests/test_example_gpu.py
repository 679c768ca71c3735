"""examples/tensor_parallel_step.py: its gradients against automatic
differentiation of the same network in 64 bits on the host, its training, and
its 8-bit inference pass."""
import importlib.util
import os

import pytest

pytestmark = pytest.mark.gpu

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.fixture(scope="module")
def example():
    spec = importlib.util.spec_from_file_location(
        "tensor_parallel_step", os.path.join(ROOT, "examples", "tensor_parallel_step.py"))
    m = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(m)
    return m


@pytest.mark.parametrize("R,tokens,hidden", [(2, 3, 64), (4, 17, 200), (8, 32, 256)])
def test_gradients(example, R, tokens, hidden):
    """Float32 sums of at most 400 terms through five products and two norms:
    off by at most about 5 * 400 * 2^-24 of the terms' sizes, 1.2e-4; the norms
    of whole tensors are compared to 2e-4."""
    import torch
    block = example.Block(R, tokens, hidden, seed=3)
    g = torch.Generator().manual_seed(4)
    shape = (R, tokens * hidden)
    stream, d_out = (torch.randn(shape, generator=g) for _ in range(2))
    out = block.forward(stream.cuda()).clone()
    d_stream = block.backward(stream.cuda(), d_out.cuda())
    torch.cuda.synchronize()

    d = torch.float64
    W1, W2, w1, w2 = (p.detach().cpu().to(d).requires_grad_() for p in
                      (block.W1, block.W2, block.w1, block.w2))
    s = stream.to(d).view(-1, hidden).requires_grad_()

    def norm(x, w):
        return x * torch.rsqrt((x * x).mean(1, keepdim=True) + example.EPS) * w
    n = norm(s, w1)
    s2 = s + sum(torch.nn.functional.gelu(n @ W1[q]) @ W2[q] for q in range(R))
    want = norm(s2, w2)
    want.backward(d_out.to(d).view(-1, hidden))

    def near(got, ref, what):
        got, ref = got.detach().cpu().to(d).reshape(ref.shape), ref.detach()
        assert float((got - ref).norm() / ref.norm()) < 2e-4, what
    near(out, want, "out")
    near(d_stream, s.grad, "d_stream")
    for got, ref, what in zip(block.grads.tensors, (W1, W2, w1, w2), ("W1", "W2", "w1", "w2")):
        near(got, ref.grad, what)
    for rows in block.dw_all:
        assert all(torch.equal(rows[q], rows[0]) for q in range(R))
    total = sum(float((t.double() ** 2).sum()) for t in block.grads.tensors) ** 0.5
    assert abs(float(block.clip(total / 2)) - total) < 1e-6 * total
    after = sum(float((t.double() ** 2).sum()) for t in block.grads.tensors) ** 0.5
    assert abs(after - total / 2) < 1e-5 * total


def test_training_and_inference(example):
    import torch
    block = example.Block(4, 16, 256)
    stream, seen = example.train(block, steps=12)
    losses = [loss for loss, _ in seen]
    assert all(b < a for a, b in zip(losses, losses[1:])), losses
    want = block.forward(stream).view(-1, block.H).clone()
    for group in (0, 64, 128):
        got = block.infer_e4m3(stream, group)
        assert bool((got == got[0]).all())
        # a value is off by at most half a step of its e4m3 binade, 2^-4 of it, or
        # half the smallest step, 2^-10, of its group's scale (at most max |v| / 448)
        bound = want.abs() * 2.0 ** -4 * 1.001 + 2.0 ** -10 * want.abs().amax(1, keepdim=True) / 448
        assert bool(((got[0] - want).abs() <= bound).all()), group
    assert block.comm.check() == 0
