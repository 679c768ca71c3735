"""A training step of one tensor- and sequence-parallel block over R logical
ranks, and its 8-bit inference pass, on the library's operators.

The residual stream is cut by tokens: rank q owns tokens [q t, (q + 1) t), and
its stream is row q of an [R, t * H] array.  A block is

    n   = norm(stream)                 api.rmsnorm
    all-gather n, so that every rank has all tokens
    p_q = gelu(n W1_q) W2_q            each rank its columns of W1, rows of W2
    stream' = stream + sum over q of p_q, out = norm'(stream')
                                       Comm.reduce_scatter_rmsnorm: one pass

and the loss is the mean square of out - target.  The backward pass mirrors it
(api.rmsnorm_backward twice, an all-gather and a reduce-scatter), the norms'
weight gradients, one row per rank, are all-reduced, and the gradients are
clipped to a global norm (Comm.grad_norm, Comm.grad_clip) before a plain
gradient step.  The products are torch's.

    python examples/tensor_parallel_step.py [--ranks 8] [--tokens 64] [--hidden 512]
"""
import argparse
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
from collective_communication_ring_amd import api  # noqa: E402

EPS = 1e-6


def gelu(x):
    return 0.5 * x * (1.0 + torch.erf(x * 0.5 ** 0.5))


def gelu_slope(x):
    return 0.5 * (1.0 + torch.erf(x * 0.5 ** 0.5)) + \
        x * torch.exp(-0.5 * x * x) * (0.5 / torch.pi) ** 0.5


class Block:
    """Weights, buffers and communicators of R ranks on one GPU, float32."""

    def __init__(self, R=8, tokens=64, hidden=512, seed=0, device="cuda"):
        g = torch.Generator().manual_seed(seed)
        F = 2 * hidden // R  # a rank's inner width
        make = lambda *shape, scale=1.0: (torch.randn(shape, generator=g) * scale).to(device)  # noqa: E731
        self.R, self.t, self.H, n = R, tokens, hidden, R * tokens
        self.W1 = make(R, hidden, F, scale=hidden ** -0.5)
        self.W2 = make(R, F, hidden, scale=(R * F) ** -0.5)
        self.w1 = 1.0 + make(hidden, scale=0.1)  # the norms' weights
        self.w2 = 1.0 + make(hidden, scale=0.1)
        self.comm = api.Comm(R, n * hidden, "float32", device=device)
        self.small = api.Comm(R, hidden, "float32", device=device)
        # e4m3 bytes travel as int32 words
        self.words = api.Comm(R, n * hidden // 4, "int32", device=device)
        row = lambda *shape: torch.empty(shape, device=device)  # noqa: E731
        self.normed, self.stream2, self.out, self.d_n = (row(R, tokens * hidden) for _ in range(4))
        self.every, self.partial = row(R, n * hidden), row(R, n * hidden)
        self.rstd1, self.rstd2, self.norm = row(n), row(R, tokens), row(1)
        self.d_stream2, self.d_stream = row(n, hidden), row(n, hidden)
        self.dw = [row(R, hidden), row(R, hidden)]
        self.workspace = api.rmsnorm_backward_workspace(R, n, hidden, device)
        self.dW1, self.dW2 = torch.empty_like(self.W1), torch.empty_like(self.W2)
        self.dw_all = [row(R, hidden), row(R, hidden)]
        # what is clipped: every rank's own shards, and one copy of what all ranks share
        self.grads = api.TensorList([self.dW1, self.dW2, self.dw_all[0][0], self.dw_all[1][0]])

    def forward(self, stream):
        """out [R, t * H] of a stream [R, t * H]; keeps what backward needs."""
        H = self.H
        tokens = stream.view(-1, H)
        api.rmsnorm(tokens, self.w1, self.normed.view(-1, H), EPS, rstd=self.rstd1)
        self.comm.all_gather(self.normed, self.every)
        self.inner = []
        for q in range(self.R):
            a = self.every[q].view(-1, H) @ self.W1[q]
            self.inner.append(a)
            torch.mm(gelu(a), self.W2[q], out=self.partial[q].view(-1, H))
        self.comm.reduce_scatter_rmsnorm(self.partial, self.w2, self.out, EPS, residual=stream,
                                         sum=self.stream2, rstd=self.rstd2)
        return self.out

    def backward(self, stream, d_out):
        """Gradients of the weights (self.grads) and of the stream, given out's."""
        H = self.H
        api.rmsnorm_backward(d_out.view(-1, H), self.stream2.view(-1, H), self.w2,
                             self.rstd2.view(-1), self.d_stream2, self.dw[1],
                             workspace=self.workspace)
        # each rank needs all tokens' gradient of its partial sums
        d_every = torch.empty_like(self.partial)
        self.comm.all_gather(self.d_stream2.view(self.R, -1), d_every)
        for q in range(self.R):
            n, d, a = self.every[q].view(-1, H), d_every[q].view(-1, H), self.inner[q]
            torch.mm(gelu(a).t(), d, out=self.dW2[q])
            da = (d @ self.W2[q].t()) * gelu_slope(a)
            torch.mm(n.t(), da, out=self.dW1[q])
            torch.mm(da, self.W1[q].t(), out=self.partial[q].view(-1, H))
        self.comm.reduce_scatter(self.partial, self.d_n)
        # the stream's gradient also comes past the block, through stream2
        api.rmsnorm_backward(self.d_n.view(-1, H), stream.view(-1, H), self.w1, self.rstd1,
                             self.d_stream, self.dw[0], dsum=self.d_stream2,
                             workspace=self.workspace)
        for own, whole in zip(self.dw, self.dw_all):
            self.small.allreduce(own, whole)
        return self.d_stream

    def clip(self, max_norm):
        """Clips the gradients to a global norm; their norm before it, on the
        device."""
        self.comm.grad_norm(self.grads, self.norm)
        self.comm.grad_clip(self.grads, self.norm, max_norm)
        return self.norm

    def update(self, rate):
        for w, d in zip((self.W1, self.W2, self.w1, self.w2), self.grads.tensors):
            w -= rate * d

    def infer_e4m3(self, stream, group=128):
        """The block's output in 8 bits with scales, gathered to every rank: a
        quarter of float32's bytes in the all-gather.  Values [R, tokens, H],
        equal for all ranks."""
        R, H = self.R, self.H
        self.forward(stream)
        groups = -(-H // group) if group else 1
        y = torch.empty((R, self.t * H), dtype=torch.float8_e4m3fn, device=stream.device)
        scale = torch.empty((R, self.t * groups), device=stream.device)
        self.comm.reduce_scatter_rmsnorm(self.partial, self.w2, y, EPS, residual=stream, scale=scale,
                                         group=group)
        every = torch.empty((R, R * self.t * H // 4), dtype=torch.int32, device=stream.device)
        self.words.all_gather(y.view(torch.int32), every)
        scales = torch.empty((R, R * self.t * groups), device=stream.device)
        self.comm.all_gather(scale, scales)
        wide = scales.view(R, -1, groups).repeat_interleave(group or H, dim=2)[:, :, :H]
        return every.view(torch.float8_e4m3fn).view(R, -1, H).to(torch.float32) * wide


def train(block, steps=20, rate=0.5, max_norm=1.0, seed=1):
    """Loss and gradient norm of each step towards a random target."""
    g = torch.Generator().manual_seed(seed)
    device = block.W1.device
    shape = (block.R, block.t * block.H)
    stream, target = (torch.randn(shape, generator=g).to(device) for _ in range(2))
    seen = []
    for _ in range(steps):
        diff = block.forward(stream) - target
        block.backward(stream, diff * (2.0 / diff.numel()))
        seen.append((float((diff * diff).mean()), float(block.clip(max_norm))))
        block.update(rate)
    return stream, seen


def main():
    ap = argparse.ArgumentParser(description=__doc__.split("\n\n")[0])
    ap.add_argument("--ranks", type=int, default=8)
    ap.add_argument("--tokens", type=int, default=64, help="per rank")
    ap.add_argument("--hidden", type=int, default=512)
    ap.add_argument("--steps", type=int, default=20)
    a = ap.parse_args()
    block = Block(a.ranks, a.tokens, a.hidden)
    stream, seen = train(block, a.steps)
    for k, (loss, norm) in enumerate(seen):
        if k % 5 == 0 or k == len(seen) - 1:
            print("step %3d  loss %.5f  gradient norm %.5f" % (k, loss, norm), flush=True)
    want = block.forward(stream).view(-1, block.H).clone()
    got = block.infer_e4m3(stream)
    err = float((got[0] - want).norm() / want.norm())
    print("8-bit output, gathered: %.4f off (2-norm), equal on all ranks: %s"
          % (err, bool((got == got[0]).all())))
    assert block.comm.check() == api.AR_SUCCESS and seen[-1][0] < seen[0][0]


if __name__ == "__main__":
    main()
