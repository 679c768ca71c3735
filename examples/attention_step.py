"""A training step of one tensor- and sequence-parallel attention block over R
logical ranks, with an orthogonalised update, and its single-token steps, on the
library's operators.

The residual stream is cut by tokens, the heads by ranks: rank q owns tokens
[q t, (q + 1) t) of the stream, `heads` query heads and `kv_heads` key and value
heads.  A block is

    n   = norm(stream)                 api.rmsnorm
    all-gather n, so that every rank has all tokens
    q, k, v = n Wqkv_q                 each rank its heads
    q, k = norm of each head, rotated  api.head_rmsnorm, from one product's heads
                                       (or api.rotary alone, without head norms)
    p_q = attention(q, k, v) Wo_q      causal
    stream' = stream + sum over q of p_q, out = norm'(stream')
                                       Comm.reduce_scatter_rmsnorm: one pass

and the loss is the mean square of out - target.  The backward pass mirrors it
(api.head_rmsnorm_backward writes into the gradient of the one product).  The
weight matrices go along their momentum's orthogonal directions
(api.orthogonalize, all ranks' matrices in one call), the norms' weights along
their gradients.  In single-token steps the new key goes straight into the cache.
The products and the attention itself are torch's.

    python examples/attention_step.py [--ranks 8] [--tokens 32] [--hidden 512]
"""
import argparse
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
from collective_communication_ring_amd import api  # noqa: E402

EPS = 1e-6


class Attention:
    """Weights, buffers and communicators of R ranks on one GPU, float32."""

    def __init__(self, R=8, tokens=32, hidden=512, heads=4, kv_heads=2, dim=32, layout="halves",
                 head_norms=True, seed=0, device="cuda"):
        g = torch.Generator().manual_seed(seed)
        make = lambda *shape, scale=1.0: (torch.randn(shape, generator=g) * scale).to(device)  # noqa: E731
        row = lambda *shape: torch.empty(shape, device=device)  # noqa: E731
        self.R, self.t, self.H, self.n = R, tokens, hidden, R * tokens
        self.heads, self.kv_heads, self.D = heads, kv_heads, dim
        n, each = self.n, heads + 2 * kv_heads
        self.Wqkv = make(R, hidden, each * dim, scale=hidden ** -0.5)
        self.Wo = make(R, heads * dim, hidden, scale=(R * heads * dim) ** -0.5)
        self.w1, self.w2 = (1.0 + make(hidden, scale=0.1) for _ in range(2))  # the norms'
        self.wq, self.wk = (1.0 + make(dim, scale=0.1) for _ in range(2))  # the heads' norms'
        self.head_norms = head_norms
        self.rotation = api.Rotation(dim, 10000.0, layout, device=device)
        self.positions = torch.arange(n, dtype=torch.int32, device=device)
        self.hidden_mask = torch.ones(n, n, dtype=torch.bool, device=device).triu(1)
        self.comm = api.Comm(R, n * hidden, "float32", device=device)
        self.small = api.Comm(R, hidden, "float32", device=device)
        self.head_comm = api.Comm(R, dim, "float32", device=device)
        self.normed, self.stream2, self.out, self.d_n = (row(R, tokens * hidden) for _ in range(4))
        self.every, self.partial = row(R, n * hidden), row(R, n * hidden)
        self.rstd1, self.rstd2 = row(n), row(R, tokens)
        self.d_stream2, self.d_stream = row(n, hidden), row(n, hidden)
        self.qkv, self.d_qkv = row(R, n, each, dim), row(R, n, each, dim)
        self.q, self.k = row(R, n, heads, dim), row(R, n, kv_heads, dim)
        self.dw = [row(R, hidden), row(R, hidden), row(R, dim), row(R, dim)]
        self.dw_all = [torch.empty_like(d) for d in self.dw]
        self.norm_workspace = api.rmsnorm_backward_workspace(R, n, hidden, device)
        self.head_workspace = api.head_rmsnorm_backward_workspace(R, dim, device)
        self.matrices = [self.Wqkv, self.Wo]
        self.d_matrices = [torch.empty_like(w) for w in self.matrices]
        self.momenta = [torch.zeros_like(w) for w in self.matrices]
        self.workspaces = [api.orthogonalize_workspace(R, *w.shape[1:], w.dtype, device)
                           for w in self.matrices]

    def split(self, x):
        """The queries', keys' and values' heads of [..., heads + 2 kv_heads, D]."""
        return x.split([self.heads, self.kv_heads, self.kv_heads], dim=-2)

    def turn(self, q, k, q_out, k_out, positions):
        if self.head_norms:
            api.head_rmsnorm(q, self.wq, q_out, EPS, k=k, k_weight=self.wk, k_out=k_out,
                             positions=positions, rotation=self.rotation)
        else:
            api.rotary(q, positions, self.rotation, q_out, k=k, k_out=k_out)

    def by_head(self, x, heads):
        """[R, tokens, heads, D] as [R, query heads, tokens, D], keys' and values'
        heads repeated for the queries that share them."""
        return x.repeat_interleave(self.heads // heads, dim=2).transpose(1, 2).contiguous()

    def forward(self, stream):
        """out [R, t * H] of a stream [R, t * H]; keeps what backward needs."""
        R, H, n = self.R, self.H, self.n
        api.rmsnorm(stream.view(-1, H), self.w1, self.normed.view(-1, H), EPS, rstd=self.rstd1)
        self.comm.all_gather(self.normed, self.every)
        torch.bmm(self.every.view(R, n, H), self.Wqkv, out=self.qkv.view(R, n, -1))
        q, k, v = self.split(self.qkv)
        self.turn(q, k, self.q, self.k, self.positions)
        q, k, v = (self.by_head(x, h) for x, h in ((self.q, self.heads), (self.k, self.kv_heads),
                                                   (v, self.kv_heads)))
        s = q @ k.transpose(2, 3) * self.D ** -0.5
        p = torch.softmax(s.masked_fill_(self.hidden_mask, float("-inf")), dim=3)
        self.mixed = (p @ v).transpose(1, 2).reshape(R, n, -1)
        self.kept = q, k, v, p
        torch.bmm(self.mixed, self.Wo, out=self.partial.view(R, n, H))
        self.comm.reduce_scatter_rmsnorm(self.partial, self.w2, self.out, EPS, residual=stream,
                                         sum=self.stream2, rstd=self.rstd2)
        return self.out

    def backward(self, stream, d_out):
        """Gradients of the weights (self.d_matrices, self.dw_all) and of the
        stream, given out's."""
        R, H, n = self.R, self.H, self.n
        api.rmsnorm_backward(d_out.view(-1, H), self.stream2.view(-1, H), self.w2,
                             self.rstd2.view(-1), self.d_stream2, self.dw[1],
                             workspace=self.norm_workspace)
        d_every = torch.empty_like(self.partial)
        self.comm.all_gather(self.d_stream2.view(R, -1), d_every)
        d_every = d_every.view(R, n, H)
        torch.bmm(self.mixed.transpose(1, 2), d_every, out=self.d_matrices[1])
        q, k, v, p = self.kept
        d_o = (d_every @ self.Wo.transpose(1, 2)).view(R, n, self.heads, -1).transpose(1, 2)
        d_p = d_o @ v.transpose(2, 3)
        d_s = p * (d_p - (d_p * p).sum(3, keepdim=True)) * self.D ** -0.5
        shared = lambda x: x.transpose(1, 2).reshape(  # noqa: E731
            R, n, self.kv_heads, -1, self.D).sum(3)  # heads that share a key add up
        dq, dk, dv = self.split(self.d_qkv)
        dv.copy_(shared(p.transpose(2, 3) @ d_o))
        dq_out, dk_out = (d_s @ k).transpose(1, 2), shared(d_s.transpose(2, 3) @ q)
        if self.head_norms:
            q, k, _ = self.split(self.qkv)
            api.head_rmsnorm_backward(dq_out, q, self.wq, dq, self.dw[2], EPS, dk_out=dk_out, k=k,
                                      k_weight=self.wk, dk=dk, k_dweight=self.dw[3],
                                      positions=self.positions, rotation=self.rotation,
                                      workspace=self.head_workspace)
        else:
            api.rotary(dq_out, self.positions, self.rotation, dq, k=dk_out, k_out=dk, inverse=True)
        d_qkv = self.d_qkv.view(R, n, -1)
        torch.bmm(self.every.view(R, n, H).transpose(1, 2), d_qkv, out=self.d_matrices[0])
        torch.bmm(d_qkv, self.Wqkv.transpose(1, 2), out=self.partial.view(R, n, H))
        self.comm.reduce_scatter(self.partial, self.d_n)
        api.rmsnorm_backward(self.d_n.view(-1, H), stream.view(-1, H), self.w1, self.rstd1,
                             self.d_stream, self.dw[0], dsum=self.d_stream2,
                             workspace=self.norm_workspace)
        comms = (self.small, self.small, self.head_comm, self.head_comm)
        for comm, own, whole in list(zip(comms, self.dw, self.dw_all))[:4 if self.head_norms else 2]:
            comm.allreduce(own, whole)
        return self.d_stream

    def update(self, rate, momentum=0.9):
        for w, d, m, workspace in zip(self.matrices, self.d_matrices, self.momenta, self.workspaces):
            m.mul_(momentum).add_(d)
            direction = torch.empty_like(m)
            api.orthogonalize(m, direction, scale=max(1.0, m.shape[1] / m.shape[2]) ** 0.5,
                              workspace=workspace)
            w.sub_(direction, alpha=rate)
        for w, d in list(zip((self.w1, self.w2, self.wq, self.wk), self.dw_all))[:4 if self.head_norms else 2]:
            w.sub_(d[0], alpha=rate)

    def start(self, room):
        """Caches of keys and values for `room` tokens, of none yet."""
        self.cache = torch.zeros((2, self.R, room, self.kv_heads, self.D), device=self.w1.device)
        self.length = 0

    def next_token(self, x):
        """out [H] of the next token's stream [H], which all ranks have."""
        R, H, at = self.R, self.H, self.length
        keys, values = self.cache
        y, s, rstd = torch.empty(1, H, device=x.device), x.view(1, H), torch.empty(1, device=x.device)
        api.rmsnorm(s, self.w1, y, EPS, rstd=rstd)
        qkv = torch.matmul(y, self.Wqkv).view(R, 1, -1, self.D)
        q, k, v = self.split(qkv)
        position = torch.full((1,), at, dtype=torch.int32, device=x.device)
        self.turn(q, k, q, keys[:, at:at + 1], position)  # the query in place, the key to the cache
        values[:, at:at + 1] = v
        self.length = at + 1
        q, k, v = (self.by_head(a, h) for a, h in ((q, self.heads), (keys[:, :at + 1], self.kv_heads),
                                                   (values[:, :at + 1], self.kv_heads)))
        p = torch.softmax(q @ k.transpose(2, 3) * self.D ** -0.5, dim=3)
        s = s + torch.bmm((p @ v).view(R, 1, -1), self.Wo).sum(0)
        out = torch.empty_like(s)
        api.rmsnorm(s, self.w2, out, EPS, rstd=rstd)
        return out.view(H)


def train(block, steps=20, rate=0.02, seed=1):
    """Loss of each step towards a random target."""
    g = torch.Generator().manual_seed(seed)
    shape = (block.R, block.t * block.H)
    stream, target = (torch.randn(shape, generator=g).to(block.w1.device) for _ in range(2))
    seen = []
    for _ in range(steps):
        diff = block.forward(stream) - target
        block.backward(stream, diff * (2.0 / diff.numel()))
        seen.append(float((diff * diff).mean()))
        block.update(rate)
    return stream, seen


def main():
    ap = argparse.ArgumentParser(description=__doc__.split("\n\n")[0])
    ap.add_argument("--ranks", type=int, default=8)
    ap.add_argument("--tokens", type=int, default=32, help="per rank")
    ap.add_argument("--hidden", type=int, default=512)
    ap.add_argument("--steps", type=int, default=20)
    ap.add_argument("--no-head-norms", action="store_true")
    a = ap.parse_args()
    block = Attention(a.ranks, a.tokens, a.hidden, head_norms=not a.no_head_norms)
    stream, seen = train(block, a.steps)
    for k, loss in enumerate(seen):
        if k % 5 == 0 or k == len(seen) - 1:
            print("step %3d  loss %.5f" % (k, loss), flush=True)
    want = block.forward(stream).view(-1, block.H)
    block.start(block.n)
    got = torch.stack([block.next_token(x) for x in stream.view(-1, block.H)])
    print("token by token: %.1e off (2-norm)" % float((got - want).norm() / want.norm()))
    assert block.comm.check() == api.AR_SUCCESS


if __name__ == "__main__":
    main()
