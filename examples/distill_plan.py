"""Distils entropic transport plans into a cross attention, then answers point by point.

Pairs of ordered point clouds (two noisy turns of a helix) are matched with
`fs_sinkhorn_solve`; the barycentric map of each plan is what the attention learns: its
queries are the points of one cloud, its keys and values those of the other, which has
another length in every pair, and a learned bias by relative position knows that the
clouds are ordered.  Training takes `fs_cross_attention` with its gradients; answering
keeps the keys and values and asks for one point at a time.

    python examples/distill_plan.py [--steps 300]
"""
import argparse
import math
import os
import sys

import torch

sys.path.insert(0, os.path.join(os.path.dirname(os.path.abspath(__file__)), ".."))

from streaming_sinkhorn_solver_gb300 import binding as fs  # noqa: E402

HEADS, KEY_HEADS, D = 8, 4, 64
BUCKETS, DISTANCE = 16, 64
TYPE = torch.bfloat16


class CrossAttention(torch.autograd.Function):
    """The library's cross attention as a step that PyTorch can differentiate."""

    @staticmethod
    def forward(ctx, q, k, v, bias, how):
        out, lse = fs.fs_cross_attention(q, k, v, bias=bias, **how)
        ctx.save_for_backward(q, k, v, bias, out, lse)
        ctx.how = how
        return out

    @staticmethod
    def backward(ctx, dout):
        q, k, v, bias, out, lse = ctx.saved_tensors
        return fs.fs_cross_attention_grad(q, k, v, out, lse, dout.contiguous(), bias=bias,
                                          **ctx.how) + (None,)


def clouds(batch, n, m, generator):
    """Batches of n source and up to m target points (lengths differ), with the counts."""
    def helix(points, shift):
        t = torch.linspace(0, 1, points, device="cuda") * 4 * math.pi + shift
        return torch.stack([t.cos(), t.sin(), t / (4 * math.pi)], -1)

    lens = [m - (m // (2 * batch)) * b for b in range(batch)]
    x, y = torch.zeros(batch, n, 3, device="cuda"), torch.zeros(batch, m, 3, device="cuda")
    for b in range(batch):
        noise = 0.05 * torch.randn(n + lens[b], 3, generator=generator, device="cuda")
        x[b] = helix(n, 0.0) + noise[:n]
        y[b, :lens[b]] = 0.8 * helix(lens[b], 0.3 + 0.1 * b) + noise[n:]
    return x, y, torch.tensor(lens, dtype=torch.int32, device="cuda")


def targets(x, y, lens, eps):
    """The barycentric map of the entropic plan of every pair."""
    maps = torch.empty_like(x)
    for b in range(x.shape[0]):
        yb = y[b, :int(lens[b])].contiguous()
        wx = torch.full((x.shape[1],), 1.0 / x.shape[1], device="cuda")
        wy = torch.full((yb.shape[0],), 1.0 / yb.shape[0], device="cuda")
        f, g = fs.fs_sinkhorn_solve(x[b], wx, yb, wy, eps, 200)
        maps[b] = fs.fs_barycentric(x[b], wx, yb, wy, eps, f, g)
    return maps


class Model(torch.nn.Module):
    def __init__(self):
        super().__init__()
        self.q = torch.nn.Linear(9, HEADS * D)
        self.k = torch.nn.Linear(9, KEY_HEADS * D)
        self.v = torch.nn.Linear(9, KEY_HEADS * D)
        self.o = torch.nn.Linear(HEADS * D, 3)
        self.bias = torch.nn.Parameter(torch.zeros(HEADS, BUCKETS))
        self.buckets = torch.from_numpy(fs.fs_relative_buckets(BUCKETS, DISTANCE)).cuda()

    @staticmethod
    def features(p):
        return torch.cat([p, (3 * p).sin(), (3 * p).cos()], -1)

    def queries(self, x):
        return self.q(self.features(x)).unflatten(-1, (HEADS, D)).to(TYPE)

    def cache(self, y):
        """Keys and values of a target cloud: all that answering keeps of it."""
        u = self.features(y)
        return tuple(f(u).unflatten(-1, (KEY_HEADS, D)).to(TYPE) for f in (self.k, self.v))

    def attend(self, q, k, v, lens, first=None):
        how = dict(kv_len=lens, bias_buckets=self.buckets, q_pos=first)
        return self.o(CrossAttention.apply(q, k, v, self.bias.to(TYPE), how).flatten(-2).float())


def main(steps=300, batch=4, n=96, m=192, eps=0.05, report=True):
    """Trains and answers; returns the first loss, the last, and how far the answers of
    single points are from those of whole clouds."""
    torch.manual_seed(0)
    generator = torch.Generator(device="cuda").manual_seed(1)
    x, y, lens = clouds(batch, n, m, generator)
    want = targets(x, y, lens, eps)
    model = Model().cuda()
    optimizer = torch.optim.Adam(model.parameters(), lr=3e-3)
    losses = []
    for step in range(steps):
        loss = (model.attend(model.queries(x), *model.cache(y), lens) - want).square().mean()
        optimizer.zero_grad()
        loss.backward()
        optimizer.step()
        losses.append(loss.detach())
        if report and step % 50 == 0:
            print(f"step {step:4d}  loss {float(loss):.5f}")
    with torch.no_grad():
        whole = model.attend(model.queries(x), *model.cache(y), lens)
        k, v = model.cache(y)
        answers = []
        for i in range(n):
            first = torch.full((batch,), i, dtype=torch.int32, device="cuda")
            answers.append(model.attend(model.queries(x[:, i:i + 1]), k, v, lens, first))
        apart = float((torch.cat(answers, 1) - whole).abs().max())
    fs.fs_check()
    if report:
        print(f"loss {float(losses[0]):.5f} -> {float(losses[-1]):.5f}; "
              f"one point at a time differs by {apart:.2g} at most")
    return float(losses[0]), float(losses[-1]), apart


if __name__ == "__main__":
    parser = argparse.ArgumentParser(description=__doc__.splitlines()[0])
    parser.add_argument("--steps", type=int, default=300)
    main(parser.parse_args().steps)
