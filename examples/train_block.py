"""Trains one decoder block under ZeRO with the library's dense operators.

    python examples/train_block.py [--stage 2] [--steps 40] [--dim 256] ...

The block's weights are views of the engine's flat bf16 weights, its gradients
views of the ranks' flat bf16 gradient buffers; between the two run

    qkv = x wqkv^T + bqkv                      zero_linear
    q, k turned by position, in place          zero_rope
    a   = x + D(attention(q, k, v) wo^T + bo)  zero_linear (the attention itself: torch)
    h   = gelu(a w1^T + b1)                    zero_linear, keeping the pre-activation
    y   = a + D(h w2^T + b2)                   zero_linear

and backward the gradient calls, none of which store a mask.  The task is to
follow a fixed random map of the input; each simulated rank has its own tokens.
"""
from __future__ import annotations

import argparse
import math
import os
import sys

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

import torch  # noqa: E402

import zero_sharded_mixed_gb300 as zero  # noqa: E402

BF = torch.bfloat16


def shapes(d: int, ffn: int) -> dict:
    return {"wqkv": (3 * d, d), "bqkv": (3 * d,), "wo": (d, d), "bo": (d,),
            "w1": (ffn, d), "b1": (ffn,), "w2": (d, ffn), "b2": (d,)}


def views(flat: torch.Tensor, offsets: list[int], sizes: dict) -> dict:
    """The block's tensors inside a flat buffer."""
    return {n: flat[o:o + math.prod(s)].view(s) for (n, s), o in zip(sizes.items(), offsets)}


def attention(qkv: torch.Tensor, batch: int) -> torch.Tensor:
    """Causal attention of [tokens, 3 heads, dim], plain torch, for the example only."""
    t, h, d = qkv.shape[0] // batch, qkv.shape[1] // 3, qkv.shape[2]
    q, k, v = (p.view(batch, t, h, d).transpose(1, 2).float() for p in qkv.split(h, dim=1))
    scores = q @ k.transpose(2, 3) / math.sqrt(d)
    scores = scores.masked_fill(torch.ones(t, t, dtype=torch.bool, device=qkv.device).triu(1), float("-inf"))
    return (scores.softmax(-1) @ v).transpose(1, 2).reshape(batch * t, h * d).to(BF)


class Block:
    """One rank's buffers for `batch` sequences of `length` tokens."""

    def __init__(self, batch: int, length: int, d: int, ffn: int, heads: int, p: float, rank: int = 0, seed: int = 1):
        self.batch, self.heads, self.p, self.rank, self.seed = batch, heads, p, rank, seed
        rows = batch * length

        def new(cols):
            return torch.empty(rows, cols, dtype=BF, device="cuda")

        self.qkv, self.a, self.pre, self.h, self.y = new(3 * d), new(d), new(ffn), new(ffn), new(d)
        self.dz2, self.dz1, self.da, self.dzo, self.datt, self.dx = new(d), new(ffn), new(d), new(d), new(d), new(d)
        self.plan = zero.zero_rope_plan(d // heads)
        self.at = torch.arange(length, device="cuda").repeat(batch)

    def drops(self, step: int):
        """A site for each place, a step for each pass; ranks draw apart by their sites."""
        if not self.p:
            return None, None
        return [zero.ZeroDropout.make(self.p, seed=self.seed, site=2 * self.rank + i, step=step) for i in (0, 1)]

    def turned(self, qkv, inverse=False):
        """Queries and keys of the packed projection, turned where they stand."""
        part = qkv.view(qkv.shape[0], 3 * self.heads, -1)[:, :2 * self.heads]
        zero.zero_rope(self.plan, part, part, positions=self.at, inverse=inverse)

    def forward(self, x, w, step):
        self.x, self.drop = x, self.drops(step)
        zero.zero_linear(x, w["wqkv"], self.qkv, bias=w["bqkv"])
        self.turned(self.qkv)
        self.att = attention(self.qkv.view(x.shape[0], 3 * self.heads, -1), self.batch)
        zero.zero_linear(self.att, w["wo"], self.a, bias=w["bo"], residual=x, drop=self.drop[0])
        zero.zero_linear(self.a, w["w1"], self.h, bias=w["b1"], act=zero.ZERO_ACT_GELU_TANH, pre=self.pre)
        zero.zero_linear(self.h, w["w2"], self.y, bias=w["b2"], residual=self.a, drop=self.drop[1])
        return self.y

    def backward(self, dy, w, g):
        """Writes every gradient into g (views of the rank's flat buffer); returns dx."""
        zero.zero_dropout_grad(dy, self.dz2, self.drop[1], db=g["b2"])
        zero.zero_linear_grad_weight(self.dz2, self.h, g["w2"])
        zero.zero_linear_grad_input(self.dz2, w["w2"], self.dz1, act=zero.ZERO_ACT_GELU_TANH, pre=self.pre)
        zero.zero_linear_grad_weight(self.dz1, self.a, g["w1"], db=g["b1"])
        zero.zero_linear_grad_input(self.dz1, w["w1"], self.da, residual=dy)
        zero.zero_dropout_grad(self.da, self.dzo, self.drop[0], db=g["bo"])
        zero.zero_linear_grad_weight(self.dzo, self.att, g["wo"])
        zero.zero_linear_grad_input(self.dzo, w["wo"], self.datt)
        qkv = self.qkv.view(self.qkv.shape[0], 3 * self.heads, -1).detach().requires_grad_()
        with torch.enable_grad():
            dqkv, = torch.autograd.grad(attention(qkv, self.batch), qkv, self.datt)
        dqkv = dqkv.reshape(self.qkv.shape).contiguous()
        self.turned(dqkv, inverse=True)
        zero.zero_linear_grad_weight(dqkv, self.x, g["wqkv"], db=g["bqkv"])
        zero.zero_linear_grad_input(dqkv, w["wqkv"], self.dx, residual=self.da)
        return self.dx


def train(stage=2, steps=40, ranks=2, batch=4, length=128, d=256, ffn=1024, heads=4, p=0.1, lr=2e-3, seed=0,
          report=lambda step, loss: None) -> list[float]:
    """Losses of `steps` steps (the mean over the ranks)."""
    sizes = shapes(d, ffn)
    numels = [math.prod(s) for s in sizes.values()]
    cfg = zero.ZeroConfig.from_dict({
        "zero_optimization": {"stage": stage},
        "optimizer": {"type": "AdamW", "params": {"lr": lr, "betas": [0.9, 0.95], "weight_decay": 0.01}}})
    layout, offsets = zero.zero_layout(numels, ranks, with_offsets=True)
    gen = torch.Generator(device="cuda").manual_seed(seed)
    master = torch.zeros(layout.padded_n, device="cuda")
    for (name, s), o in zip(sizes.items(), offsets):
        if len(s) == 2:
            master[o:o + math.prod(s)].normal_(0.0, 1 / math.sqrt(s[1]), generator=gen)
    engine = zero.ZeroEngine(numels, ranks, cfg, master=master)
    w = views(engine.weights, offsets, sizes)
    grads = torch.zeros(ranks, layout.padded_n, dtype=BF, device="cuda")
    blocks = [Block(batch, length, d, ffn, heads, p, r, seed + 1) for r in range(ranks)]
    target = torch.randn(d, d, generator=gen, device="cuda") / math.sqrt(d)
    losses = []
    for step in range(steps):
        total = 0.0
        for r, block in enumerate(blocks):
            x = torch.randn(batch * length, d, generator=gen, device="cuda").to(BF)
            y = block.forward(x, w, step)
            off = y.float() - x.float() @ target
            total = total + off.square().mean()
            block.backward((off * (2 / off.numel())).to(BF), w, views(grads[r], offsets, sizes))
        engine.backward(grads)
        engine.step()
        losses.append(float(total) / ranks)
        report(step, losses[-1])
    return losses


def main(argv=None):
    ap = argparse.ArgumentParser(description=__doc__.splitlines()[0])
    for name, kind, default in (("stage", int, 2), ("steps", int, 40), ("ranks", int, 2), ("batch", int, 4),
                                ("length", int, 128), ("d", int, 256), ("ffn", int, 1024), ("heads", int, 4),
                                ("p", float, 0.1), ("lr", float, 2e-3), ("seed", int, 0)):
        ap.add_argument("--" + name, type=kind, default=default)
    args = ap.parse_args(argv)
    losses = train(**vars(args), report=lambda s, l: print(f"step {s:4d}  loss {l:.4f}", flush=True))
    print(f"loss {losses[0]:.4f} -> {losses[-1]:.4f}")


if __name__ == "__main__":
    main()
