"""The example's decoder block (examples/train_block.py): its loss and every
gradient against the same block in 64 bits under autograd, and that training
under the engines lowers the loss."""
import importlib.util
import math
import os

import pytest
import torch

from tests import dense_plain as dp

pytestmark = pytest.mark.gpu

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.fixture(scope="module")
def example(zlib):
    spec = importlib.util.spec_from_file_location("train_block", os.path.join(ROOT, "examples", "train_block.py"))
    mod = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(mod)
    return mod


def _reference(x, w, heads, batch, p, seed, rank, step):
    """The block in float64, differentiable; x [tokens, d], w a dict of tensors."""
    t, d = x.shape
    length = t // batch
    theta, _ = dp.rope_theta(d // heads)
    qkv = (x @ w["wqkv"].t() + w["bqkv"]).view(t, 3 * heads, -1)
    ang = torch.arange(length, dtype=torch.float64).repeat(batch)[:, None] * torch.from_numpy(theta)[None, :]
    c, s = torch.cos(ang)[:, None], torch.sin(ang)[:, None]
    half = qkv.shape[2] // 2
    a, b = qkv[:, :2 * heads, :half], qkv[:, :2 * heads, half:]
    qk = torch.cat([a * c - b * s, b * c + a * s], -1)
    q, k, v = (z.reshape(batch, length, heads, -1).transpose(1, 2) for z in (qk[:, :heads], qk[:, heads:], qkv[:, 2 * heads:]))
    scores = (q @ k.transpose(2, 3) / math.sqrt(q.shape[-1])).masked_fill(torch.ones(length, length).triu(1).bool(), float("-inf"))
    att = (scores.softmax(-1) @ v).transpose(1, 2).reshape(t, d)
    f = [dp.factor(t, d, p, seed, 2 * rank + i, step) for i in (0, 1)]
    a1 = x + f[0] * (att @ w["wo"].t() + w["bo"])
    h = dp.act(a1 @ w["w1"].t() + w["b1"], dp.GELU_TANH)
    return a1 + f[1] * (h @ w["w2"].t() + w["b2"])


@pytest.mark.parametrize("d,ffn,heads,batch,length,p", [(64, 256, 4, 2, 24, 0.1), (96, 200, 3, 1, 37, 0.0), (128, 512, 2, 3, 65, 0.3)])
def test_block_against_64_bits(example, zlib, cuda_device, d, ffn, heads, batch, length, p):
    sizes = example.shapes(d, ffn)
    numels = [math.prod(s) for s in sizes.values()]
    layout, offsets = zlib.zero_layout(numels, 2, with_offsets=True)
    g = torch.Generator().manual_seed(d)
    flat = torch.zeros(layout.padded_n, dtype=torch.bfloat16)
    for (name, s), o in zip(sizes.items(), offsets):
        flat[o:o + math.prod(s)] = (torch.randn(math.prod(s), generator=g) / math.sqrt(s[-1])).to(torch.bfloat16)
    x = torch.randn(batch * length, d, generator=g).to(torch.bfloat16)
    dy = torch.randn(batch * length, d, generator=g).to(torch.bfloat16)
    w = example.views(flat.cuda(), offsets, sizes)
    grads = torch.zeros(layout.padded_n, dtype=torch.bfloat16, device="cuda")
    gv = example.views(grads, offsets, sizes)
    block = example.Block(batch, length, d, ffn, heads, p, rank=1, seed=5)
    y = block.forward(x.cuda(), w, step=3)
    dx = block.backward(dy.cuda(), w, gv)
    zlib.zero_status_check()

    wr = {n: v.double().requires_grad_() for n, v in example.views(flat, offsets, sizes).items()}
    xr = x.double().requires_grad_()
    ref = _reference(xr, wr, heads, batch, p, 5, 1, 3)
    rg = torch.autograd.grad(ref, [xr, *wr.values()], dy.double())
    # about twenty tensors between input and gradient are rounded to bf16, 2^-9 of
    # themselves each on average (2^-8 at most), independently: 2^-9 sqrt(20) of the
    # norm is 0.009; three times that
    for name, got, want in [("y", y, ref.detach()), ("dx", dx, rg[0]), *[(n, gv[n], r) for n, r in zip(wr, rg[1:])]]:
        off = float((got.double().cpu() - want).norm() / want.norm())
        assert off <= 0.027, (name, off)


@pytest.mark.parametrize("stage,p", [(1, 0.0), (2, 0.1)])
def test_training_lowers_the_loss(example, zlib, cuda_device, stage, p):
    losses = example.train(stage=stage, steps=30, d=128, ffn=512, batch=2, length=64, p=p)
    assert all(math.isfinite(x) for x in losses)
    assert losses[-1] < 0.6 * losses[0], losses


def test_training_repeats(example, zlib, cuda_device):
    runs = [example.train(steps=4, d=64, ffn=256, batch=2, length=32) for _ in range(2)]
    assert runs[0] == runs[1]
