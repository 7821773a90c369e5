"""A step by orthogonalised momentum through the engine: the elementwise ends bit for bit
against the 32-bit statement, the orthogonalised part by the library's own call on the
same momentum (held against the iteration in its own tests), vectors bit for bit as
AdamW's; accumulation in both stages, resuming, a captured step, and the example's block
with its norms."""
import importlib.util
import math
import os

import numpy as np
import pytest
import torch

from tests import dense_plain as dp
from tests import norm_plain as npl
from zero_sharded_mixed_gb300 import step as zs
from zero_sharded_mixed_gb300.config import ZeroConfig
from zero_sharded_mixed_gb300.engine import ZeroEngine

pytestmark = pytest.mark.gpu
BF = torch.bfloat16
ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))

# matrices wide, tall, equal at equal distances, one by itself; vectors between; odd sizes
SHAPES = [(33, 65), (33,), (40, 24), (24,), (40, 24), (24,), (40, 24), (3,), (130, 7), (), (1, 50), (2, 3, 4)]
LR, WD, MU = 0.01, 0.1, 0.9


def _config(stage, K):
    return ZeroConfig.from_dict({"gradient_accumulation_steps": K, "zero_optimization": {"stage": stage, "reduce_bucket_size": 4000},
                                 "optimizer": {"type": "Muon", "params": {"lr": LR, "momentum": MU, "weight_decay": WD, "betas": [0.9, 0.95]}}})


def _adamw(g, w, m, v, t):
    f = np.float32
    b1, b2 = f(0.9), f(0.95)
    bc1, bc2 = f(1 - float(b1) ** t), f(1 - float(b2) ** t)
    m = (b1 * m + (f(1) - b1) * g).astype(f)
    v = (b2 * v + (f(1) - b2) * (g * g).astype(f)).astype(f)
    w = (w - (f(LR) * f(WD)) * w).astype(f)
    return (w - f(LR) * ((m / bc1) / (np.sqrt(v / bc2) + f(1e-8)))).astype(f), m, v


@pytest.mark.parametrize("stage,K,ranks", [(2, 1, 2), (1, 1, 4), (2, 3, 2), (1, 2, 3)])
def test_steps(zlib, cuda_device, stage, K, ranks):
    numels = [math.prod(s) for s in SHAPES]
    g = torch.Generator().manual_seed(stage * 10 + K)
    L, offsets = zlib.zero_layout(numels, ranks, with_offsets=True)
    w0 = torch.zeros(L.padded_n)
    w0[:L.n] = torch.randn(L.n, generator=g) * 0.1
    eng = ZeroEngine(numels, ranks, _config(stage, K), master=w0.cuda(), shapes=SHAPES)
    f = np.float32
    w, m, v = w0.numpy().copy(), np.zeros(L.padded_n, f), np.zeros(L.padded_n, f)
    for t in (1, 2, 3):
        micro = []
        for _ in range(K):
            grad = torch.zeros(ranks, L.padded_n, dtype=BF)
            grad[:, :L.n] = (torch.randn(ranks, L.n, generator=g) * 0.01).to(BF)
            micro.append(grad.float().numpy())
            eng.backward(grad.cuda())
        eng.step()
        zlib.zero_status_check()
        if K == 1:
            srcs = list(micro[0])
        elif stage == 1:
            srcs = [sum_in_order([x[r] for x in micro]) for r in range(ranks)]
        else:
            srcs = [sum_in_order([sum_in_order(list(x), f(0)) for x in micro])]
        update = torch.zeros(L.padded_n, dtype=BF)
        for o, s in zip(offsets, SHAPES):
            n = math.prod(s)
            part = slice(o, o + n)
            mean = (sum_in_order([x[part] for x in srcs], f(0)) / f(ranks * K)).astype(f)
            if len(s) != 2:
                w[part], m[part], v[part] = _adamw(mean, w[part], m[part], v[part], t)
                continue
            m[part], u = npl.momentum([x[part] for x in srcs], ranks * K, m[part], MU, True)
            x = torch.from_numpy(u).to(BF).view(s).cuda()
            y = torch.empty_like(x)
            zlib.zero_orthogonalize(x, y, workspace=torch.empty(zlib.zero_orthogonalize_workspace(1, *s), dtype=torch.uint8, device="cuda"))
            update[part] = y.cpu().reshape(-1)
            w[part] = npl.muon_update(w[part], update[part].float().numpy(), f(LR), f(WD), f(0.2 * max(s) ** 0.5))
        assert torch.equal(eng.m.cpu(), torch.from_numpy(m)), t
        assert torch.equal(eng.v.cpu(), torch.from_numpy(v)), t
        assert torch.equal(eng.muon.update.cpu(), update), t
        assert torch.equal(eng.master.cpu(), torch.from_numpy(w)), t
        assert torch.equal(eng.weights.cpu(), torch.from_numpy(w).to(BF)), t
    assert bool((eng.weights[L.n:] == 0).all())


def sum_in_order(xs, start=None):
    s = xs[0] if start is None else (np.zeros_like(xs[0]) + xs[0]).astype(np.float32)
    for x in xs[1:]:
        s = (s + x).astype(np.float32)
    return s


def test_equal_matrices_are_one_call(zlib, cuda_device):
    numels = [math.prod(s) for s in SHAPES]
    eng = ZeroEngine(numels, 2, _config(2, 1), shapes=SHAPES)
    assert sorted(tuple(b.shape) for b in eng.muon.batches) == [(1, 1, 50), (1, 33, 65), (1, 130, 7), (3, 40, 24)]
    assert eng.memory_estimate()["this_process_bytes"] > 0
    for bad in (None, SHAPES[:-1], [(66, 33), *SHAPES[1:]]):
        with pytest.raises(ValueError):
            ZeroEngine(numels, 2, _config(2, 1), shapes=bad)


def test_resume_and_graph(zlib, cuda_device, tmp_path):
    """Saved and restored, a run goes on bit for bit; and so does a captured step."""
    numels, ranks = [math.prod(s) for s in SHAPES], 2
    g = torch.Generator().manual_seed(1)
    L, offsets = zlib.zero_layout(numels, ranks, with_offsets=True)
    w0 = torch.zeros(L.padded_n)
    w0[:L.n] = torch.randn(L.n, generator=g)
    grads = [torch.zeros(ranks, L.padded_n, dtype=BF) for _ in range(4)]
    for x in grads:
        x[:, :L.n] = torch.randn(ranks, L.n, generator=g).to(BF)
    a = ZeroEngine(numels, ranks, _config(2, 1), master=w0.cuda(), shapes=SHAPES)
    for t in range(4):
        if t == 2:
            a.save_checkpoint(tmp_path)
        a.backward(grads[t].cuda())
        a.step()
    b = ZeroEngine(numels, ranks, _config(2, 1), shapes=SHAPES)
    assert b.load_checkpoint(tmp_path) == 2
    for t in (2, 3):
        b.backward(grads[t].cuda())
        b.step()
    assert torch.equal(a.master, b.master) and torch.equal(a.m, b.m) and torch.equal(a.weights, b.weights)

    muon = zs.MuonStep(L, offsets, SHAPES)
    sched = zs.StepSchedule(LR, 0.9, 0.95, 1e-8, WD, 10)
    master, m, v = w0.cuda(), torch.zeros(L.padded_n, device="cuda"), torch.zeros(L.padded_n, device="cuda")
    out, fixed = torch.zeros(L.padded_n, dtype=BF, device="cuda"), grads[0].cuda()

    def one_step():
        sched.advance()
        muon.run([fixed[r] for r in range(ranks)], zlib.ZERO_BF16, float(ranks), master, m, v, out, sched.hp(), 99.0, MU)

    graph = zs.GraphStep(one_step)   # the first step
    for t in (1, 2, 3):
        fixed.copy_(grads[t])
        graph.replay()
    torch.cuda.synchronize()
    zlib.zero_status_check()
    assert torch.equal(master, a.master) and torch.equal(m, a.m) and torch.equal(out, a.weights)


@pytest.fixture(scope="module")
def example(zlib):
    spec = importlib.util.spec_from_file_location("train_block", os.path.join(ROOT, "examples", "train_block.py"))
    mod = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(mod)
    return mod


def _reference(x, w, heads, batch, p, seed, rank, step):
    """The block with its norms in float64, differentiable."""
    def norm(z, g, c):
        return torch.nn.functional.layer_norm(z, (z.shape[1],), g, c, 1e-5)

    t, d = x.shape
    length = t // batch
    theta, _ = dp.rope_theta(d // heads)
    qkv = (norm(x, w["g1"], w["c1"]) @ w["wqkv"].t() + w["bqkv"]).view(t, 3 * heads, -1)
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
    h = dp.act(norm(a1, w["g2"], w["c2"]) @ w["w1"].t() + w["b1"], dp.GELU_TANH)
    return a1 + f[1] * (h @ w["w2"].t() + w["b2"])


@pytest.mark.parametrize("d,ffn,heads,batch,length,p", [(64, 256, 4, 2, 24, 0.1), (96, 200, 3, 1, 37, 0.0)])
def test_block_with_norms_against_64_bits(example, zlib, cuda_device, d, ffn, heads, batch, length, p):
    sizes = example.shapes(d, ffn, norms=True)
    numels = [math.prod(s) for s in sizes.values()]
    layout, offsets = zlib.zero_layout(numels, 2, with_offsets=True)
    g = torch.Generator().manual_seed(d)
    flat = torch.zeros(layout.padded_n, dtype=BF)
    for (name, s), o in zip(sizes.items(), offsets):
        flat[o:o + math.prod(s)] = ((torch.randn(math.prod(s), generator=g) / math.sqrt(s[-1])) + name.startswith("g")).to(BF)
    x = torch.randn(batch * length, d, generator=g).to(BF)
    dy = torch.randn(batch * length, d, generator=g).to(BF)
    grads = torch.zeros(layout.padded_n, dtype=BF, device="cuda")
    gv = example.views(grads, offsets, sizes)
    block = example.Block(batch, length, d, ffn, heads, p, rank=1, seed=5, norms=True)
    w = example.views(flat.cuda(), offsets, sizes)
    y = block.forward(x.cuda(), w, step=3)
    dx = block.backward(dy.cuda(), w, gv)
    zlib.zero_status_check()
    wr = {n: t.double().requires_grad_() for n, t in example.views(flat, offsets, sizes).items()}
    xr = x.double().requires_grad_()
    ref = _reference(xr, wr, heads, batch, p, 5, 1, 3)
    rg = torch.autograd.grad(ref, [xr, *wr.values()], dy.double())
    # about twenty-five tensors between input and gradient are rounded to bf16, 2^-9 of
    # themselves each on average, independently: 2^-9 sqrt(25) of the norm is 0.01; three times that
    for name, got, want in [("y", y, ref.detach()), ("dx", dx, rg[0]), *[(n, gv[n], r) for n, r in zip(wr, rg[1:])]]:
        off = float((got.double().cpu() - want).norm() / want.norm())
        assert off <= 0.03, (name, off)


@pytest.mark.parametrize("optimizer,stage", [("AdamW", 2), ("Muon", 1), ("Muon", 2)])
def test_the_example_runs_with_norms(example, zlib, cuda_device, optimizer, stage):
    """Finite losses, the same each time."""
    kw = dict(stage=stage, steps=5, d=64, ffn=256, batch=2, length=32, norms=True, optimizer=optimizer)
    runs = [example.train(**kw) for _ in range(2)]
    assert runs[0] == runs[1] and all(math.isfinite(x) for x in runs[0])
