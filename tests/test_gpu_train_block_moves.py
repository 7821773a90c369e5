"""The example's block with norms moves every tensor under either optimizer, and by its own
rule: vectors as AdamW does, matrices along minus their orthogonalised momentum."""
import importlib.util
import math
import os

import numpy as np
import pytest
import torch

from tests import norm_plain as npl

pytestmark = pytest.mark.gpu
BF = torch.bfloat16
ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.fixture(scope="module")
def example(zlib):
    spec = importlib.util.spec_from_file_location("train_block", os.path.join(ROOT, "examples", "train_block.py"))
    mod = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(mod)
    return mod


@pytest.mark.parametrize("stage", [1, 2])
@pytest.mark.parametrize("optimizer", ["AdamW", "Muon"])
def test_the_first_step(example, zlib, cuda_device, monkeypatch, stage, optimizer):
    d, ffn, lr, wd = 64, 256, 2e-3, 0.01
    seen = {}
    real = example.zero.ZeroEngine

    class Watched(real):
        def __init__(self, *a, **k):
            super().__init__(*a, **k)
            seen["engine"], seen["before"] = self, self.master.clone()

        def backward(self, grads):
            seen["grads"] = grads.clone()
            super().backward(grads)

    monkeypatch.setattr(example.zero, "ZeroEngine", Watched)
    losses = example.train(stage=stage, steps=1, d=d, ffn=ffn, batch=2, length=32, norms=True, optimizer=optimizer, lr=lr)
    assert all(math.isfinite(x) for x in losses)
    sizes = example.shapes(d, ffn, norms=True)
    numels = [math.prod(s) for s in sizes.values()]
    _, offsets = zlib.zero_layout(numels, 2, with_offsets=True)
    before, after = seen["before"].double(), seen["engine"].master.double()
    mean = seen["grads"].double().mean(0)
    for (name, s), o in zip(sizes.items(), offsets):
        part = slice(o, o + math.prod(s))
        moved, g, w = after[part] - before[part], mean[part], before[part]
        assert int(g.count_nonzero()) > 0.5 * g.numel(), name
        if len(s) == 2 and optimizer == "Muon":
            # g is exact and m = g; u = g + mu m in bf16 is what is orthogonalised.  By norm: 1e-2 for
            # a bf16 matrix of 64 rows, as the header states, 2^-8 / sqrt 3 for the result's rounding,
            # 1e-3 for the rounding of the weights, 2^-24 of some 0.1 beside steps of some 1e-4
            _, u = npl.momentum([x.float().cpu().numpy() for x in seen["grads"][:, part]], 2.0, np.zeros(g.numel(), np.float32), 0.95, True)
            step = npl.orthogonalize(torch.from_numpy(u).to(BF).double().view(s)).reshape(-1).cuda()
            want = -lr * wd * w - lr * 0.2 * max(s) ** 0.5 * step
            assert float((moved - want).norm() / want.norm()) < 1e-2 + 2.0 ** -8 / 3 ** 0.5 + 1e-3, name
        else:
            # m / bc1 = g and v / bc2 = g^2 at the first step, to some 2^-20; then the weights' rounding
            want = -lr * wd * w - lr * g / (g.abs() + 1e-8)
            assert float((moved - want).abs().max()) <= 1e-5 * float(want.abs().max()) + 2.0 ** -23 * float(w.abs().max()), name
