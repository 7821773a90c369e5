"""Bounded waits count their own kernel's time alone."""
import math

import pytest
import torch

pytestmark = pytest.mark.gpu
BF = torch.bfloat16


def test_a_long_predecessor_is_no_timeout(zlib, cuda_device):
    """The orthogonalisation's kernels start while the calls before them still run, here for
    seconds (one CTA a row), where its own waits give up after about one."""
    rows, cols = 1, 1 << 28
    x = torch.ones(rows, cols, device="cuda")
    y = torch.empty(rows, cols, dtype=BF, device="cuda")
    g = torch.Generator().manual_seed(1)
    for shape in ((40, 64), (300, 520)):
        u = torch.randn(*shape, generator=g).to(BF).cuda()
        ws = torch.empty(zlib.zero_orthogonalize_workspace(1, *shape), dtype=torch.uint8, device="cuda")
        alone, after = torch.empty_like(u), torch.empty_like(u)
        zlib.zero_orthogonalize(u, alone, workspace=ws)
        ev = [torch.cuda.Event(enable_timing=True) for _ in range(2)]
        ev[0].record()
        zlib.zero_layer_norm(x, y)
        ev[1].record()
        ev[1].synchronize()
        calls = math.ceil(2500 / ev[0].elapsed_time(ev[1]))
        for _ in range(calls):
            zlib.zero_layer_norm(x, y)
        zlib.zero_orthogonalize(u, after, workspace=ws)
        zlib.zero_status_check()
        assert torch.equal(after, alone)
