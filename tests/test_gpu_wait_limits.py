"""Bounded waits count their own kernel's time alone, and give up in order."""
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


def test_a_team_gives_up_together(zlib, cuda_device):
    """A wait that gives up in one warp and ends in time in another: both leave their ring, and
    the gradient whose ring that is goes on as before."""
    g = torch.Generator().manual_seed(2)
    rows, cols = 300, 1601   # off the 16-byte grid, a row to several warps
    x, dy = (torch.randn(rows, cols, generator=g).to(BF).cuda() for _ in range(2))
    y, mean, rstd = torch.empty_like(x), torch.empty(rows, device="cuda"), torch.empty(rows, device="cuda")
    zlib.zero_layer_norm(x, y, mean=mean, rstd=rstd)
    ws = torch.empty(zlib.zero_layer_norm_grad_workspace(rows, cols), dtype=torch.uint8, device="cuda")

    def grad():
        out = [torch.empty_like(x), *(torch.empty(cols, device="cuda") for _ in range(2))]
        zlib.zero_layer_norm_grad(dy, x, mean, rstd, out[0], dgamma=out[1], dbeta=out[2], workspace=ws)
        return out

    before = grad()
    zlib.zero_status_check()
    for limit in (1, 50_000, 2_000_000):
        zlib.zero_selftest_bounded_wait(limit)
        with pytest.raises(zlib.ZeroError) as e:
            zlib.zero_status_check()
        assert e.value.code == zlib.ZERO_ETIMEOUT
        after = grad()
        zlib.zero_status_check()
        assert all(torch.equal(a, b) for a, b in zip(after, before))
