"""MuonStep's calls stay within what a call takes, whatever the number of matrices (CPU)."""
import pytest
import torch

from zero_sharded_mixed_gb300 import binding as zb
from zero_sharded_mixed_gb300 import step as zs


@pytest.mark.parametrize("count", [1, 65535, 65536, 140000])
def test_many_small_matrices(count):
    L, offsets = zb.zero_layout([8] * count, 1, with_offsets=True)
    muon = zs.MuonStep(L, offsets, [(2, 4)] * count, device="cpu")
    sizes = [b.shape[0] for b in muon.batches]
    assert sum(sizes) == count and max(sizes) <= 65535
    covered = [b.storage_offset() + i * b.stride(0) for b in muon.batches for i in range(b.shape[0])]
    assert sorted(covered) == list(offsets)
    assert muon.workspace.numel() >= max(zb.zero_orthogonalize_workspace(b.shape[0], 2, 4) for b in muon.batches)


@pytest.mark.gpu
def test_a_step_of_them(zlib, cuda_device):
    count = 70000
    L, offsets = zb.zero_layout([8] * count, 1, with_offsets=True)
    muon = zs.MuonStep(L, offsets, [(2, 4)] * count)
    g = torch.Generator().manual_seed(1)
    grads = torch.randn(L.padded_n, generator=g).to(torch.bfloat16).cuda()
    m = torch.zeros(L.padded_n, device="cuda")
    hp = zb.ZeroMuon.make(nesterov=True)
    zb.zero_reduce_scatter_momentum(L, [grads], zb.ZERO_BF16, 0, 1.0, 0, 1, 0, L.n, m, muon.update, zb.ZERO_OUT_FULL, hp)
    u = muon.update.clone()
    for x in muon.batches:
        zb.zero_orthogonalize(x, x, workspace=muon.workspace)
    zb.zero_status_check()
    for i in (0, 1, 65534, 65535, count - 1):
        x, y = u[8 * i:8 * i + 8].view(2, 4), torch.empty(2, 4, dtype=torch.bfloat16, device="cuda")
        zb.zero_orthogonalize(x, y, workspace=muon.workspace)
        # the norm of so small a matrix has one part alone and in a batch
        assert torch.equal(y, muon.update[8 * i:8 * i + 8].view(2, 4)), i
