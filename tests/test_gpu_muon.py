"""zero_reduce_scatter_momentum and zero_muon_update bit for bit against their 32-bit
statement: rank counts, both source types, ranges anywhere, both output places, a
device-resident learning rate, pinned sources."""
import numpy as np
import pytest
import torch

from tests import norm_plain as npl

pytestmark = pytest.mark.gpu
BF, F32 = torch.bfloat16, torch.float32


def _bits(t):
    return t.cpu().view(torch.int16 if t.dtype == BF else torch.int32)


RANGES = [(1, 0, 1), (1, 5, 6), (2, 0, 64), (2, 3, 1003), (3, 40, 977), (4, 1, 20001), (8, 4801, 4809), (8, 77, 300000), (8, 0, 1 << 20),
          (5, 8, 9999), (64, 11, 5000)]


@pytest.mark.parametrize("ranks,begin,end", RANGES)
@pytest.mark.parametrize("src", ["bf16", "f32"])
@pytest.mark.parametrize("nesterov", [True, False])
def test_momentum(zlib, cuda_device, ranks, begin, end, src, nesterov):
    g = torch.Generator().manual_seed(end)
    L = zlib.zero_layout([end + 7], ranks)
    P = L.padded_n
    grads = [torch.randn(P, generator=g).to(BF if src == "bf16" else F32) for _ in range(ranks)]
    m = torch.randn(P, generator=g)
    md, u = m.cuda(), torch.full((P,), 3.0, dtype=BF, device="cuda")
    hp = zlib.ZeroMuon.make(momentum=0.95, nesterov=nesterov)
    zlib.zero_reduce_scatter_momentum(L, [x.cuda() for x in grads], zlib.ZERO_BF16 if src == "bf16" else zlib.ZERO_F32, 0, float(ranks),
                                      0, ranks, begin, end, md, u, zlib.ZERO_OUT_FULL, hp)
    part = slice(begin, end)
    rm, ru = m.clone(), torch.full((P,), 3.0, dtype=BF)
    a, b = npl.momentum([x[part].float().numpy() for x in grads], float(ranks), m[part].numpy(), 0.95, nesterov)
    rm[part], ru[part] = torch.from_numpy(a), torch.from_numpy(b).to(BF)
    assert torch.equal(_bits(md), _bits(rm)) and torch.equal(_bits(u), _bits(ru))


@pytest.mark.parametrize("ranks,begin,end", RANGES)
@pytest.mark.parametrize("on_device", [False, True])
def test_update(zlib, cuda_device, ranks, begin, end, on_device):
    g = torch.Generator().manual_seed(end)
    L = zlib.zero_layout([end + 7], ranks)
    P = L.padded_n
    w, o = torch.randn(P, generator=g), torch.randn(P, generator=g).to(BF)
    wd, out = w.cuda(), torch.full((P,), 3.0, dtype=BF, device="cuda")
    lr = 0.0213
    sched = torch.tensor([lr, 1.0, 1.0], device="cuda") if on_device else None
    hp = zlib.ZeroMuon.make(lr=99.0 if on_device else lr, weight_decay=0.1, scale=0.37, sched=sched)
    zlib.zero_muon_update(L, o.cuda(), 0, 0, ranks, begin, end, wd, out, zlib.ZERO_OUT_FULL, hp)
    part = slice(begin, end)
    rw, ro = w.clone(), torch.full((P,), 3.0, dtype=BF)
    a = npl.muon_update(w[part].numpy(), o[part].float().numpy(), np.float32(lr), np.float32(0.1), np.float32(0.37))
    rw[part], ro[part] = torch.from_numpy(a), torch.from_numpy(a).to(BF)
    assert torch.equal(_bits(wd), _bits(rw)) and torch.equal(_bits(out), _bits(ro))


def test_owners_ranges_and_bases(zlib, cuda_device):
    """A middle owner's shard: state and output by the shard, sources from a base, one launch an owner."""
    g = torch.Generator().manual_seed(0)
    L = zlib.zero_layout([5000], 4)
    S, P = L.shard, L.padded_n
    grads = [torch.randn(P, generator=g).to(BF) for _ in range(4)]
    m, w, o = torch.randn(P, generator=g), torch.randn(P, generator=g), torch.randn(P, generator=g).to(BF)
    hp = zlib.ZeroMuon.make(lr=0.1, momentum=0.9, weight_decay=0.01, scale=0.2)
    rm, ru = npl.momentum([x.float().numpy() for x in grads], 4.0, m.numpy(), 0.9, True)
    rw = npl.muon_update(w.numpy(), o.float().numpy(), np.float32(0.1), np.float32(0.01), np.float32(0.2))
    for rank in range(4):
        lo, hi = rank * S, (rank + 1) * S
        base = max(0, lo - 3)
        md, u = m[lo:hi].cuda(), torch.zeros(S, dtype=BF, device="cuda")
        zlib.zero_reduce_scatter_momentum(L, [x[base:hi].cuda() for x in grads], zlib.ZERO_BF16, base, 4.0, rank, rank + 1, lo, hi,
                                          md, u, zlib.ZERO_OUT_SHARD, hp)
        assert torch.equal(_bits(md), _bits(torch.from_numpy(rm[lo:hi])))
        assert torch.equal(_bits(u), _bits(torch.from_numpy(ru[lo:hi]).to(BF)))
        wd, out = w[lo:hi].cuda(), torch.zeros(S, dtype=BF, device="cuda")
        zlib.zero_muon_update(L, o[base:hi].cuda(), base, rank, rank + 1, lo, hi, wd, out, zlib.ZERO_OUT_SHARD, hp)
        assert torch.equal(_bits(wd), _bits(torch.from_numpy(rw[lo:hi])))
        assert torch.equal(_bits(out), _bits(torch.from_numpy(rw[lo:hi]).to(BF)))


def test_pinned_sources(zlib, cuda_device):
    L = zlib.zero_layout([4099], 2)
    grads = [torch.randn(L.padded_n).to(BF) for _ in range(2)]
    hp = zlib.ZeroMuon.make()
    out = []
    for where in ([x.cuda() for x in grads], [x.pin_memory() for x in grads]):
        m, u = torch.ones(L.padded_n, device="cuda"), torch.zeros(L.padded_n, dtype=BF, device="cuda")
        zlib.zero_reduce_scatter_momentum(L, where, zlib.ZERO_BF16, 0, 2.0, 0, 2, 0, L.padded_n, m, u, zlib.ZERO_OUT_FULL, hp)
        torch.cuda.synchronize()
        out.append((m, u))
    assert torch.equal(out[0][0], out[1][0]) and torch.equal(out[0][1], out[1][1])


def test_special_values(zlib, cuda_device):
    L = zlib.zero_layout([64], 1)
    grad = torch.zeros(64, dtype=BF)
    grad[3], grad[9], grad[20] = float("nan"), float("inf"), 3e38
    m, u = torch.zeros(64, device="cuda"), torch.zeros(64, dtype=BF, device="cuda")
    zlib.zero_reduce_scatter_momentum(L, [grad.cuda()], zlib.ZERO_BF16, 0, 1.0, 0, 1, 0, 64, m, u, zlib.ZERO_OUT_FULL, zlib.ZeroMuon.make())
    assert torch.isnan(m[3]) and torch.isnan(u[3]) and torch.isinf(u[9]) and torch.isfinite(m[20]) and torch.isinf(u[20])
    assert int(torch.isfinite(u).sum()) == 61
