"""zero_orthogonalize against the exact iteration, by absolute bounds: those that the
header states for each input type and shorter side, with directions of very different
strength, where the products' fp16 operands cost the most.  (test_gpu_orthogonalize
compares with the library's roundings, of whatever size they are.)"""
import pytest
import torch

from tests import norm_plain as npl
from tests.test_orthogonalize_roundings import LIMITS, limit, matrices, rounded

pytestmark = pytest.mark.gpu
BF, F32 = torch.bfloat16, torch.float32


def _off(zlib, x, **kw):
    """By norm, each matrix of a batch."""
    b, rows, cols = x.shape
    y = torch.empty(x.shape, dtype=BF, device="cuda")
    ws = torch.full((zlib.zero_orthogonalize_workspace(b, rows, cols),), 0xFF, dtype=torch.uint8, device="cuda")
    zlib.zero_orthogonalize(x.cuda(), y, workspace=ws, **kw)
    zlib.zero_status_check()
    ref = npl.orthogonalize(x.double().cuda(), **kw)
    return (y.double() - ref).norm(dim=(-2, -1)) / ref.norm(dim=(-2, -1))


# the result's rounding to bf16: half a step of 2^-8 at most, evenly spread 2^-8 / sqrt 3 of an element
BF16 = 2.0 ** -8 / 3 ** 0.5


@pytest.mark.parametrize("side", [3, 4, *sorted(LIMITS)[1:], 200])
@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("tall", [False, True])
@pytest.mark.parametrize("scaled", [False, True])
@pytest.mark.parametrize("rest", [1e-1, 1e-2, 1e-3, 3e-4, 1e-4])
def test_directions_of_different_strength(zlib, cuda_device, side, dtype, tall, scaled, rest):
    for directions in sorted({1, 2, 4, 8, side - 1}):
        if directions >= side:
            continue
        x = matrices(side, directions, rest, 12 if side < 100 else 3, seed=directions, scaled=scaled).to(dtype)
        off = _off(zlib, x.mT.contiguous() if tall else x)
        assert float(off.max()) <= limit(side, dtype) + BF16, (directions, float(off.max()))


@pytest.mark.parametrize("shape", [(300, 520), (520, 300), (700, 520), (512, 2048), (64, 6000), (777, 1300)])
@pytest.mark.parametrize("dtype", [BF, F32])
def test_larger_matrices(zlib, cuda_device, shape, dtype):
    """Several tiles, and a sum in parts; from no strong direction to many."""
    side = min(shape)
    for directions, rest in ((1, 1e-3), (side // 16, 1e-3), (side // 2, 1e-2), (0, 1.0)):
        for scaled in (False, True):
            x = matrices(side, directions, rest, 1, longer=max(shape), seed=directions, scaled=scaled).to(dtype)
            off = _off(zlib, x.mT.contiguous() if shape[0] > shape[1] else x)
            assert float(off.max()) <= limit(side, dtype) + BF16, (directions, rest, scaled, float(off.max()))


def test_a_batch_of_both_kinds(zlib, cuda_device):
    """Matrices whose singular values are alike beside others: each by itself, as alone."""
    x = torch.cat([matrices(48, 1, 1e-3, 2), matrices(48, 0, 1.0, 2, seed=5), matrices(48, 1, 3e-4, 1, seed=2)]).to(F32)
    y = torch.empty(x.shape, dtype=BF, device="cuda")
    ws = torch.empty(zlib.zero_orthogonalize_workspace(5, 48, x.shape[2]), dtype=torch.uint8, device="cuda")
    for _ in range(2):   # a workspace used before
        zlib.zero_orthogonalize(x.cuda(), y, workspace=ws)
    for i in range(5):
        one = torch.empty_like(y[i])
        zlib.zero_orthogonalize(x[i].cuda(), one, workspace=ws)
        assert torch.equal(one, y[i])


@pytest.mark.parametrize("side,longer", [(64, 300), (128, 192), (512, 2048), (333, 517)])
@pytest.mark.parametrize("tall", [False, True])
def test_equal_directions_cost_no_more(zlib, cuda_device, side, longer, tall):
    """Where the diagonal stands for B on lo in all steps that matter, the call's error is its
    model's in size (not entry by entry: a perturbation of 1e-11 changes which operands round
    up).  Without the diagonal it is 1.6 times that and more.  The result's own rounding is that of
    the exact one, and independent: squares of norms add, to 2 % of the larger for some 19000 entries."""
    x = matrices(side, 0, 1.0, 2, longer=longer, seed=7).to(F32)
    exact, model = npl.orthogonalize(x.double()), rounded(x.double())
    given = (x.mT.contiguous() if tall else x).cuda()
    y = torch.empty(given.shape, dtype=BF, device="cuda")
    ws = torch.full((zlib.zero_orthogonalize_workspace(*given.shape),), 0xFF, dtype=torch.uint8, device="cuda")
    zlib.zero_orthogonalize(given, y, workspace=ws)
    zlib.zero_status_check()
    y = (y.mT if tall else y).cpu().double()
    off, own, cost = ((t - exact).square().sum((-2, -1)) for t in (y, exact.to(BF).double(), model))
    assert bool((off <= 1.02 * own + 1.25 ** 2 * cost).all()), ((off - own) / cost).sqrt()
