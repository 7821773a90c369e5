"""zero_orthogonalize over axes of a million and more: the tensor core's sums lose 7e-8 of
themselves for every 64 terms, so that no sum may be of more than 2^16 of them."""
import pytest
import torch

from tests import norm_plain as npl

pytestmark = pytest.mark.gpu
BF, F32 = torch.bfloat16, torch.float32


def _exact(x):
    """Through the short side: the iteration's X is a matrix P [side, side] times the input."""
    x = x.double()
    a, b, c = npl.NS
    eye = torch.eye(x.shape[0], dtype=torch.float64, device=x.device)
    n = x.square().sum().sqrt() + 1e-7
    gram, p = x @ x.mT / (n * n), eye / n
    for _ in range(5):
        m = a * eye + b * gram + c * gram @ gram
        p, gram = m @ p, m @ gram @ m.mT
    return p @ x


@pytest.mark.parametrize("side,longer", [(1, 1 << 26), (1, (1 << 24) + 7), (4, 1 << 24), (64, 1 << 22), (300, 1 << 20), (520, 300_001), (3, 70_000)])
@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("tall", [False, True])
def test_long_axes(zlib, cuda_device, side, longer, dtype, tall):
    """How long the result is along the exact one: A is cut by 2^10 blocks' worth, 7e-5, and rounded
    to fp16, 2^-12, at each of five steps, in which its error comes through about 1.5 times:
    2.5e-3, where few entries do not average.  By norm besides the roundings to bf16, 2^-8 / sqrt 3,
    and of the rest, a thousandth."""
    g = torch.Generator(device="cuda").manual_seed(side)
    x = torch.randn(side, longer, generator=g, device="cuda").to(dtype)
    ref = _exact(x)
    if tall:
        x = x.mT.contiguous()
    y = torch.empty(x.shape, dtype=BF, device="cuda")
    ws = torch.full((zlib.zero_orthogonalize_workspace(1, *x.shape),), 0xFF, dtype=torch.uint8, device="cuda")
    zlib.zero_orthogonalize(x, y, workspace=ws)
    zlib.zero_status_check()
    y = (y.mT if tall else y).double()
    along = float((y * ref).sum() / ref.square().sum())
    assert abs(along - 1) <= 2.5e-3
    assert float((y - ref).norm() / ref.norm()) <= 2.5e-3 + 2.0 ** -8 / 3 ** 0.5 + 1e-3


def test_a_batch(zlib, cuda_device):
    """Sums in parts for matrices of several tiles, each as alone."""
    x = torch.randint(-8, 9, (3, 300, 140_000), generator=torch.Generator().manual_seed(1)).to(BF).cuda()
    ws = torch.empty(zlib.zero_orthogonalize_workspace(3, 300, 140_000), dtype=torch.uint8, device="cuda")
    y, one = torch.empty_like(x), torch.empty_like(x[0])
    zlib.zero_orthogonalize(x, y, workspace=ws)
    for i in range(3):
        zlib.zero_orthogonalize(x[i], one, workspace=ws)
        assert torch.equal(one, y[i])
        ref = _exact(x[i])
        assert float((y[i].double() - ref).norm() / ref.norm()) <= 1e-3 + 2.0 ** -8 / 3 ** 0.5
