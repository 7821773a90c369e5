"""What the roundings of the orthogonalisation cost, against the exact iteration (CPU):
matrices with directions of very different strength, of both input types."""
import pytest
import torch

from tests import norm_plain as npl

BF, F32 = torch.bfloat16, torch.float32

# from this shorter side on: the most off by norm before the result's rounding, for x in bf16
# and in fp32, as the header states it
LIMITS = {1: (1.5e-2, 1.3e-2), 8: (1.3e-2, 7e-3), 16: (1e-2, 6e-3), 40: (1e-2, 3e-3), 128: (7.5e-3, 2e-3)}


def limit(side, dtype):
    return LIMITS[max(s for s in LIMITS if s <= side)][dtype == F32]


def matrices(side, directions, rest, batch, longer=None, seed=0, scaled=False):
    """[batch, side, longer]: some directions alike and everything else `rest` times that;
    scaled: rows of different size as well."""
    g = torch.Generator().manual_seed(100 * side + seed)
    longer = longer or side + side // 2 + 1

    def normal(*shape):
        return torch.randn(batch, *shape, generator=g, dtype=torch.float64)

    x = rest * normal(side, longer)
    if directions:
        x = x + normal(side, directions) @ normal(directions, longer)
    return x * torch.exp(normal(side, 1)) if scaled else x


def rounded(x, steps=5, coefficients=npl.NS, eps=1e-7):
    """The iteration with the library's roundings for an fp32 input [..., side, longer]:
    operands in fp16, X as hi + lo, B's diagonal in fp32, which stands for B on lo where it
    is most of every row of A; else nothing does."""
    def half(t, scale):
        return (t * scale).float().half().double() / scale

    a, b, c = coefficients
    n = x.square().sum((-2, -1), keepdim=True).sqrt() + eps
    f, e = torch.frexp(n)
    x, s = x * torch.pow(2.0, -e.double()), 1 / f
    for _ in range(steps):
        hi = half(x, 2.0 ** 12)
        lo = half(x - hi, 2.0 ** 23)
        g = half(hi @ hi.mT * s * s, 2.0 ** 10)
        gg = g @ g
        p = b * g + c * gg
        even = (g.diagonal(dim1=-2, dim2=-1) ** 2 / gg.diagonal(dim1=-2, dim2=-1)).amin(-1)[..., None, None]
        even = even > (0.75 if x.shape[-2] < 8 else 0.5)
        d = p.diagonal(dim1=-2, dim2=-1)
        q = half(p - torch.diag_embed(d), 2.0 ** 10)
        d = d.unsqueeze(-1)
        x = s * ((a + d) * hi + (a + d * even) * lo + q @ hi)
        s = torch.ones_like(s)
    return x


@pytest.mark.parametrize("side", [3, 4, 8, 16, 40, 128])
@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("scaled", [False, True])
@pytest.mark.parametrize("rest", [1e-1, 1e-2, 1e-3, 3e-4, 1e-4])
def test_directions_of_different_strength(side, dtype, scaled, rest):
    for directions in sorted({1, 2, 4, 8, side - 1}):
        if directions >= side:
            continue
        x = matrices(side, directions, rest, 12 if side < 100 else 3, seed=directions, scaled=scaled).to(dtype).double()
        ref = npl.orthogonalize(x)
        y = rounded(x) if dtype == F32 else npl.orthogonalize_rounded(x, source_lo=False)
        assert float(((y - ref).norm(dim=(-2, -1)) / ref.norm(dim=(-2, -1))).max()) <= limit(side, dtype), directions


def test_equal_directions_cost_no_more():
    """What decides on B's product with lo leaves matrices without such directions as they were."""
    for side, longer in ((64, 300), (128, 192), (9, 2000)):
        x = matrices(side, 0, 1.0, 2, longer=longer).to(F32).double()
        ref = npl.orthogonalize(x)
        off = [float((y - ref).norm() / ref.norm()) for y in (rounded(x), npl.orthogonalize_rounded(x))]
        assert off[0] <= 1.1 * off[1]
