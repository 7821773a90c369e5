"""zero_rope against its 64-bit statement: both layouts, part of the head, every
scaling, contiguous and given positions up to the largest, strided and in-place
tensors, and the turn back as the gradient."""
import math

import numpy as np
import pytest
import torch

from tests import dense_plain as dp

pytestmark = pytest.mark.gpu
BF, F32 = torch.bfloat16, torch.float32


def _tol(x, ref, rot, dtype, scale):
    """The reduced angle is an fp32 number of turns (2^-24 of half a turn: an error
    of pi 2^-24 radians, doubled for forming it) and sine and cosine are within
    2^-22: 2^-20 of a pair's magnitude; then storing."""
    size = x.abs().max() if x.numel() else torch.tensor(0.0)
    return 2.0 ** -20 * 2 * scale * size + dp.eps_out(dtype) * ref.abs() + 1e-30


def _x(g, shape, dtype):
    return torch.randn(*shape, generator=g, dtype=torch.float64).clamp(-4, 4).to(dtype)


CASES = [  # tokens, heads, dim, rot
    (1, 1, 2, 2), (1, 64, 128, 128), (5, 3, 64, 32), (33, 25, 64, 64), (100, 4, 80, 20), (7, 2, 256, 256),
    (19, 5, 96, 2), (257, 8, 128, 64), (3, 1, 300, 250), (2, 7, 33, 6),
]


@pytest.mark.parametrize("case", CASES)
@pytest.mark.parametrize("layout", [0, 1])
@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("scaling", [0, 3])
def test_rope(zlib, cuda_device, case, layout, dtype, scaling):
    t, h, d, rot = case
    g = torch.Generator().manual_seed(t * 100 + d)
    x = _x(g, (t, h, d), dtype)
    plan = zlib.zero_rope_plan(rot, layout=layout, scaling=scaling, factor=4.0, context=512)
    theta, scale = dp.rope_theta(rot, 10000.0, scaling, 4.0, 512)
    pos = torch.randint(0, 1 << 20, (t,), generator=g)
    for inverse in (False, True):
        y = torch.empty(t, h, d, dtype=dtype, device="cuda")
        zlib.zero_rope(plan, x.cuda(), y, positions=pos.cuda(), inverse=inverse)
        ref = dp.rope(x.double(), pos.numpy(), rot, layout, theta, scale, inverse)
        dp.close(y, ref, _tol(x.double(), ref, rot, dtype, scale))
        assert torch.equal(y.cpu()[..., rot:], x[..., rot:])


@pytest.mark.parametrize("scaling", [0, 1, 2, 3])
@pytest.mark.parametrize("pos0", [0, 131071, 2 ** 40, -5])
def test_rope_positions_in_order(zlib, cuda_device, scaling, pos0):
    g = torch.Generator().manual_seed(3)
    x = _x(g, (40, 6, 64), F32)
    plan = zlib.zero_rope_plan(64, scaling=scaling, factor=8.0, context=4096)
    theta, scale = dp.rope_theta(64, 10000.0, scaling, 8.0, 4096)
    y = torch.empty(40, 6, 64, device="cuda")
    zlib.zero_rope(plan, x.cuda(), y, pos0=pos0)
    if abs(pos0) <= 1 << 20:
        ref = dp.rope(x.double(), np.arange(pos0, pos0 + 40), 64, 0, theta, scale)
    else:   # too far for a product in doubles: the plan's integers turn exactly
        turns = np.array([[((pos0 + t) * plan.turn[i]) % 2 ** 64 / 2.0 ** 64 for i in range(32)] for t in range(40)])
        ang = torch.from_numpy(turns * 2 * math.pi)[:, None, :]
        a, b = x.double()[..., :32], x.double()[..., 32:]
        c, s = torch.cos(ang) * scale, torch.sin(ang) * scale
        ref = torch.cat([a * c - b * s, b * c + a * s], -1)
    dp.close(y, ref, _tol(x.double(), ref, 64, F32, scale))
    same = torch.empty_like(y)
    zlib.zero_rope(plan, x.cuda(), same, positions=torch.arange(pos0, pos0 + 40, device="cuda"))
    assert torch.equal(y, same)


@pytest.mark.parametrize("layout", [0, 1])
@pytest.mark.parametrize("dtype", [BF, F32])
def test_rope_strided_and_in_place(zlib, cuda_device, layout, dtype):
    """Queries and keys inside a packed projection, in place: the values beside them
    stay; heads outermost; odd strides and places."""
    g = torch.Generator().manual_seed(5)
    t, h, d = 50, 12, 64
    packed = _x(g, (t, h, d), dtype).cuda()
    plan = zlib.zero_rope_plan(48, layout=layout)
    theta, _ = dp.rope_theta(48)
    ref = dp.rope(packed[:, :8].double().cpu(), np.arange(t), 48, layout, theta, 1.0)
    keep = packed.clone()
    zlib.zero_rope(plan, packed[:, :8], packed[:, :8])
    dp.close(packed[:, :8], ref, _tol(keep.double().cpu(), ref, 48, dtype, 1.0))
    assert torch.equal(packed[:, 8:], keep[:, 8:]) and torch.equal(packed[:, :8, 48:], keep[:, :8, 48:])
    # [heads, tokens, dim] taken as [tokens, heads, dim]
    out = torch.empty(8, t, d, dtype=dtype, device="cuda").transpose(0, 1)
    zlib.zero_rope(plan, keep[:, :8], out)
    assert torch.equal(out, packed[:, :8])
    # every pointer and stride odd
    buf = torch.full((t * (8 * (d + 1) + 3) + 64,), dp.SENTINEL, dtype=dtype, device="cuda")
    odd = torch.as_strided(buf, (t, 8, d), (8 * (d + 1) + 3, d + 1, 1), 1)
    odd.copy_(keep[:, :8])
    zlib.zero_rope(plan, odd, odd)
    assert torch.equal(odd, packed[:, :8])
    odd.fill_(dp.SENTINEL)
    assert bool((buf == dp.SENTINEL).all())


@pytest.mark.parametrize("layout", [0, 1])
def test_turning_back_is_the_gradient(zlib, cuda_device, layout):
    """<R x, c> = <x, R' c> for the turn R and the inverse call R' (by the same
    scale), and differences of <R x, c> along random directions are <v, R' c>."""
    g = torch.Generator().manual_seed(6)
    x, c, v = (_x(g, (20, 3, 64), F32) for _ in range(3))
    plan = zlib.zero_rope_plan(32, layout=layout, scaling=3, factor=4.0, context=128)
    theta, scale = dp.rope_theta(32, 10000.0, 3, 4.0, 128)
    back = torch.empty(20, 3, 64, device="cuda")
    zlib.zero_rope(plan, c.cuda(), back, inverse=True, pos0=1000)
    pos = np.arange(1000, 1020)

    def value(xd):
        return float((dp.rope(xd, pos, 32, layout, theta, scale) * c.double()).sum())

    want = (value(x.double() + 1e-4 * v.double()) - value(x.double() - 1e-4 * v.double())) / 2e-4
    got = float((back.double().cpu() * v.double()).sum())
    assert abs(want - got) <= 2.0 ** -19 * 2 * scale * 4 * float(v.double().abs().sum())
    y = torch.empty_like(back)
    zlib.zero_rope(plan, back, y, pos0=1000)
    turned = c.double().clone()
    turned[..., :32] *= scale * scale
    dp.close(y, turned, 2.0 ** -18 * scale * scale * 4 * 2)


def test_rope_nothing(zlib, cuda_device):
    plan = zlib.zero_rope_plan(64)
    for shape in ((0, 4, 64), (4, 0, 64)):
        x = torch.empty(*shape, dtype=BF, device="cuda")
        zlib.zero_rope(plan, x, torch.empty_like(x))


def test_rope_refusals(zlib, cuda_device):
    plan, x = zlib.zero_rope_plan(64), torch.zeros(4, 2, 64, dtype=BF, device="cuda")
    for bad in (x[:3], x.float(), torch.zeros(4, 2, 32, dtype=BF, device="cuda")):
        with pytest.raises((ValueError, zlib.ZeroError)):
            zlib.zero_rope(plan, x, bad)
    with pytest.raises(zlib.ZeroError):   # heads of the output on top of one another
        zlib.zero_rope(plan, x, x[:, :1].expand(4, 2, 64))
    with pytest.raises(ValueError):
        zlib.zero_rope(plan, x, x, positions=torch.zeros(3, dtype=torch.int64, device="cuda"))
    with pytest.raises(TypeError):
        zlib.zero_rope(plan, x, x, positions=torch.zeros(4, dtype=torch.int32, device="cuda"))
    with pytest.raises(TypeError):
        zlib.zero_rope(plan, x.half(), x.half())


@pytest.mark.slow
def test_offsets_past_32_bits(zlib, cuda_device):
    t, stride = 70, 1 << 26
    big = torch.empty(t * stride, dtype=BF, device="cuda")
    view = torch.as_strided(big, (t, 2, 64), (stride, 64, 1))
    x = torch.randn(t, 2, 64, device="cuda").to(BF)
    view.copy_(x)
    plan = zlib.zero_rope_plan(64)
    ref = torch.empty_like(x)
    zlib.zero_rope(plan, x, ref)
    zlib.zero_rope(plan, view, view)
    assert torch.equal(view, ref)
