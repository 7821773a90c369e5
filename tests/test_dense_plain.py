"""CPU checks of the dense operators: the 64-bit statements that the kernels are
compared with (the generator against its published vectors, gradients against
differences), the rotary plan, and the argument checks that return before any
CUDA call."""
import ctypes
import math

import numpy as np
import pytest
import torch

from tests import dense_plain as dp

FAKE = 0x10000   # never dereferenced


def test_philox_published_vectors():
    """The known answers published with the generator for Philox4x32-10."""
    for counter, key, want in [
        ((0, 0, 0, 0), (0, 0), (0x6627E8D5, 0xE169C58D, 0xBC57AC4C, 0x9B00DBD8)),
        ((0xFFFFFFFF,) * 4, (0xFFFFFFFF,) * 2, (0x408F276D, 0x41C83B0E, 0xA20BC7C6, 0x6D5451FD)),
        ((0x243F6A88, 0x85A308D3, 0x13198A2E, 0x03707344), (0xA4093822, 0x299F31D0),
         (0xD16CFE09, 0x94FDCCEB, 0x5001E420, 0x24126EA1)),
    ]:
        assert tuple(int(x) for x in dp.philox4x32(counter, key)) == want


def test_dropout_factor_statistics():
    """The kept share and the mean of the factor over 2^20 elements, within six
    standard deviations of a binomial."""
    for p in (0.1, 0.5, 0.9):
        f = dp.factor(1024, 1024, p, seed=5, site=2, step=9)
        q = 1 - dp.cut_of(p) / 65536
        n = f.numel()
        share = float((f != 0).double().mean())
        assert abs(share - q) <= 6 * math.sqrt(q * (1 - q) / n)
        assert abs(float(f.mean()) - 1) <= 6 * math.sqrt((1 - q) / q / n)
    assert not torch.equal(dp.factor(8, 64, 0.5, site=1), dp.factor(8, 64, 0.5, site=2))
    assert not torch.equal(dp.factor(8, 64, 0.5, step=1), dp.factor(8, 64, 0.5, step=2))
    assert float(dp.factor(8, 64, 1.0).abs().max()) == 0


@pytest.mark.parametrize("a", dp.ACTS)
def test_slopes_against_differences(a):
    z = torch.linspace(-6, 6, 1201, dtype=torch.float64) + 1e-3
    h = 1e-6
    diff = (dp.act(z + h, a) - dp.act(z - h, a)) / (2 * h)
    assert float((diff - dp.slope(z, a)).abs().max()) < 1e-8


@pytest.mark.parametrize("scaling", [0, 1, 2, 3])
def test_rope_plan(zlib, scaling):
    for rot in (2, 16, 64, 256):
        plan = zlib.zero_rope_plan(rot, layout=1, base=10000.0, scaling=scaling, factor=8.0, context=2048)
        theta, scale = dp.rope_theta(rot, 10000.0, scaling, 8.0, 2048)
        assert plan.rot == rot and plan.layout == 1
        assert plan.scale == pytest.approx(scale, rel=1e-7)
        for i in range(rot // 2):   # 2^-52 relative of pow and division, and half a unit
            want = theta[i] / (2 * math.pi) * 2.0 ** 64
            assert abs(plan.turn[i] - want) <= 0.5 + want * 2.0 ** -49
        assert all(plan.turn[i] == 0 for i in range(rot // 2, 128))


@pytest.mark.parametrize("args", [
    dict(rot=0), dict(rot=3), dict(rot=258), dict(layout=2), dict(base=1.0), dict(base=float("nan")),
    dict(scaling=4), dict(scaling=-1), dict(scaling=1, factor=0.5), dict(scaling=2, factor=float("inf")),
    dict(scaling=3, factor=2.0, context=0.0),
])
def test_rope_plan_refusals(zlib, args):
    kw = dict(rot=64, layout=0, base=10000.0, scaling=0, factor=1.0, context=0.0) | args
    with pytest.raises(zlib.ZeroError) as e:
        zlib.zero_rope_plan(kw.pop("rot"), **kw)
    assert e.value.code == zlib.ZERO_EINVAL


def _drop(zlib, **over):
    d = zlib.ZeroDropout.make(0.1, seed=1)
    for k, v in over.items():
        setattr(d, k, v)
    return d


BAD_DROPS = [(dict(p=-0.1), -1), (dict(p=1.5), -1), (dict(p=float("nan")), -1), (dict(reserved=1), -1),
             (dict(step=1 << 32), -3), (dict(step_ptr=FAKE + 4), -2)]


@pytest.mark.parametrize("over,code", [
    (dict(m=-1), -1), (dict(n=-1), -1), (dict(k=-1), -1), (dict(x=None), -1), (dict(w=None), -1), (dict(y=None), -1),
    (dict(ldx=15), -1), (dict(ldw=15), -1), (dict(ldy=31), -1), (dict(residual=FAKE, ldr=31), -1),
    (dict(pre=FAKE, ldp=31), -1), (dict(act=5), -1), (dict(act=-1), -1), (dict(dt=2), -1),
    (dict(x=FAKE + 1), -2), (dict(y=FAKE + 1), -2), (dict(y=FAKE + 2, dt=1), -2), (dict(bias=FAKE + 1), -2),
    (dict(m=1 << 40, ldx=1 << 40), -3), (dict(m=0, x=None, y=None), 0), (dict(n=0, w=None, y=None), 0),
])
def test_linear_argument_checks(zlib, over, code):
    a = dict(m=8, n=32, k=16, x=FAKE, ldx=16, w=FAKE, ldw=16, bias=None, act=0, drop=None, residual=None, ldr=32,
             pre=None, ldp=32, y=FAKE, dt=0, ldy=32, stream=None) | over
    assert zlib.load().zero_linear(*a.values()) == code


@pytest.mark.parametrize("over,code", BAD_DROPS)
def test_dropout_block_checks(zlib, over, code):
    lib, d = zlib.load(), _drop(zlib, **over)
    assert lib.zero_linear(8, 32, 16, FAKE, 16, FAKE, 16, None, 0, d, None, 32, None, 32, FAKE, 0, 32, None) == code
    assert lib.zero_linear_grad_input(8, 32, 16, FAKE, 32, FAKE, 16, 0, d, None, 16, None, 16, FAKE, 0, 16, None) == code
    assert lib.zero_dropout(8, 32, FAKE, 32, 0, d, None, 32, FAKE, 32, None) == code
    assert lib.zero_dropout_grad(8, 32, FAKE, 32, 0, d, 0, None, 32, FAKE, 0, 32, None, None, 0, None) == code


def test_dropout_rows_past_the_counter(zlib):
    lib, d = zlib.load(), _drop(zlib)
    assert lib.zero_dropout((1 << 32) + 1, 1, FAKE, 1, 0, d, None, 1, FAKE, 1, None) == -3


@pytest.mark.parametrize("over,code", [
    (dict(m=-1), -1), (dict(dz=None), -1), (dict(w=None), -1), (dict(dx=None), -1), (dict(lddz=31), -1),
    (dict(ldw=15), -1), (dict(lddx=15), -1), (dict(act=1), -1), (dict(pre=FAKE), -1), (dict(act=7), -1),
    (dict(dt=3), -1), (dict(dz=FAKE + 1), -2), (dict(act=1, pre=FAKE + 1), -2), (dict(k=0, dx=None), 0),
])
def test_linear_grad_input_argument_checks(zlib, over, code):
    a = dict(m=8, n=32, k=16, dz=FAKE, lddz=32, w=FAKE, ldw=16, act=0, drop=None, pre=None, ldp=16, residual=None,
             ldr=16, dx=FAKE, dt=0, lddx=16, stream=None) | over
    assert zlib.load().zero_linear_grad_input(*a.values()) == code


@pytest.mark.parametrize("over,code", [
    (dict(n=-1), -1), (dict(dz=None), -1), (dict(x=None), -1), (dict(dw=None), -1), (dict(lddz=31), -1),
    (dict(ldx=15), -1), (dict(lddw=15), -1), (dict(acc=FAKE, ldacc=15), -1), (dict(db_acc=FAKE), -1), (dict(dt=2), -1),
    (dict(dw=FAKE + 2, dt=1), -2), (dict(db=FAKE + 1), -2), (dict(db=FAKE, db_acc=FAKE + 1), -2), (dict(n=0, dw=None), 0),
])
def test_linear_grad_weight_argument_checks(zlib, over, code):
    a = dict(m=8, n=32, k=16, dz=FAKE, lddz=32, x=FAKE, ldx=16, acc=None, ldacc=16, dw=FAKE, dt=0, lddw=16,
             db_acc=None, db=None, stream=None) | over
    assert zlib.load().zero_linear_grad_weight(*a.values()) == code


@pytest.mark.parametrize("over,code", [
    (dict(rows=-1), -1), (dict(x=None), -1), (dict(y=None), -1), (dict(ldx=31), -1), (dict(ldy=31), -1),
    (dict(res=FAKE, ldr=31), -1), (dict(dt=2), -1), (dict(x=FAKE + 1), -2), (dict(rows=0, x=None, y=None), 0),
])
def test_dropout_argument_checks(zlib, over, code):
    a = dict(rows=8, cols=32, x=FAKE, ldx=32, dt=0, drop=None, res=None, ldr=32, y=FAKE, ldy=32, stream=None) | over
    assert zlib.load().zero_dropout(*a.values()) == code


@pytest.mark.parametrize("over,code", [
    (dict(rows=-1), -1), (dict(dy=None), -1), (dict(dx=None), -1), (dict(act=1), -1), (dict(pre=FAKE), -1),
    (dict(act=9, pre=FAKE), -1), (dict(db_acc=FAKE), -1), (dict(db=FAKE, bdt=4), -1), (dict(lddx=31), -1),
    (dict(db=FAKE + 2, bdt=1), -2), (dict(dx=FAKE + 1), -2), (dict(cols=0), 0), (dict(rows=0, dy=None, dx=None), 0),
])
def test_dropout_grad_argument_checks(zlib, over, code):
    a = dict(rows=8, cols=32, dy=FAKE, lddy=32, dt=0, drop=None, act=0, pre=None, ldp=32, dx=FAKE, xdt=0, lddx=32,
             db_acc=None, db=None, bdt=0, stream=None) | over
    assert zlib.load().zero_dropout_grad(*a.values()) == code


@pytest.mark.parametrize("over,code", [
    (dict(plan=None), -1), (dict(tokens=-1), -1), (dict(heads=-1), -1), (dict(dim=63), -1), (dict(x=None), -1),
    (dict(y=None), -1), (dict(dt=2), -1), (dict(inverse=2), -1), (dict(xt=-1), -1), (dict(yh=63), -1), (dict(yt=255), -1),
    (dict(x=FAKE, y=FAKE, yt=512), -1), (dict(xt=1 << 60), -3), (dict(x=FAKE + 1), -2), (dict(pos=FAKE + 4), -2),
    (dict(tokens=0), 0), (dict(heads=0, x=None), 0),
])
def test_rope_argument_checks(zlib, over, code):
    plan = zlib.zero_rope_plan(64)
    a = dict(plan=plan, tokens=8, heads=4, dim=64, x=FAKE, xt=256, xh=64, y=FAKE + 4096, yt=256, yh=64, dt=0, pos=None,
             pos0=0, inverse=0, stream=None) | over
    assert zlib.load().zero_rope(*a.values()) == code


def test_rope_hand_made_plan_is_refused(zlib):
    for field, value in (("rot", 0), ("rot", 65), ("rot", 512), ("layout", 2), ("scale", float("inf"))):
        plan = zlib.zero_rope_plan(64)
        setattr(plan, field, value)
        assert zlib.load().zero_rope(plan, 8, 4, 1024, FAKE, 4096, 1024, FAKE, 4096, 1024, 0, None, 0, 0, None) == -1


def test_binding_refusals(zlib):
    """Host tensors, wrong shapes and blocks out of range are refused in Python."""
    x, w, y = torch.zeros(4, 8, dtype=torch.bfloat16), torch.zeros(6, 8, dtype=torch.bfloat16), torch.zeros(4, 6, dtype=torch.bfloat16)
    with pytest.raises(ValueError):
        zlib.zero_linear(x, w, y)
    with pytest.raises(ValueError):
        zlib.zero_linear(x[0], w, y)
    with pytest.raises(ValueError):
        zlib.zero_dropout(x, x, None)
    with pytest.raises(ValueError):
        zlib.zero_rope(zlib.zero_rope_plan(8), x, x)
    for bad in (dict(seed=-1), dict(seed=1 << 64), dict(site=1 << 32), dict(step=-1), dict(step=1 << 32)):
        with pytest.raises(ValueError):
            zlib.ZeroDropout.make(0.1, **bad)
    assert ctypes.sizeof(zlib.ZeroDropout) == 40 and ctypes.sizeof(zlib.ZeroRopePlan) == 16 + 8 * 128
    assert np.dtype(np.uint64).itemsize == 8
