"""zero_dropout and zero_dropout_grad against their 64-bit statement."""
import pytest
import torch

from tests import dense_plain as dp

pytestmark = pytest.mark.gpu
BF, F32 = torch.bfloat16, torch.float32
SIZES = [(1, 1), (1, 8), (1, 5003), (7, 9), (65, 64), (333, 1600), (1025, 257), (3, 40001), (5000, 3)]
PLACES = [(0, 0), (8, 8), (1, 0), (0, 1), (5, 3), (4, 4)]


def _mat(g, rows, cols, dtype=BF, std=1.0):
    return (torch.randn(rows, cols, generator=g, dtype=torch.float64) * std).to(dtype)


@pytest.mark.parametrize("size", SIZES)
@pytest.mark.parametrize("place", PLACES)
@pytest.mark.parametrize("dtype", [BF, F32])
def test_dropout(zlib, cuda_device, size, place, dtype):
    rows, cols = size
    g = torch.Generator().manual_seed(rows + cols)
    for p, residual in [(0.1, False), (0.5, True), (0.0, True), (1.0, False)]:
        x, r = _mat(g, rows, cols, dtype), _mat(g, rows, cols, dtype)
        y, ok = dp.blank(rows, cols, dtype, cols + place[0], place[1])
        drop = zlib.ZeroDropout.make(p, seed=(1 << 63) + 5, site=4000000000, step=(1 << 32) - 1)
        zlib.zero_dropout(dp.inside(x, cols + place[0], place[1])[0], y, drop,
                          residual=dp.inside(r, cols + place[0], place[1])[0] if residual else None)
        f = dp.factor(rows, cols, p, (1 << 63) + 5, 4000000000, (1 << 32) - 1)
        ref = x.double() * f + (r.double() if residual else 0.0)
        # the product and the sum each rounded to fp32, then stored
        tol = 2.0 ** -23 * (x.double().abs() * f + ref.abs()) + dp.eps_out(dtype) * ref.abs()
        dp.close(y, ref, tol + 1e-30)
        if not residual:   # what is dropped is exactly 0, what is kept is not
            assert torch.equal(y.cpu() != 0, (x.double() * f) != 0)
        assert ok()


def test_dropped_elements_are_zero_whatever_they_held(zlib, cuda_device):
    x = torch.full((64, 96), float("nan"), dtype=BF, device="cuda")
    x[:, ::2] = float("inf")
    y = torch.empty_like(x)
    for p in (0.5, 1.0):
        zlib.zero_dropout(x, y, zlib.ZeroDropout.make(p, seed=3))
        f = dp.factor(64, 96, p, 3)
        got = y.cpu()
        assert bool((got[f == 0] == 0).all()) and not bool(torch.isfinite(got[f != 0]).any())
        zlib.zero_dropout_grad(x, y, zlib.ZeroDropout.make(p, seed=3))
        assert bool((y.cpu()[f == 0] == 0).all())


def test_no_dropout_copies(zlib, cuda_device):
    x = torch.randn(40, 33, device="cuda").to(BF)
    for drop in (None, zlib.ZeroDropout.make(0.0), zlib.ZeroDropout.make(2.0 ** -18)):
        y = torch.empty_like(x)
        zlib.zero_dropout(x, y, drop)
        assert torch.equal(x, y)


@pytest.mark.parametrize("size", SIZES)
@pytest.mark.parametrize("place", PLACES)
def test_dropout_grad_with_slope_and_sums(zlib, cuda_device, size, place):
    rows, cols = size
    g = torch.Generator().manual_seed(rows * 3 + cols)
    for act, p, dt, xt, bt, acc in [(dp.NONE, 0.3, BF, BF, F32, False), (dp.GELU_TANH, 0.1, BF, BF, BF, True),
                                    (dp.RELU, 0.0, F32, BF, F32, True), (dp.SILU, 0.5, F32, F32, BF, False),
                                    (dp.GELU, 0.0, BF, F32, F32, False)]:
        dy, z, a = _mat(g, rows, cols, dt), _mat(g, rows, cols), _mat(g, 1, cols, bt)
        dx, ok = dp.blank(rows, cols, xt, cols + place[0], place[1])
        db, b_ok = dp.blank(1, cols, bt, cols, place[1])
        zlib.zero_dropout_grad(dp.inside(dy, cols + place[0], place[1])[0], dx, zlib.ZeroDropout.make(p, seed=8) if p else None,
                               act=act, pre=dp.inside(z, cols + place[0], place[1])[0] if act else None, db=db[0],
                               db_acc=dp.inside(a, cols, place[1])[0][0] if acc else None)
        zlib.zero_status_check()
        f = dp.factor(rows, cols, p, 8)
        s = dp.slope(z.double(), act)
        ref = dy.double() * s * f
        t = (2.0 ** -17 * (dy.double().abs() * f) if act else 0.0) + 2.0 ** -22 * ref.abs()   # slope forms, products
        dp.close(dx, ref, t + dp.eps_out(xt) * ref.abs() + 1e-30, "dx")
        sums = ref.sum(0, keepdim=True) + (a.double() if acc else 0.0)
        mag = ref.abs().sum(0, keepdim=True) + (a.double().abs() if acc else 0.0)
        off = t.sum(0, keepdim=True) if isinstance(t, torch.Tensor) else 0.0
        dp.close(db, sums, dp.tol_product(mag, rows, off) + dp.eps_out(bt) * sums.abs(), "db")
        assert ok() and b_ok()


@pytest.mark.parametrize("size", [(1025, 264), (2049, 1600), (600, 4800), (5000, 24), (129, 6400), (1100, 32)])
def test_sums_of_aligned_rows(zlib, cuda_device, size):
    """Every share of rows and width of a warp that the sums are split by."""
    test_dropout_grad_with_slope_and_sums(zlib, cuda_device, size, (8, 8))


@pytest.mark.parametrize("shape", [(300, 520), (77, 41)])
def test_dropout_grad_in_place_and_repeatable(zlib, cuda_device, shape):
    g = torch.Generator().manual_seed(4)
    dy, z = _mat(g, *shape).cuda(), _mat(g, *shape).cuda()
    drop = zlib.ZeroDropout.make(0.2, seed=2)
    out, db = torch.empty_like(dy), torch.empty(shape[1], device="cuda")
    zlib.zero_dropout_grad(dy, out, drop, act=dp.GELU, pre=z, db=db)
    for _ in range(4):
        same, sb = dy.clone(), torch.empty_like(db)
        zlib.zero_dropout_grad(same, same, drop, act=dp.GELU, pre=z, db=sb)
        assert torch.equal(out, same) and torch.equal(db, sb)


def test_extreme_pre_activations(zlib, cuda_device):
    """Slopes at infinities and the type's largest values are 0 or 1, not NaN; a
    NaN gives NaN where the slope is smooth."""
    big = float(torch.finfo(BF).max)
    z = torch.tensor([[big, -big, float("inf"), float("-inf"), 1e20, -1e20, 100.0, -100.0]], dtype=BF, device="cuda")
    one = torch.ones_like(z)
    dx = torch.empty_like(z)
    for act in (dp.RELU, dp.GELU, dp.GELU_TANH, dp.SILU):
        zlib.zero_dropout_grad(one, dx, act=act, pre=z)
        assert torch.equal(dx.cpu().abs(), torch.tensor([[1, 0, 1, 0, 1, 0, 1, 0]], dtype=BF)), act
    z.fill_(float("nan"))
    for act in (dp.GELU, dp.GELU_TANH, dp.SILU):
        zlib.zero_dropout_grad(one, dx, act=act, pre=z)
        assert bool(torch.isnan(dx).all())


def test_rows_of_no_gradient(zlib, cuda_device):
    dy = torch.empty(0, 40, dtype=BF, device="cuda")
    db, a = torch.full((40,), 5.0, device="cuda"), torch.randn(40, device="cuda")
    zlib.zero_dropout_grad(dy, torch.empty_like(dy), db=db)
    assert float(db.abs().max()) == 0
    zlib.zero_dropout_grad(dy, torch.empty_like(dy), db=db, db_acc=a)
    assert torch.equal(db, a)


def test_linear_epilogue_drops_the_same_elements(zlib, cuda_device):
    x = torch.randn(50, 64, device="cuda").to(BF)
    w = torch.randn(72, 64, device="cuda").to(BF)
    drop = zlib.ZeroDropout.make(0.4, seed=77, site=1, step=2)
    fused, plain, apart = (torch.empty(50, 72, device="cuda") for _ in range(3))
    zlib.zero_linear(x, w, fused, drop=drop)
    zlib.zero_linear(x, w, plain)
    zlib.zero_dropout(plain, apart, drop)
    assert torch.equal(fused, apart)


@pytest.mark.slow
def test_offsets_past_32_bits(zlib, cuda_device):
    rows, cols, ld = 70, 100, 1 << 26
    big = torch.empty(rows * ld, dtype=BF, device="cuda").view(rows, ld)
    x = torch.randn(rows, cols, device="cuda").to(BF)
    big[:, :cols].copy_(x)
    drop = zlib.ZeroDropout.make(0.3, seed=1)
    ref = torch.empty_like(x)
    zlib.zero_dropout(x, ref, drop)
    zlib.zero_dropout(big[:, :cols], big[:, 128:128 + cols], drop)
    assert torch.equal(big[:, 128:128 + cols], ref)


def test_refusals(zlib, cuda_device):
    x = torch.zeros(4, 8, dtype=BF, device="cuda")
    with pytest.raises(TypeError):
        zlib.zero_dropout(x, x.float(), None)
    with pytest.raises(TypeError):
        zlib.zero_dropout(x.half(), x.half(), None)
    with pytest.raises(ValueError):
        zlib.zero_dropout(x, x[:2], None)
    with pytest.raises(ValueError):
        zlib.zero_dropout(x[:1].expand(4, 8), x, None)
    with pytest.raises(ValueError):
        zlib.zero_dropout_grad(x, x, db=torch.zeros(7, device="cuda"))
    with pytest.raises(zlib.ZeroError):
        zlib.zero_dropout_grad(x, x, act=dp.RELU)
    host = torch.zeros(1, dtype=torch.int64)
    with pytest.raises(ValueError):
        zlib.ZeroDropout.make(0.5, step_ptr=host)
