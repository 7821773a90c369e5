"""zero_layer_norm and zero_layer_norm_grad against their 64-bit statement: every team
(part of a warp, a warp, a CTA, several passes), both types, rows off the 16-byte grid,
weights anywhere, one row and none, a mean far from the deviations, NaN in one row."""
import pytest
import torch

from tests import dense_plain as dp
from tests import norm_plain as npl

pytestmark = pytest.mark.gpu
BF, F32 = torch.bfloat16, torch.float32

# A row's sums take at most 64 additions one after the other (32 values of a thread, five
# exchanges, 16 warps and the like; 100 for the widest rows here), each off by 2^-24 of the
# sum of magnitudes, and the root, the division and the end a few more.
STEP = 2.0 ** -17

SHAPES = [  # rows, cols
    (1, 1), (3, 2), (5, 7), (1, 8), (9, 8), (70, 16), (33, 24), (1, 64), (257, 65), (19, 200), (1000, 256), (7, 257), (2, 511), (300, 512),
    (1, 520), (45, 1023), (1, 1600), (333, 1600), (1300, 1600), (77, 1601), (5, 4096), (700, 4097), (3, 4104), (31, 6401), (1, 8192),
    (40, 8200), (200, 11008), (2, 16384), (3, 16391), (5, 16392), (2, 33000),
    (1, 1601), (152, 2049), (153, 2049), (400, 2050), (305, 6401), (1, 8191), (460, 4099),   # rows of a CTA from one on, off the grid
]


def _inputs(rows, cols, dtype, seed, far=0.0):
    g = torch.Generator().manual_seed(seed)

    def normal(*shape, std=1.0, dt=dtype):
        return (torch.randn(*shape, generator=g) * std).to(dt)

    x = (torch.randn(rows, cols, generator=g) + far + 0.5 * torch.randn(rows, 1, generator=g)).to(dtype)
    return x, normal(rows, cols, std=2.0), 1 + normal(cols, std=0.3, dt=BF), normal(cols, std=0.3, dt=BF), normal(rows, cols, dt=BF)


def _weights(t, shift):
    buf = torch.full((t.numel() + shift + 8,), float("nan"), dtype=t.dtype, device="cuda")
    view = buf[shift:shift + t.numel()]
    view.copy_(t)
    return view


def _check_forward(zlib, x, res, gamma, beta, out, lds=(None,) * 4, shifts=(0,) * 5, eps=1e-5):
    rows, cols = x.shape
    xd, _ = dp.inside(x, lds[0], shifts[0])
    y, y_ok = dp.blank(rows, cols, out, lds[1], shifts[1])
    stat = torch.full((2, rows + 2), dp.SENTINEL, device="cuda")
    kw, s_ok = {}, None
    if res is not None:
        rd, _ = dp.inside(res, lds[2], shifts[2])
        s, s_ok = dp.blank(rows, cols, x.dtype, lds[3], shifts[3])
        kw = {"residual": rd, "sum": s}
    zlib.zero_layer_norm(xd, y, gamma=None if gamma is None else _weights(gamma, shifts[4]),
                         beta=None if beta is None else _weights(beta, shifts[4]), eps=eps,
                         mean=stat[0, 1:rows + 1], rstd=stat[1, 1:rows + 1], **kw)
    h = x.double()
    if res is not None:
        exact = h + res.double()
        # one fp32 addition, then the type's rounding
        dp.close(s, exact, (dp.eps_out(x.dtype) + 2.0 ** -23) * exact.abs(), "sum")
        assert s_ok()
        h = s.cpu().double()   # what is normalised is the sum as kept
    ref, mean, rstd, xhat = npl.layer_norm(h, None if gamma is None else gamma.double(), None if beta is None else beta.double(), eps)
    g = torch.ones(cols).double() if gamma is None else gamma.double().abs()
    b = torch.zeros(cols).double() if beta is None else beta.double().abs()
    dp.close(y, ref, STEP * (xhat.abs() + 1) * g + 2.0 ** -23 * b + dp.eps_out(out) * ref.abs(), "y")
    dev = (h - mean[:, None]).abs().mean(1)
    dp.close(stat[0, 1:rows + 1], mean, 2.0 ** -23 * mean.abs() + STEP * dev, "mean")
    dp.close(stat[1, 1:rows + 1], rstd, STEP * rstd, "rstd")
    assert y_ok() and bool((stat[:, [0, rows + 1]] == dp.SENTINEL).all())


@pytest.mark.parametrize("shape", SHAPES)
@pytest.mark.parametrize("dtype,out", [(BF, BF), (F32, F32), (F32, BF)])
def test_forward(zlib, cuda_device, shape, dtype, out):
    x, res, gamma, beta, _ = _inputs(*shape, dtype, shape[0] + shape[1])
    _check_forward(zlib, x, res if shape[1] % 2 else None, gamma, beta, out)


@pytest.mark.parametrize("shape", [(1, 5), (37, 96), (129, 1600), (41, 1601), (6, 6401), (9, 8192), (2, 17000)])
@pytest.mark.parametrize("dtype,out", [(BF, BF), (F32, F32), (F32, BF)])
def test_forward_places(zlib, cuda_device, shape, dtype, out):
    """Strides and starts that differ from tensor to tensor, with and without the weights."""
    x, res, gamma, beta, _ = _inputs(*shape, dtype, 5)
    c = shape[1]
    _check_forward(zlib, x, res, gamma, beta, out, (c + 8, c + 16, c, c + 24), (0, 8, 16, 8, 3))
    _check_forward(zlib, x, res, None, None, out, (c + 3, c, c + 1, c + 5), (1, 0, 3, 2, 0))
    _check_forward(zlib, x, None, gamma, None, out, (c, c + 2, None, None), (8, 1, 0, 0, 8))
    _check_forward(zlib, x, None, None, beta, out, (c + 8, c + 8, None, None), (0, 0, 0, 0, 1))


@pytest.mark.parametrize("cols", [40, 1600, 5000])
@pytest.mark.parametrize("far", [1000.0, -30000.0])
def test_forward_far_mean(zlib, cuda_device, cols, far):
    """Deviations of about 1 around a mean of 30000: the mean's own rounding costs nothing."""
    x, _, gamma, beta, _ = _inputs(50, cols, F32, 9, far)
    _check_forward(zlib, x, None, gamma, beta, F32)


def test_forward_special_rows(zlib, cuda_device):
    x, _, gamma, beta, _ = _inputs(6, 1600, F32, 2)
    clean = x.clone()
    x[1, 7], x[2, 1599], x[3] = float("nan"), float("inf"), 4.25
    y, ref = torch.empty(6, 1600, device="cuda"), torch.empty(6, 1600, device="cuda")
    rstd = torch.empty(6, device="cuda")
    zlib.zero_layer_norm(x.cuda(), y, gamma.cuda(), beta.cuda(), eps=1e-5, rstd=rstd)
    zlib.zero_layer_norm(clean.cuda(), ref, gamma.cuda(), beta.cuda(), eps=1e-5)
    assert bool(torch.isnan(y[1:3]).all())
    for r in (0, 4, 5):   # neighbours of such rows are as without them
        assert torch.equal(y[r], ref[r])
    # a row of one value: no deviation, rstd of eps alone, y = beta
    assert torch.equal(y[3].cpu(), beta.float())
    assert abs(float(rstd[3]) * 1e-5 ** 0.5 - 1) < 1e-5


@pytest.mark.parametrize("cols", [3, 24, 57, 513, 1601, 6400, 17001])
@pytest.mark.parametrize("value", [3.3e10, -7.1e13, 1e17])
@pytest.mark.parametrize("out", [BF, F32])
def test_forward_rows_of_one_large_value(zlib, cuda_device, cols, value, out):
    """No deviation: rounding must not make the variance negative.  The number that stands
    for the mean at first is off by at most 2^-17 of the value (64 additions and the
    share), what corrects it by 2^-17 of that, and eps alone makes rstd at most eps^-1/2."""
    x = torch.full((3, cols), value, device="cuda")
    x[1] = 1.0
    y, stat = torch.empty(3, cols, dtype=out, device="cuda"), torch.empty(2, 3, device="cuda")
    zlib.zero_layer_norm(x, y, eps=1e-5, mean=stat[0], rstd=stat[1])
    assert bool((y.double().abs() <= 2.0 ** -34 * x.double().abs() * 1.01e-5 ** -0.5).all())
    assert bool((stat[1] <= 1.001 * 1e-5 ** -0.5).all()) and bool((stat[1] > 0).all())
    dp.close(stat[0].cpu(), x[:, 0].cpu().double(), 2.0 ** -23 * x[:, 0].cpu().double().abs(), "mean")


@pytest.mark.parametrize("shape", [(70, 16), (257, 65), (333, 1600), (77, 1601), (31, 6401), (3, 16391), (5, 16392), (9, 20001)])
@pytest.mark.parametrize("dtype", [BF, F32])
def test_in_place(zlib, cuda_device, shape, dtype):
    """y over x; dx over dy, over x and over the residual: as beside them."""
    x, res, gamma, beta, dy = (t.cuda() for t in _inputs(*shape, dtype, 6))
    dy = dy.to(dtype)
    y, dx = torch.empty_like(x), torch.empty_like(x)
    mean, rstd = torch.empty(shape[0], device="cuda"), torch.empty(shape[0], device="cuda")
    ws = torch.empty(zlib.zero_layer_norm_grad_workspace(*shape), dtype=torch.uint8, device="cuda")
    zlib.zero_layer_norm(x, y, gamma, beta, mean=mean, rstd=rstd)
    over = x.clone()
    zlib.zero_layer_norm(over, over, gamma, beta)
    assert torch.equal(over, y)

    def grads(dy, x, res, dx):
        dg, db = torch.empty(shape[1], device="cuda"), torch.empty(shape[1], device="cuda")
        zlib.zero_layer_norm_grad(dy, x, mean, rstd, dx, gamma, residual=res, dgamma=dg, dbeta=db, workspace=ws)
        return dx, dg, db

    want = grads(dy, x, res, dx)
    for i in range(3):
        args = [t.clone() for t in (dy, x, res)]
        assert all(torch.equal(a, b) for a, b in zip(grads(*args, args[i]), want)), i


def test_forward_in_place_sum(zlib, cuda_device):
    x, res, gamma, beta, _ = (t.cuda() for t in _inputs(120, 1600, BF, 4))
    for cols in (1600, 40):
        a, b = x[:, :cols].clone(memory_format=torch.contiguous_format), res[:, :cols].clone(memory_format=torch.contiguous_format)
        s, y, y2 = (torch.empty_like(a) for _ in range(3))
        zlib.zero_layer_norm(a, y, gamma[:cols], beta[:cols], residual=b, sum=s)
        zlib.zero_layer_norm(a, y2, gamma[:cols], beta[:cols], residual=b, sum=b)
        assert torch.equal(s, b) and torch.equal(y, y2)
        b = res[:, :cols].clone(memory_format=torch.contiguous_format)
        zlib.zero_layer_norm(a, y2, gamma[:cols], beta[:cols], residual=b, sum=a)
        assert torch.equal(s, a) and torch.equal(y, y2)


def _check_grad(zlib, x, dy, res, gamma, wtype, acc=False, lds=(None,) * 4, shifts=(0,) * 5, which=(True, True), in_place=False):
    rows, cols = x.shape
    g = torch.Generator().manual_seed(cols)
    h = x.double()
    _, mean, rstd, _ = npl.layer_norm(h, None, None, 1e-5)
    mean, rstd = mean.float(), rstd.float()
    xd, _ = dp.inside(x, lds[0], shifts[0])
    dyd, _ = dp.inside(dy, lds[1], shifts[1])
    dx, dx_ok = dp.blank(rows, cols, x.dtype, lds[2], shifts[2])
    rd = None if res is None else dp.inside(res, lds[3], shifts[3])[0]
    accs = [torch.randn(cols, generator=g).to(wtype) if acc else None for _ in range(2)]
    bufs = [torch.full((cols + shifts[4] + 3,), dp.SENTINEL, dtype=wtype, device="cuda") for _ in range(2)]
    outs = [b[shifts[4]:shifts[4] + cols] for b in bufs]
    given = [None if a is None else a.cuda() for a in accs]
    if in_place:
        for i in range(2):
            outs[i].copy_(accs[i])
            given[i] = outs[i]
    ws = torch.full((zlib.zero_layer_norm_grad_workspace(rows, cols) + 64,), 0xFF, dtype=torch.uint8, device="cuda")   # NaN on entry
    zlib.zero_layer_norm_grad(dyd, xd, mean.cuda(), rstd.cuda(), dx, gamma=None if gamma is None else _weights(gamma, shifts[4]),
                              residual=rd, dgamma=outs[0] if which[0] else None, dbeta=outs[1] if which[1] else None,
                              dgamma_acc=given[0] if which[0] else None, dbeta_acc=given[1] if which[1] else None,
                              workspace=ws[:-64] if any(which) else None)
    rdx, rdg, rdb, mag, mg, mb = npl.layer_norm_grad(dy.double(), h, mean.double(), rstd.double(), None if gamma is None else gamma.double())
    add = 0.0 if res is None else res.double()
    rdx = rdx + add
    dp.close(dx, rdx, STEP * mag + 2.0 ** -23 * (rdx.abs() + (res.double().abs() if res is not None else 0.0)) + dp.eps_out(x.dtype) * rdx.abs(), "dx")
    assert dx_ok()
    # a column's sum: at most all rows one after the other, each term off by a few 2^-24
    for out, ref, m, a, buf, asked in zip(outs, (rdg, rdb), (mg, mb), accs, bufs, which):
        if not asked:
            assert bool((buf == dp.SENTINEL).all())
            continue
        if a is not None:
            ref, m = ref + a.double(), m + a.double().abs()
        dp.close(out, ref, (rows + 64) * 2.0 ** -24 * m + dp.eps_out(wtype) * ref.abs(), "weights")
        keep = out.clone()
        out.fill_(dp.SENTINEL)
        assert bool((buf == dp.SENTINEL).all())
        out.copy_(keep)
    if any(which):
        assert bool((ws[-64:] == 0xFF).all())


@pytest.mark.parametrize("shape", SHAPES)
@pytest.mark.parametrize("dtype,dy_dtype,wtype", [(BF, BF, BF), (F32, BF, F32), (F32, F32, BF)])
def test_grad(zlib, cuda_device, shape, dtype, dy_dtype, wtype):
    x, res, gamma, _, dy = _inputs(*shape, dtype, shape[0] * 3 + shape[1])
    _check_grad(zlib, x, dy.to(dy_dtype), res if shape[0] % 2 else None, gamma, wtype, acc=shape[1] % 3 == 1)


@pytest.mark.parametrize("shape", [(1, 5), (37, 96), (129, 1600), (41, 1601), (6, 6401), (9, 12000), (3, 17000)])
@pytest.mark.parametrize("dtype,dy_dtype", [(BF, BF), (F32, BF), (F32, F32)])
def test_grad_places(zlib, cuda_device, shape, dtype, dy_dtype):
    x, res, gamma, _, dy = _inputs(*shape, dtype, 6)
    dy, c = dy.to(dy_dtype), shape[1]
    _check_grad(zlib, x, dy, res, gamma, BF, True, (c + 8, c + 16, c, c + 24), (0, 8, 16, 8, 3))
    _check_grad(zlib, x, dy, res, gamma, F32, False, (c + 3, c, c + 1, c + 5), (1, 0, 3, 2, 8))
    _check_grad(zlib, x, dy, None, None, F32, True, (c, c + 8, c, None), (0, 8, 0, 0, 1), in_place=True)
    _check_grad(zlib, x, dy, None, gamma, BF, which=(True, False))
    _check_grad(zlib, x, dy, None, gamma, BF, which=(False, True))
    _check_grad(zlib, x, dy, None, gamma, BF, which=(False, False))


def test_grad_dx_is_the_residual(zlib, cuda_device):
    x, res, gamma, _, dy = (t.cuda() for t in _inputs(200, 1600, BF, 8))
    _, mean, rstd, _ = npl.layer_norm(x.double(), None, None, 1e-5)
    mean, rstd, dx = mean.float(), rstd.float(), torch.empty_like(x)
    zlib.zero_layer_norm_grad(dy, x, mean, rstd, dx, gamma, residual=res)
    zlib.zero_layer_norm_grad(dy, x, mean, rstd, res, gamma, residual=res)
    assert torch.equal(dx, res)


@pytest.mark.parametrize("cols", [16, 1600, 20000])
def test_no_rows(zlib, cuda_device, cols):
    """The weights' gradients of no rows are what they are added to, or 0; nothing else is touched."""
    empty = torch.empty(0, cols, dtype=BF, device="cuda")
    none = torch.empty(0, device="cuda")
    dg, db, acc = torch.full((cols,), 7.0, device="cuda"), torch.full((cols,), 7.0, device="cuda"), torch.randn(cols, device="cuda")
    zlib.zero_layer_norm(empty, empty.clone())
    zlib.zero_layer_norm_grad(empty, empty, none, none, empty.clone(), dgamma=dg, dbeta=db, dbeta_acc=acc)
    assert bool((dg == 0).all()) and torch.equal(db, acc)
    zlib.zero_layer_norm_grad(empty, empty, none, none, empty.clone())


def test_no_columns(zlib, cuda_device):
    empty, v = torch.empty(5, 0, dtype=BF, device="cuda"), torch.full((5,), 3.0, device="cuda")
    zlib.zero_layer_norm(empty, empty.clone(), mean=v, rstd=v.clone())
    zlib.zero_layer_norm_grad(empty, empty, v, v, empty.clone(), dgamma=torch.empty(0, device="cuda"))
    assert bool((v == 3.0).all())


@pytest.mark.parametrize("shape", [(3000, 48), (2000, 1600), (300, 9000)])
def test_repeats(zlib, cuda_device, shape):
    x, res, gamma, beta, dy = (t.cuda() for t in _inputs(*shape, BF, 8))
    _, mean, rstd, _ = npl.layer_norm(x.double(), None, None, 1e-5)
    ws = torch.empty(zlib.zero_layer_norm_grad_workspace(*shape), dtype=torch.uint8, device="cuda")
    first = None
    for _ in range(4):
        out = [torch.empty_like(x), torch.empty(shape[1], device="cuda"), torch.empty(shape[1], device="cuda")]
        zlib.zero_layer_norm_grad(dy, x, mean.float(), rstd.float(), out[0], gamma, dgamma=out[1], dbeta=out[2], workspace=ws)
        first = first or out
        assert all(torch.equal(a, b) for a, b in zip(out, first))


def test_gradient_of_the_forward_call(zlib, cuda_device):
    """The gradient's calls against differences of the forward call's 64-bit statement,
    on what the forward call itself kept."""
    x, res, gamma, beta, dy = _inputs(12, 72, F32, 3)
    g = torch.Generator().manual_seed(1)
    s, y = torch.empty(12, 72, device="cuda"), torch.empty(12, 72, device="cuda")
    mean, rstd = torch.empty(12, device="cuda"), torch.empty(12, device="cuda")
    zlib.zero_layer_norm(x.cuda(), y, gamma.cuda(), beta.cuda(), residual=res.cuda(), sum=s, mean=mean, rstd=rstd)
    dx, dg, db = torch.empty(12, 72, device="cuda"), torch.empty(72, device="cuda"), torch.empty(72, device="cuda")
    ws = torch.empty(zlib.zero_layer_norm_grad_workspace(12, 72), dtype=torch.uint8, device="cuda")
    zlib.zero_layer_norm_grad(dy.cuda(), s, mean, rstd, dx, gamma.cuda(), dgamma=dg, dbeta=db, workspace=ws)
    base = [s.cpu().double(), gamma.double(), beta.double()]
    step = 1e-5
    for at, grad in enumerate((dx, dg, db)):
        way = torch.randn(base[at].shape, generator=g, dtype=torch.float64)
        ends = []
        for sign in (1, -1):
            args = list(base)
            args[at] = args[at] + sign * step * way
            ends.append((npl.layer_norm(*args, 1e-5)[0] * dy.double()).sum())
        diff = float(ends[0] - ends[1]) / (2 * step)
        got = float((grad.cpu().double() * way).sum())
        # the difference: third derivatives times step^2 and 2^-52 / step; the call: STEP of the terms
        assert abs(diff - got) <= 1e-6 * float((grad.cpu().double().abs() * way.abs()).sum()) * 10 + 1e-6
