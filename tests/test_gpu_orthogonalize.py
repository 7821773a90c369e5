"""zero_orthogonalize against the iteration in 64 bits: one element to several tiles,
wide, tall and square, sizes off every grid, batches, strides and starts, both types,
faint and strong directions, matrices that are zero, infinite or NaN beside others."""
import pytest
import torch

from tests import dense_plain as dp
from tests import norm_plain as npl

pytestmark = pytest.mark.gpu
BF, F32 = torch.bfloat16, torch.float32


def _close(y, x, steps=5, coefficients=npl.NS, eps=1e-7):
    """Against the iteration with the library's roundings, its sums in 64 bits
    (test_norm_plain holds that against the exact one).  The kernel's fp32 sums are off by
    up to 7e-8 for every 64 elements, 2e-6 here, so that in up to 0.5 % of the cases an
    operand is rounded to the other side: by a whole step, where the rounding itself costs
    half of one at most and sqrt(1/12) by mean square.  By norm that is up to
    sqrt(0.005 * 12) = a quarter of what the roundings cost together; of one element, where
    one such operand may be the largest, up to twice the most that they cost.  Then bf16:
    2^-8 at most, 2^-8 / sqrt 3 by norm."""
    x64 = x.double().cuda()
    ref = npl.orthogonalize_rounded(x64, steps, coefficients, eps, x.dtype == F32).cpu()
    cost = (ref - npl.orthogonalize(x64, steps, coefficients, eps).cpu()).abs().amax((-2, -1), keepdim=True)
    y = y.cpu().double()
    off = (y - ref).abs() - 2.0 ** -8 * ref.abs() - 2 * cost - 1e-300
    assert float(off.max()) <= 0, (int((off > 0).sum()), float(off.max()), float(cost.max()))
    norm = (y - ref).norm(dim=(-2, -1)) / (ref.norm(dim=(-2, -1)) + 1e-300)
    assert float(norm.max()) < 6.3e-4 + 2.0 ** -8 / 3 ** 0.5, norm


def _run(zlib, x, **kw):
    b, rows, cols = x.shape if x.dim() == 3 else (1, *x.shape)
    y = torch.full(x.shape, dp.SENTINEL, dtype=BF, device="cuda")
    need = zlib.zero_orthogonalize_workspace(b, rows, cols)
    ws = torch.full((need + 128,), 0xFF, dtype=torch.uint8, device="cuda")   # NaN on entry
    zlib.zero_orthogonalize(x, y, workspace=ws[:need], **kw)
    assert bool((ws[need:] == 0xFF).all())
    return y


def _x(shape, dtype=BF, seed=0, kind="plain"):
    g = torch.Generator().manual_seed(seed)
    x = torch.randn(*shape, generator=g, dtype=torch.float64)
    if kind == "faint":   # a few directions, the rest a thousandth of them
        r = max(1, min(shape[-2:]) // 16)
        x = torch.randn(*shape[:-1], r, generator=g, dtype=torch.float64) @ torch.randn(*shape[:-2], r, shape[-1], generator=g, dtype=torch.float64) + 1e-3 * x
    if kind == "heavy":
        x = x * torch.exp(torch.randn(*shape[:-1], 1, generator=g, dtype=torch.float64))
    return (1e-3 * x).to(dtype)


SHAPES = [
    (1, 1), (1, 7), (9, 1), (2, 2), (5, 3), (16, 16), (8, 200), (31, 33), (64, 64), (64, 257), (70, 64), (128, 128), (127, 129), (130, 70),
    (1, 8192), (3000, 9), (200, 200), (256, 256), (257, 255), (100, 1600), (513, 129), (333, 517), (517, 333), (640, 1000), (1025, 264),
    (512, 2048), (1100, 1100), (777, 1601),
]


@pytest.mark.parametrize("shape", SHAPES)
@pytest.mark.parametrize("dtype", [BF, F32])
def test_one_matrix(zlib, cuda_device, shape, dtype):
    x = _x(shape, dtype, shape[0])
    y = _run(zlib, x.cuda())
    zlib.zero_status_check()
    _close(y, x)


@pytest.mark.parametrize("shape", [(3, 40, 100), (2, 333, 129), (5, 256, 264), (70, 16, 24), (4, 129, 700), (3, 700, 520)])
@pytest.mark.parametrize("kind", ["faint", "heavy"])
def test_batches(zlib, cuda_device, shape, kind):
    x = _x(shape, BF, 3, kind)
    y = _run(zlib, x.cuda())
    _close(y, x)


@pytest.mark.parametrize("shape", [(40, 100), (333, 517), (520, 264), (16, 1024)])
@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("shift,pad", [(0, 8), (1, 0), (3, 5), (8, 16)])
def test_places(zlib, cuda_device, shape, dtype, shift, pad):
    """A batch of views: rows apart, matrices apart, anywhere; what lies between stays."""
    rows, cols = shape
    x = _x((3, rows, cols), dtype, 7)
    ld, stride = cols + pad, (rows + 1) * (cols + pad) + shift

    def place(t, fill, dt):
        buf = torch.full((shift + 3 * stride + 8,), fill, dtype=dt, device="cuda")
        view = buf[shift:].as_strided((3, rows, cols), (stride, ld, 1), shift)
        if t is not None:
            view.copy_(t)
        return view, buf

    xd, _ = place(x, float("nan"), dtype)
    y, buf = place(None, dp.SENTINEL, BF)
    ws = torch.empty(zlib.zero_orthogonalize_workspace(3, rows, cols), dtype=torch.uint8, device="cuda")
    zlib.zero_orthogonalize(xd, y, workspace=ws)
    _close(y, x)
    y.fill_(dp.SENTINEL)
    assert bool((buf == dp.SENTINEL).all())


@pytest.mark.parametrize("shape", [(48, 80), (300, 520), (520, 300)])
def test_in_place(zlib, cuda_device, shape):
    x = _x((2, *shape), BF, 1).cuda()
    y = _run(zlib, x)
    ws = torch.empty(zlib.zero_orthogonalize_workspace(2, *shape), dtype=torch.uint8, device="cuda")
    zlib.zero_orthogonalize(x, x, workspace=ws)
    assert torch.equal(x, y)


@pytest.mark.parametrize("shape", [(64, 11008), (11008, 64), (1, 5000), (17, 4100), (300, 6000), (6003, 301), (512, 2048), (3, 40, 9000), (5, 4999, 33),
                                   (2, 260, 3001)])
@pytest.mark.parametrize("dtype", [BF, F32])
def test_long_axes(zlib, cuda_device, shape, dtype):
    """Few tiles over a long axis, whose sums are formed in parts."""
    x = _x(shape, dtype, 11)
    y = _run(zlib, x.cuda())
    zlib.zero_status_check()
    _close(y, x)
    assert torch.equal(_run(zlib, x.cuda()), y)


@pytest.mark.parametrize("shape", [(48, 80), (270, 131)])
def test_side_by_side(zlib, cuda_device, shape):
    """Matrices that are column blocks of a wider one, orthogonalised one by one, in place too."""
    rows, cols = shape
    x = _x((3, rows, cols), BF, 2).cuda()
    y = _run(zlib, x)
    wide = torch.full((rows, 3 * cols + 5), dp.SENTINEL, dtype=BF, device="cuda")
    blocks = wide[:, :3 * cols].view(rows, 3, cols).transpose(0, 1)
    blocks.copy_(x)
    ws = torch.empty(zlib.zero_orthogonalize_workspace(3, *shape), dtype=torch.uint8, device="cuda")
    zlib.zero_orthogonalize(blocks, blocks, workspace=ws)
    assert torch.equal(blocks, y) and bool((wide[:, 3 * cols:] == dp.SENTINEL).all())


@pytest.mark.parametrize("shape", [(24, 40), (300, 270)])
@pytest.mark.parametrize("steps,coefficients", [(1, (1.5, -0.5, 0.0)), (8, (1.5, -0.5, 0.0)), (3, (2.0, -1.5, 0.5)), (1, npl.NS), (2, npl.NS),
                                                (0, npl.NS)])
def test_steps_and_coefficients(zlib, cuda_device, shape, steps, coefficients):
    x = _x(shape, F32, 2)
    if steps == 0:
        with pytest.raises(zlib.ZeroError):
            _run(zlib, x.cuda(), steps=0)
        return
    y = _run(zlib, x.cuda(), steps=steps, coefficients=coefficients)
    _close(y, x, steps, coefficients)


@pytest.mark.parametrize("dtype,power", [(BF, 100), (BF, -90), (F32, 120), (F32, -110)])
def test_scales(zlib, cuda_device, dtype, power):
    """The iteration sees the matrix over its norm: a power of two changes nothing, also
    where squares leave fp32's range."""
    for shape in ((40, 60), (300, 280)):
        x = _x(shape, dtype, 4).float().to(torch.float64)
        big = (x * 2.0 ** power).to(dtype)
        y = _run(zlib, big.cuda(), eps=0.0)
        _close(y, big, eps=0.0)


@pytest.mark.parametrize("shape", [(20, 30), (300, 270)])
def test_zeros_and_not_finite(zlib, cuda_device, shape):
    x = _x((5, *shape), F32, 5)
    clean = _run(zlib, x.cuda())
    x[1], x[2, 3, 4], x[3, 0, 0] = 0.0, float("nan"), float("inf")
    for eps in (1e-7, 0.0):
        y = _run(zlib, x.cuda(), eps=eps)
        assert bool((y[1] == 0).all()) and bool(torch.isnan(y[2]).all()) and bool(torch.isnan(y[3]).all())
        if eps:
            assert torch.equal(y[0], clean[0]) and torch.equal(y[4], clean[4])


def test_eps_against_a_faint_matrix(zlib, cuda_device):
    """A norm far below eps: X starts near zero and grows by a (3.4445) a step."""
    x = (_x((30, 50), F32, 6) * 1e-9)
    y = _run(zlib, x.cuda())
    _close(y, x)


def test_empty(zlib, cuda_device):
    for shape in ((0, 4, 4), (2, 0, 5), (2, 5, 0)):
        x = torch.empty(shape, dtype=BF, device="cuda")
        zlib.zero_orthogonalize(x, torch.empty_like(x))


def test_repeats_and_streams(zlib, cuda_device):
    """Two calls at once, each with its workspace, and one captured and replayed."""
    x = [_x((2, 300, 400), BF, i).cuda() for i in range(2)]
    ref = [_run(zlib, t) for t in x]
    need = zlib.zero_orthogonalize_workspace(2, 300, 400)
    ws = [torch.empty(need, dtype=torch.uint8, device="cuda") for _ in range(2)]
    streams = [torch.cuda.Stream() for _ in range(2)]
    torch.cuda.synchronize()
    ys = [[torch.empty_like(t) for _ in range(6)] for t in x]
    for i in range(6):
        for t, w, s, y in zip(x, ws, streams, ys):
            with torch.cuda.stream(s):
                zlib.zero_orthogonalize(t, y[i], workspace=w)
    torch.cuda.synchronize()
    for y, r in zip(ys, ref):
        assert all(torch.equal(t, r) for t in y)
    graph, inp, out = torch.cuda.CUDAGraph(), x[0].clone(), torch.empty_like(x[0])
    with torch.cuda.graph(graph):
        zlib.zero_orthogonalize(inp, out, workspace=ws[0])
    for i in (1, 0, 1):
        inp.copy_(x[i])
        graph.replay()
        assert torch.equal(out, ref[i])
    zlib.zero_status_check()
