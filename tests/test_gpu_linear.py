"""zero_linear, zero_linear_grad_input and zero_linear_grad_weight against their
64-bit statement: sizes from nothing and one to several tiles with ragged ends,
every operand aligned and at odd places, both result types, each activation,
dropout, residuals and accumulation in place; nothing outside an output is
written and nothing beside an input is read (inputs lie in buffers of NaNs)."""
import math

import pytest
import torch

from tests import dense_plain as dp

pytestmark = pytest.mark.gpu
BF, F32 = torch.bfloat16, torch.float32

# (m, n, k): one element, one row, ragged ends of every tile, several tiles
SIZES = [(1, 1, 1), (1, 64, 64), (1, 1600, 1600), (3, 17, 5), (128, 128, 64), (130, 250, 72), (257, 513, 200),
         (64, 1000, 40), (300, 65, 1031), (5, 4096, 264), (1000, 48, 48), (513, 776, 136), (40, 40, 2600)]
# (row padding, shift) of the operands and of the results, in elements
PLACES = [((0, 0), (0, 0)), ((8, 8), (8, 16)), ((1, 3), (0, 0)), ((0, 0), (1, 1)), ((3, 1), (5, 7)), ((0, 1), (4, 4))]


def _mat(g, rows, cols, std=1.0, dtype=BF):
    return (torch.randn(rows, cols, generator=g, dtype=torch.float64) * std).to(dtype)


def _in(t, place):
    return dp.inside(t, t.shape[1] + place[0], place[1])[0]


def _out(rows, cols, dtype, place):
    return dp.blank(rows, cols, dtype, cols + place[0], place[1])


def _check_linear(zlib, m, n, k, pin=(0, 0), pout=(0, 0), dtype=BF, act=0, p=0.0, bias=True, residual=True, pre=True, seed=0):
    g = torch.Generator().manual_seed(seed * 1000 + m + 3 * n + 7 * k)
    x, w = _mat(g, m, k), _mat(g, n, k, 1 / math.sqrt(k))
    b = _mat(g, 1, n, 0.5) if bias else None
    r = _mat(g, m, n, dtype=dtype) if residual else None
    y, y_ok = _out(m, n, dtype, pout)
    z_out, z_ok = _out(m, n, BF, pout) if pre else (None, lambda: True)
    drop = zlib.ZeroDropout.make(p, seed=seed + 99, site=3, step=12) if p else None
    zlib.zero_linear(_in(x, pin), _in(w, pin), y, bias=None if b is None else _in(b, (0, pin[1]))[0], act=act,
                     residual=None if r is None else _in(r, pout), drop=drop, pre=z_out)
    zlib.zero_status_check()
    xd, wd = x.double(), w.double()
    bd = b.double() if bias else torch.zeros(1, n, dtype=torch.float64)
    z = xd @ wd.t() + bd
    f = dp.factor(m, n, p, seed + 99, 3, 12)
    ref = dp.act(z, act) * f + (r.double() if residual else 0.0)
    tz = dp.tol_product(xd.abs() @ wd.abs().t() + bd.abs(), k)
    # the end: activation error 2^-19, residual addition, storing
    tol = (1.13 * tz + 2.0 ** -19 * z.abs()) * f + 2.0 ** -23 * ref.abs() + dp.eps_out(dtype) * ref.abs() + 1e-30
    dp.close(y, ref, tol, "y")
    if pre:
        dp.close(z_out, z, tz + dp.eps_out(BF) * z.abs(), "pre")
    assert y_ok() and z_ok()


@pytest.mark.parametrize("size", SIZES)
@pytest.mark.parametrize("pin,pout", PLACES)
def test_linear_sizes_and_places(zlib, cuda_device, size, pin, pout):
    _check_linear(zlib, *size, pin, pout, act=dp.GELU_TANH, p=0.1)


@pytest.mark.parametrize("act", dp.ACTS)
@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("p", [0.0, 0.5])
def test_linear_ends(zlib, cuda_device, act, dtype, p):
    for bias, residual, pre in [(True, False, True), (False, True, False), (False, False, False), (True, True, True)]:
        _check_linear(zlib, 133, 200, 96, dtype=dtype, act=act, p=p, bias=bias, residual=residual, pre=pre, seed=act)


@pytest.mark.parametrize("place", PLACES)
@pytest.mark.parametrize("dtype", [BF, F32])
def test_linear_result_types_and_places(zlib, cuda_device, place, dtype):
    _check_linear(zlib, 150, 333, 128, place[0], place[1], dtype=dtype, act=dp.SILU, p=0.25)


def test_linear_drops_everything_or_nothing(zlib, cuda_device):
    _check_linear(zlib, 70, 90, 64, p=1.0)
    _check_linear(zlib, 70, 90, 64, p=2.0 ** -18)


def test_linear_empty_sum(zlib, cuda_device):
    """k = 0: y = residual + act(bias)."""
    g = torch.Generator().manual_seed(1)
    b, r = _mat(g, 1, 70), _mat(g, 5, 70)
    y, ok = _out(5, 70, BF, (0, 0))
    x, w = torch.empty(5, 0, dtype=BF, device="cuda"), torch.empty(70, 0, dtype=BF, device="cuda")
    zlib.zero_linear(x, w, y, bias=b[0].cuda(), act=dp.RELU, residual=r.cuda())
    ref = dp.act(b.double(), dp.RELU) + r.double()
    dp.close(y, ref, 2.0 ** -8 * ref.abs() + 1e-30)
    zlib.zero_linear(x, w, y)
    assert float(y.abs().max()) == 0 and ok()
    zlib.zero_linear(torch.empty(0, 16, dtype=BF, device="cuda"), torch.zeros(70, 16, dtype=BF, device="cuda"),
                     torch.empty(0, 70, dtype=BF, device="cuda"))


def test_linear_residual_in_place(zlib, cuda_device):
    g = torch.Generator().manual_seed(2)
    for m, n, k, dtype in [(200, 320, 64, BF), (33, 77, 50, F32)]:
        x, w, r = _mat(g, m, k), _mat(g, n, k, 0.1), _mat(g, m, n, dtype=dtype)
        y = r.cuda()
        zlib.zero_linear(x.cuda(), w.cuda(), y, residual=y)
        apart = torch.empty(m, n, dtype=dtype, device="cuda")
        zlib.zero_linear(x.cuda(), w.cuda(), apart, residual=r.cuda())
        assert torch.equal(y, apart)


def test_linear_non_finite_rows_stay_apart(zlib, cuda_device):
    """An infinity or NaN in one row of x reaches that row's results alone, and a
    dropped element is 0 whatever it held."""
    g = torch.Generator().manual_seed(3)
    m, n, k = 140, 136, 100
    x, w = _mat(g, m, k), _mat(g, n, k)
    x[5, 7], x[77, 99], x[139, 0] = float("nan"), float("inf"), float("-inf")
    y = torch.empty(m, n, dtype=BF, device="cuda")
    zlib.zero_linear(x.cuda(), w.cuda(), y, drop=zlib.ZeroDropout.make(0.5, seed=4))
    f = dp.factor(m, n, 0.5, seed=4)
    z = x.double() @ w.double().t()
    ref = torch.where(f == 0, torch.zeros_like(z), z * f)
    mag = torch.nan_to_num(x.double().abs(), 0, 0, 0) @ w.double().abs().t()
    dp.close(y, ref, 2 * dp.tol_product(mag, k) + 2.0 ** -8 * torch.nan_to_num(ref.abs(), 0, 0, 0))


def _check_grad_input(zlib, m, n, k, pin=(0, 0), pout=(0, 0), dtype=BF, act=0, p=0.0, residual=True, seed=0):
    g = torch.Generator().manual_seed(seed * 1000 + m + 3 * n + 7 * k + 1)
    dz, w, z = _mat(g, m, n), _mat(g, n, k, 1 / math.sqrt(n)), _mat(g, m, k)
    r = _mat(g, m, k, dtype=dtype) if residual else None
    dx, ok = _out(m, k, dtype, pout)
    drop = zlib.ZeroDropout.make(p, seed=seed + 5, site=1) if p else None
    zlib.zero_linear_grad_input(_in(dz, pin), _in(w, pin), dx, act=act, pre=_in(z, pin) if act else None, drop=drop,
                                residual=None if r is None else _in(r, pout))
    zlib.zero_status_check()
    s = dp.slope(z.double(), act) if act else torch.ones(m, k, dtype=torch.float64)
    f = dp.factor(m, k, p, seed + 5, 1)
    prod = dz.double() @ w.double()
    ref = prod * s * f + (r.double() if residual else 0.0)
    # the slope's own fast forms: 2^-17 absolute (its terms are at most about 2)
    tol = (dp.tol_product(dz.double().abs() @ w.double().abs(), n) * (s.abs() + 2.0 ** -17) + 2.0 ** -17 * prod.abs()) * f
    dp.close(dx, ref, tol + (2.0 ** -23 + dp.eps_out(dtype)) * ref.abs() + 1e-30, "dx")
    assert ok()


@pytest.mark.parametrize("size", SIZES)
@pytest.mark.parametrize("pin,pout", PLACES)
def test_grad_input_sizes_and_places(zlib, cuda_device, size, pin, pout):
    _check_grad_input(zlib, *size, pin, pout, act=dp.SILU, p=0.1)


@pytest.mark.parametrize("act", dp.ACTS)
@pytest.mark.parametrize("dtype", [BF, F32])
def test_grad_input_ends(zlib, cuda_device, act, dtype):
    for p, residual in [(0.0, False), (0.5, False), (0.3, True), (0.0, True)]:
        _check_grad_input(zlib, 133, 96, 200, dtype=dtype, act=act, p=p, residual=residual, seed=act)


# enough tiles of 256 x 256 for the kernel of large products; widths that leave a
# narrow last tile, an unused half tile, rows past one half of a tile
BIG = [(2000, 2100, 96), (257, 10008, 72), (2305, 1600, 200), (2560, 1032, 1600), (300, 5000, 1000)]


@pytest.mark.parametrize("size", BIG)
@pytest.mark.parametrize("places", [((0, 0), (0, 0)), ((8, 16), (3, 1)), ((16, 8), (8, 8))])
@pytest.mark.parametrize("dtype", [BF, F32])
def test_large_products(zlib, cuda_device, size, places, dtype):
    _check_linear(zlib, *size, *places, dtype=dtype, act=dp.GELU_TANH, p=0.1)
    m, n, k = size
    _check_grad_input(zlib, m, k, n, *places, dtype=dtype, act=dp.GELU, p=0.1)
    _check_grad_weight(zlib, k, m, n, *places, dtype=dtype)


def _check_grad_weight(zlib, m, n, k, pin=(0, 0), pout=(0, 0), dtype=BF, acc=True, db=True, db_acc=True, seed=0):
    g = torch.Generator().manual_seed(seed * 1000 + m + 3 * n + 7 * k + 2)
    dz, x = _mat(g, m, n), _mat(g, m, k, 1 / math.sqrt(m))
    a = _mat(g, n, k, dtype=dtype) if acc else None
    ba = _mat(g, 1, n, dtype=dtype) if db_acc and db else None
    dw, w_ok = _out(n, k, dtype, pout)
    b, b_ok = _out(1, n, dtype, (0, pout[1])) if db else (None, lambda: True)
    zlib.zero_linear_grad_weight(_in(dz, pin), _in(x, pin), dw, db=None if b is None else b[0],
                                 acc=None if a is None else _in(a, pout), db_acc=None if ba is None else _in(ba, (0, pout[1]))[0])
    zlib.zero_status_check()
    ref = dz.double().t() @ x.double() + (a.double() if acc else 0.0)
    mag = dz.double().abs().t() @ x.double().abs() + (a.double().abs() if acc else 0.0)
    dp.close(dw, ref, dp.tol_product(mag, m) + dp.eps_out(dtype) * ref.abs(), "dw")
    if db:
        rb = dz.double().sum(0, keepdim=True) + (ba.double() if ba is not None else 0.0)
        mb = dz.double().abs().sum(0, keepdim=True) + (ba.double().abs() if ba is not None else 0.0)
        dp.close(b, rb, dp.tol_product(mb, m) + dp.eps_out(dtype) * rb.abs(), "db")
    assert w_ok() and b_ok()


@pytest.mark.parametrize("size", SIZES)
@pytest.mark.parametrize("pin,pout", PLACES)
def test_grad_weight_sizes_and_places(zlib, cuda_device, size, pin, pout):
    _check_grad_weight(zlib, *size, pin, pout)


# few tiles and a long sum, ended inside a block and inside either half of a tile
LONG = [(65, 96, 4096), (129, 250, 4104), (200, 1000, 6400), (257, 136, 5000), (128, 40, 8192), (384, 72, 2056)]


@pytest.mark.parametrize("size", LONG)
@pytest.mark.parametrize("dtype", [BF, F32])
def test_long_sums_of_few_tiles(zlib, cuda_device, size, dtype):
    m, n, k = size
    _check_linear(zlib, m, n, k, (8, 8), (8, 16), dtype=dtype, act=dp.GELU, p=0.1)
    _check_linear(zlib, m, n, k, (0, 0), (1, 3), dtype=dtype, bias=False, pre=False)
    _check_grad_input(zlib, m, k, n, (8, 8), (8, 16), dtype=dtype, act=dp.SILU, p=0.1)
    _check_grad_weight(zlib, k, m, n, (8, 8), (8, 16), dtype=dtype)


@pytest.mark.parametrize("size", [(129, 290, 330), (260, 129, 387), (135, 96, 256), (391, 330, 127)])
@pytest.mark.parametrize("pin", [(1, 3), (0, 5), (7, 0), (2, 6)])
def test_whole_and_partial_tiles_at_odd_places(zlib, cuda_device, size, pin):
    """Unaligned operands of a few whole tiles and stages beside ones that end inside
    a group of eight rows."""
    _check_linear(zlib, *size, pin)
    _check_grad_input(zlib, *size, pin)
    _check_grad_weight(zlib, *size, pin)


@pytest.mark.parametrize("dtype", [BF, F32])
def test_grad_weight_ends(zlib, cuda_device, dtype):
    for acc, db, db_acc in [(False, False, False), (True, False, False), (False, True, False), (False, True, True)]:
        _check_grad_weight(zlib, 300, 136, 200, dtype=dtype, acc=acc, db=db, db_acc=db_acc)


def test_grad_weight_of_no_rows(zlib, cuda_device):
    dz, x = torch.empty(0, 40, dtype=BF, device="cuda"), torch.empty(0, 24, dtype=BF, device="cuda")
    dw, db = torch.full((40, 24), 3.0, device="cuda"), torch.full((40,), 3.0, device="cuda")
    zlib.zero_linear_grad_weight(dz, x, dw, db=db)
    assert float(dw.abs().max()) == 0 and float(db.abs().max()) == 0
    a = torch.randn(40, 24, device="cuda")
    zlib.zero_linear_grad_weight(dz, x, dw, db=db, acc=a, db_acc=a[:, 0].contiguous())
    assert torch.equal(dw, a) and torch.equal(db, a[:, 0])


def test_gradients_accumulate_in_place(zlib, cuda_device):
    """Two micro-batches added to fp32 accumulators in place equal one call per
    micro-batch with separate buffers."""
    g = torch.Generator().manual_seed(8)
    acc, db = torch.zeros(200, 136, device="cuda"), torch.zeros(200, device="cuda")
    ref, rb = acc.clone(), db.clone()
    for _ in range(2):
        dz, x = _mat(g, 70, 200).cuda(), _mat(g, 70, 136).cuda()
        zlib.zero_linear_grad_weight(dz, x, acc, db=db, acc=acc, db_acc=db)
        w2, b2 = torch.empty_like(ref), torch.empty_like(rb)
        zlib.zero_linear_grad_weight(dz, x, w2, db=b2, acc=ref, db_acc=rb)
        ref, rb = w2, b2
        assert torch.equal(acc, ref) and torch.equal(db, rb)


def test_gradients_against_differences(zlib, cuda_device):
    """sum(c * y) differs along random directions of x, w and bias as the gradient
    calls say: the 64-bit function's central differences against them."""
    g = torch.Generator().manual_seed(9)
    m, n, k, act, p = 37, 72, 56, dp.GELU, 0.25
    x, w, b, c = _mat(g, m, k), _mat(g, n, k, 0.2), _mat(g, 1, n, 0.5), _mat(g, m, n)
    drop = zlib.ZeroDropout.make(p, seed=6)
    f = dp.factor(m, n, p, 6)

    def value(xd, wd, bd):
        return float((c.double() * dp.act(xd @ wd.t() + bd, act) * f).sum())

    y, z = (torch.empty(m, n, dtype=BF, device="cuda") for _ in range(2))
    zlib.zero_linear(x.cuda(), w.cuda(), y, bias=b[0].cuda(), act=act, drop=drop, pre=z)
    dz = torch.empty(m, n, dtype=BF, device="cuda")
    db, dw, dx = torch.empty(n, device="cuda"), torch.empty(n, k, device="cuda"), torch.empty(m, k, device="cuda")
    zlib.zero_dropout_grad(c.cuda(), dz, drop=drop, act=act, pre=z, db=db)
    zlib.zero_linear_grad_input(dz, w.cuda(), dx)
    zlib.zero_linear_grad_weight(dz, x.cuda(), dw)
    args = [x.double(), w.double(), b.double()]
    # pre and dz are each rounded to bf16 (2^-8): the slope moves by at most 0.8
    # times that of z, dz by that of itself, each weighed with how far the direction
    # moves its z; fp32 sums and the differences add under a hundredth of it
    z64 = args[0] @ args[1].t() + args[2]
    slack = 2.0 ** -8 * c.double().abs() * f * (1.13 + 0.8 * z64.abs())
    for i, grad in enumerate((dx, dw, db[None])):
        for trial in range(3):
            v = torch.randn(args[i].shape, generator=g, dtype=torch.float64)
            h = 1e-5
            up, down = list(args), list(args)
            up[i], down[i] = args[i] + h * v, args[i] - h * v
            want = (value(*up) - value(*down)) / (2 * h)
            got = float((grad.double().cpu() * v).sum())
            push = (v @ args[1].t() if i == 0 else args[0] @ v.t() if i == 1 else v.expand(m, n)).abs()
            assert abs(got - want) <= 1.01 * float((slack * push).sum()), (i, trial, got, want)


def test_results_repeat_and_streams(zlib, cuda_device):
    """Bit-identical from run to run, and on another stream than the default."""
    g = torch.Generator().manual_seed(10)
    m, n, k = 300, 520, 264
    x, w = _mat(g, m, k).cuda(), _mat(g, n, k).cuda()
    first = None
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    for i in range(6):
        y, dw, db = torch.empty(m, n, device="cuda"), torch.empty(n, k, device="cuda"), torch.empty(n, device="cuda")
        dx = torch.empty(m, k, device="cuda")
        torch.cuda.synchronize()
        s = side if i % 2 else None
        zlib.zero_linear(x, w, y, stream=s)
        dz = torch.randn(m, n, generator=torch.Generator(device="cuda").manual_seed(1), device="cuda").to(BF)
        torch.cuda.synchronize()
        zlib.zero_linear_grad_weight(dz, x, dw, db=db, stream=s)
        zlib.zero_linear_grad_input(dz, w, dx, stream=s)
        torch.cuda.synchronize()
        if first is None:
            first = (y, dw, db, dx)
        assert all(torch.equal(a, b) for a, b in zip(first, (y, dw, db, dx)))


def test_graph_replays_drop_other_elements(zlib, cuda_device):
    """A captured call whose block reads its step from device memory drops, at
    each replay, what a call with that step by value drops."""
    g = torch.Generator().manual_seed(11)
    x, w = _mat(g, 64, 128).cuda(), _mat(g, 96, 128).cuda()
    step = torch.zeros(1, dtype=torch.int64, device="cuda")
    drop = zlib.ZeroDropout.make(0.5, seed=1, step=10, step_ptr=step)
    y = torch.empty(64, 96, dtype=BF, device="cuda")
    zlib.zero_linear(x, w, y, drop=drop)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        zlib.zero_linear(x, w, y, drop=drop)
    for t in (0, 1, 5, 2 ** 32 - 10):
        step.fill_(t)
        graph.replay()
        want = torch.empty_like(y)
        zlib.zero_linear(x, w, want, drop=zlib.ZeroDropout.make(0.5, seed=1, step=(10 + t) % 2 ** 32))
        assert torch.equal(y, want)


def test_strides_of_slices(zlib, cuda_device):
    """Operands that are column slices of wider tensors, and a query/key/value
    projection written into a slice."""
    g = torch.Generator().manual_seed(12)
    wide, w = _mat(g, 96, 256).cuda(), _mat(g, 64, 128).cuda()
    out = torch.zeros(96, 192, dtype=BF, device="cuda")
    zlib.zero_linear(wide[:, 64:192], w, out[:, 64:128])
    ref = torch.empty(96, 64, dtype=BF, device="cuda")
    zlib.zero_linear(wide[:, 64:192].contiguous(), w, ref)
    assert torch.equal(out[:, 64:128], ref)
    assert float(out[:, :64].abs().max()) == 0 and float(out[:, 128:].abs().max()) == 0
    with pytest.raises(ValueError):
        zlib.zero_linear(wide.t()[:128].t()[:, ::2][:, :64], w, ref)
    with pytest.raises(TypeError):
        zlib.zero_linear(wide[:, :128], w.float(), ref)
    with pytest.raises(TypeError):
        zlib.zero_linear(wide[:, :128], w, ref, residual=ref.float())


def test_calls_in_a_row_wait_for_one_another(zlib, cuda_device):
    """Kernels are launched while their predecessors end: chains in which each call
    reads what the last one wrote, through every kernel, equal the same calls with a
    synchronisation after each."""
    g = torch.Generator().manual_seed(14)
    drop = zlib.ZeroDropout.make(0.1, seed=3)
    plan = zlib.zero_rope_plan(64)
    for rows, d in [(2, 320), (96, 320), (700, 1280), (2304, 1280), (77, 333)]:
        w = [_mat(g, d, d, 1 / math.sqrt(d)).cuda() for _ in range(3)]
        x0 = _mat(g, rows, d).cuda()

        def chain(wait):
            x, out = x0.clone(), []
            for i in range(6):
                y, dz = torch.empty_like(x), torch.empty_like(x)
                pre, dx, dw, db = torch.empty_like(x), torch.empty_like(x), torch.empty_like(w[0]), torch.empty(d, dtype=BF, device="cuda")
                for call in (lambda: zlib.zero_linear(x, w[i % 3], y, act=dp.SILU, pre=pre),
                             lambda: zlib.zero_dropout(y, y, drop, residual=x),
                             lambda: zlib.zero_rope(plan, y[:, :320].view(rows, 5, 64), y[:, :320].view(rows, 5, 64)) if d >= 320 and d % 8 == 0 else None,
                             lambda: zlib.zero_dropout_grad(y, dz, drop, act=dp.SILU, pre=pre, db=db),
                             lambda: zlib.zero_linear_grad_input(dz, w[i % 3], dx, residual=dz),
                             lambda: zlib.zero_linear_grad_weight(dz, y, dw, db=db)):
                    call()
                    if wait:
                        torch.cuda.synchronize()
                out += [y, dw, db]
                x = dx
            torch.cuda.synchronize()
            return out + [x]

        want = chain(True)
        for _ in range(3):
            assert all(torch.equal(a, b) for a, b in zip(chain(False), want)), (rows, d)


@pytest.mark.parametrize("rows", [1, 2, 4])
@pytest.mark.parametrize("d", [2048, 5120])
def test_few_wide_rows_in_a_row(zlib, cuda_device, rows, d):
    """One to four rows, as a few new tokens have: each call reads a buffer that the last
    one wrote, over and over the same two, without a synchronisation and in a graph,
    beside the same calls with one after each."""
    g = torch.Generator().manual_seed(19)
    w = [_mat(g, d, d, 1 / math.sqrt(d)).cuda() for _ in range(2)]
    x0 = _mat(g, rows, d).cuda()
    plan, drop = zlib.zero_rope_plan(64), zlib.ZeroDropout.make(0.1, seed=3)
    a, b = torch.empty_like(x0), torch.empty_like(x0)
    kept = torch.empty(24, rows, d, dtype=BF, device="cuda")

    def chain(wait):
        def run(call):
            call()
            if wait:
                torch.cuda.synchronize()

        a.copy_(x0)
        for i in range(12):
            run(lambda: zlib.zero_linear(a, w[i % 2], b, act=dp.SILU, residual=a))
            run(lambda: zlib.zero_rope(plan, b.view(rows, d // 64, 64), b.view(rows, d // 64, 64), pos0=i))
            run(lambda: zlib.zero_linear(b, w[1 - i % 2], a, residual=x0))
            run(lambda: zlib.zero_dropout(a, kept[2 * i], drop, residual=b))
            run(lambda: zlib.zero_dropout(b, kept[2 * i + 1], None))
        torch.cuda.synchronize()
        return kept.clone()

    want = chain(True)
    for _ in range(5):
        assert torch.equal(chain(False), want)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        a.copy_(x0)
        for i in range(12):
            zlib.zero_linear(a, w[i % 2], b, act=dp.SILU, residual=a)
            zlib.zero_rope(plan, b.view(rows, d // 64, 64), b.view(rows, d // 64, 64), pos0=i)
            zlib.zero_linear(b, w[1 - i % 2], a, residual=x0)
            zlib.zero_dropout(a, kept[2 * i], drop, residual=b)
            zlib.zero_dropout(b, kept[2 * i + 1], None)
    for _ in range(5):
        kept.zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(kept, want)


def test_products_on_two_streams(zlib, cuda_device):
    """Large and small products side by side on two streams (they share SMs, shared
    and tensor memory) give what they give alone."""
    g = torch.Generator().manual_seed(15)
    jobs = [(_mat(g, m, k).cuda(), _mat(g, n, k).cuda()) for m, n, k in ((2048, 2048, 512), (64, 1600, 1600), (300, 515, 333), (1500, 1504, 200))]
    want = []
    for x, w in jobs:
        y = torch.empty(x.shape[0], w.shape[0], dtype=BF, device="cuda")
        zlib.zero_linear(x, w, y)
        want.append(y)
    streams = [torch.cuda.Stream() for _ in range(2)]
    torch.cuda.synchronize()
    got = []
    for i in range(40):
        j = i % len(jobs)
        y = torch.empty_like(want[j])
        with torch.cuda.stream(streams[i % 3 % 2]):
            zlib.zero_linear(*jobs[j], y)
        got.append((j, y))
    torch.cuda.synchronize()
    assert all(torch.equal(y, want[j]) for j, y in got)
    zlib.zero_status_check()


def test_captured_products(zlib, cuda_device):
    """Every kind of product captured in a graph and replayed on new inputs."""
    g = torch.Generator().manual_seed(16)
    cases = []
    for m, n, k in ((3, 200, 128), (64, 320, 256), (2304, 1280, 320), (77, 333, 129)):
        x, w = _mat(g, m, k).cuda(), _mat(g, n, k).cuda()
        dz = torch.empty(m, n, dtype=BF, device="cuda")
        cases.append((x, w, dz, torch.empty_like(x), torch.empty(n, k, device="cuda"), torch.empty(n, device="cuda")))

    def run():
        for x, w, y, dx, dw, db in cases:
            zlib.zero_linear(x, w, y)
            zlib.zero_linear_grad_input(y, w, dx)
            zlib.zero_linear_grad_weight(y, x, dw, db=db)

    run()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        run()
    for x, *_ in cases:
        x.copy_(_mat(g, *x.shape))
    graph.replay()
    torch.cuda.synchronize()
    first = [[t.clone() for t in c[2:]] for c in cases]
    run()
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for c, f in zip(cases, first) for a, b in zip(c[2:], f))


def test_long_sums_in_32_bits(zlib, cuda_device):
    """fp32 results stay within 1.2e-6 of the exact ones by norm: runs of at most 13
    blocks of 64 are cut at 2^-24 a step of 16, so at most 52 2^-24 / 2 = 1.5e-6 of a
    sum that grows evenly and two thirds of it, 1.0e-6, of one that wanders; the
    additions of the runs round at 2^-24."""
    g = torch.Generator(device="cuda").manual_seed(17)
    for m, n, k in ((1024, 2048, 4096), (64, 512, 4096), (333, 250, 2050)):
        x, w = (torch.randn(r, k, generator=g, device="cuda").to(BF) for r in (m, n))
        y = torch.empty(m, n, device="cuda")
        zlib.zero_linear(x, w, y)
        ref = x.double() @ w.double().t()
        assert float((y.double() - ref).norm() / ref.norm()) <= 1.2e-6, (m, n, k)


def test_longest_sums_in_32_bits(zlib, cuda_device):
    """The same bound at any depth, of every call that sums, on the 16-byte grid and
    off it: what a run's cut loses goes with the run's own sum, so that the loss of
    the whole stays the fraction of it that a run loses, however many runs there are,
    and their additions, rounded, add 2^-24 times half the root of their number."""
    g = torch.Generator(device="cuda").manual_seed(18)

    def mat(rows, cols):
        return torch.randn(rows, cols, generator=g, device="cuda").to(BF)

    def check(got, ref, what):
        assert float((got.double() - ref).norm() / ref.norm()) <= 1.2e-6, what

    for m, n, k in ((64, 512, 16384), (64, 4096, 11008), (256, 768, 16384), (9, 300, 50257), (333, 250, 9001), (3, 200, 50257)):
        x, w, y = mat(m, k), mat(n, k), torch.empty(m, n, device="cuda")
        zlib.zero_linear(x, w, y)
        check(y, x.double() @ w.double().t(), ("y", m, n, k))
    for m, n, k in ((64, 16384, 512), (100, 50257, 200), (333, 9001, 250)):
        dz, w, dx = mat(m, n), mat(n, k), torch.empty(m, k, device="cuda")
        zlib.zero_linear_grad_input(dz, w, dx)
        check(dx, dz.double() @ w.double(), ("dx", m, n, k))
    for m, n, k in ((65536, 512, 512), (50257, 40, 48), (50257, 41, 47), (9001, 250, 333)):
        dz, x, dw = mat(m, n), mat(m, k), torch.empty(n, k, device="cuda")
        zlib.zero_linear_grad_weight(dz, x, dw)
        check(dw, dz.double().t() @ x.double(), ("dw", m, n, k))


@pytest.mark.slow
def test_offsets_past_32_bits(zlib, cuda_device):
    """Rows whose element offsets pass 2^32, in each operand and result."""
    ld = 1 << 26
    g = torch.Generator().manual_seed(13)
    m, n, k = 80, 72, 64
    big = torch.empty(m * ld, dtype=BF, device="cuda")
    x, w = _mat(g, m, k), _mat(g, n, k)
    view = big.view(m, ld)
    view[:, :k].copy_(x)
    y = torch.empty(m, n, dtype=BF, device="cuda")
    zlib.zero_linear(view[:, :k], w.cuda(), y)
    ref = torch.empty_like(y)
    zlib.zero_linear(x.cuda(), w.cuda(), ref)
    assert torch.equal(y, ref)
    zlib.zero_linear(x.cuda(), w.cuda(), view[:, 512:512 + n])
    assert torch.equal(view[:, 512:512 + n], ref)
    dz = _mat(g, m, n).cuda()
    dw, dref = torch.empty(n, k, device="cuda"), torch.empty(n, k, device="cuda")
    zlib.zero_linear_grad_weight(dz, view[:, :k], dw)
    zlib.zero_linear_grad_weight(dz, x.cuda(), dref)
    assert torch.equal(dw, dref)
