"""What the norms' and the orthogonalised step's calls refuse, on the CPU: the library's
objects over a runtime without a device (as in test_error_state), in which a valid call
succeeds, so that every refusal is the call's own, and a refused call launches nothing."""
import ctypes

import pytest

from tests.test_error_state import A, B, C, fake  # noqa: F401  (a fixture)

OK, EINVAL, EALIGN, ERANGE, ECUDA = 0, -1, -2, -3, -4
D, E, F, G = 4 << 20, 5 << 20, 6 << 20, 7 << 20
NAMES = ("zero_layer_norm", "zero_layer_norm_grad", "zero_layer_norm_grad_workspace", "zero_reduce_scatter_momentum", "zero_muon_update",
         "zero_orthogonalize", "zero_orthogonalize_workspace")
INF, NAN = float("inf"), float("nan")


@pytest.fixture(scope="module")
def lib(zlib, fake):  # noqa: F811
    for name in NAMES:
        getattr(fake, name).argtypes = getattr(zlib.load(), name).argtypes
    return fake


def norm(lib, rows=9, cols=40, x=A, ldx=40, dtype=0, residual=None, ldr=40, sum=None, lds=40, gamma=B, beta=B, eps=1e-5, y=C, y_dtype=0,
         ldy=40, mean=D, rstd=E):
    return lib.zero_layer_norm(rows, cols, x, ldx, dtype, residual, ldr, sum, lds, gamma, beta, eps, y, y_dtype, ldy, mean, rstd, None)


def grad(lib, rows=9, cols=40, dy=A, lddy=40, dy_dtype=0, x=B, ldx=40, mean=D, rstd=E, gamma=C, residual=None, ldr=40, dx=F, dtype=0,
         lddx=40, dgamma_acc=None, dgamma=G, dbeta_acc=None, dbeta=G + 4096, wtype=1, ws=G + 8192, size=1 << 20):
    return lib.zero_layer_norm_grad(rows, cols, dy, lddy, dy_dtype, x, ldx, mean, rstd, gamma, residual, ldr, dx, dtype, lddx,
                                    dgamma_acc, dgamma, dbeta_acc, dbeta, wtype, ws, size, None)


def orth(lib, batch=2, rows=40, cols=72, x=A, xs=2880, ldx=72, dtype=0, y=B, ys=2880, ldy=72, steps=5, co=(3.0, -4.0, 2.0), eps=1e-7,
         ws=C, size=1 << 30):
    c = None if co is None else (ctypes.c_float * 3)(*co)
    return lib.zero_orthogonalize(batch, rows, cols, x, xs, ldx, dtype, y, ys, ldy, steps, c, eps, ws, size, None)


def momentum(lib, zlib, n_src=2, src=A, dtype=0, base=0, div=2.0, r0=0, r1=2, begin=0, end=128, m=B, u=C, mode=0, reserved=0, nesterov=1,
             hp=True, **kw):
    L = zlib.zero_layout([128], 2)
    h = zlib.ZeroMuon.make(**kw)
    h.reserved, h.nesterov = reserved, nesterov
    srcs = (ctypes.c_void_p * max(1, n_src))(*[src] * max(1, n_src))
    return lib.zero_reduce_scatter_momentum(ctypes.byref(L), srcs, n_src, dtype, base, div, r0, r1, begin, end, m, u, mode,
                                            ctypes.byref(h) if hp else None, None)


def update(lib, zlib, o=A, base=0, r0=0, r1=2, begin=0, end=128, w=B, out=C, mode=0, hp=True, **kw):
    L = zlib.zero_layout([128], 2)
    h = zlib.ZeroMuon.make(**kw)
    return lib.zero_muon_update(ctypes.byref(L), o, base, r0, r1, begin, end, w, out, mode, ctypes.byref(h) if hp else None, None)


def check(lib, call, want, **kw):
    before = lib.fake_launches()
    assert call(**kw) == want, kw
    assert (lib.fake_launches() > before) == (want == OK and kw.get("launches", True)), kw


@pytest.mark.parametrize("kw,want", [
    ({}, OK), ({"residual": F, "sum": F}, OK), ({"gamma": None, "beta": None, "mean": None, "rstd": None}, OK), ({"dtype": 1, "y_dtype": 1}, OK),
    ({"dtype": 1}, OK), ({"eps": 0.0}, OK), ({"x": A + 2, "ldx": 41}, OK), ({"cols": 30000, "ldx": 30000, "ldy": 30000}, OK),
    ({"rows": -1}, EINVAL), ({"cols": -1}, EINVAL), ({"dtype": 2}, EINVAL), ({"dtype": -1}, EINVAL), ({"y_dtype": 1}, EINVAL), ({"y_dtype": 7}, EINVAL),
    ({"eps": -1e-9}, EINVAL), ({"eps": NAN}, EINVAL), ({"eps": INF}, EINVAL), ({"residual": F}, EINVAL), ({"sum": F}, EINVAL),
    ({"ldx": 39}, EINVAL), ({"ldy": 39}, EINVAL), ({"residual": F, "sum": F, "ldr": 39}, EINVAL), ({"residual": F, "sum": F, "lds": 1}, EINVAL),
    ({"x": None}, EINVAL), ({"y": None}, EINVAL), ({"x": A + 1}, EALIGN), ({"y": C + 1}, EALIGN), ({"dtype": 1, "x": A + 2}, EALIGN),
    ({"gamma": B + 1}, EALIGN), ({"beta": B + 1}, EALIGN), ({"mean": D + 2}, EALIGN), ({"rstd": E + 1}, EALIGN),
    ({"cols": 1 << 30, "ldx": 1 << 30, "ldy": 1 << 30}, ERANGE), ({"rows": 1 << 60}, ERANGE),
])
def test_layer_norm(lib, kw, want):
    check(lib, lambda **k: norm(lib, **k), want, **kw)


@pytest.mark.parametrize("kw,want", [
    ({}, OK), ({"residual": F}, OK), ({"dgamma": None}, OK), ({"dgamma": None, "dbeta": None, "ws": None, "size": 0, "wtype": 9}, OK),
    ({"dtype": 1}, OK), ({"dtype": 1, "dy_dtype": 1}, OK), ({"rows": 0, "ws": None, "size": 0}, OK), ({"cols": 20000, "ldx": 20000, "lddy": 20000, "lddx": 20000, "size": 1 << 24}, OK),
    ({"rows": -1}, EINVAL), ({"cols": -5}, EINVAL), ({"dtype": 3}, EINVAL), ({"dy_dtype": 1}, EINVAL), ({"dtype": 1, "dy_dtype": 2}, EINVAL),
    ({"wtype": 2}, EINVAL), ({"mean": None}, EINVAL), ({"rstd": None}, EINVAL), ({"dgamma": None, "dgamma_acc": G}, EINVAL),
    ({"dbeta": None, "dbeta_acc": G}, EINVAL), ({"dy": None}, EINVAL), ({"x": None}, EINVAL), ({"dx": None}, EINVAL), ({"lddx": 3}, EINVAL),
    ({"ldx": 39}, EINVAL), ({"lddy": 0}, EINVAL), ({"residual": F, "ldr": 8}, EINVAL), ({"ws": None}, EINVAL), ({"size": 0}, ERANGE), ({"size": 9 * 40 * 8 - 1, "rows": 100000}, ERANGE),
    ({"ws": G + 8}, EALIGN), ({"dy": A + 1}, EALIGN), ({"dx": F + 1}, EALIGN), ({"mean": D + 1}, EALIGN), ({"gamma": C + 1}, EALIGN),
    ({"dgamma": G + 2}, EALIGN), ({"dbeta_acc": G + 1}, EALIGN), ({"cols": 1 << 30}, ERANGE),
])
def test_layer_norm_grad(lib, kw, want):
    check(lib, lambda **k: grad(lib, **k), want, **kw)


@pytest.mark.parametrize("kw,want", [
    ({}, OK), ({"dtype": 1}, OK), ({"xs": 0}, OK), ({"y": A}, OK), ({"eps": 0.0}, OK), ({"batch": 1, "xs": -5, "ys": 0}, OK), ({"rows": 300, "xs": 21600, "ys": 21600}, OK),
    ({"x": A + 2, "ldx": 73, "xs": 9999}, OK), ({"ldy": 144, "ys": 72}, OK), ({"ldy": 143, "ys": 72}, EINVAL), ({"ldy": 144, "ys": 71}, EINVAL),
    ({"ys": -1}, EINVAL),
    ({"batch": -1}, EINVAL), ({"rows": -1}, EINVAL), ({"cols": -1}, EINVAL), ({"dtype": 2}, EINVAL), ({"steps": 0}, EINVAL), ({"steps": 101}, EINVAL),
    ({"co": None}, EINVAL), ({"co": (1.0, NAN, 0.0)}, EINVAL), ({"co": (INF, 1.0, 0.0)}, EINVAL), ({"eps": -1.0}, EINVAL), ({"eps": NAN}, EINVAL),
    ({"x": None}, EINVAL), ({"y": None}, EINVAL), ({"ws": None}, EINVAL), ({"ldx": 71}, EINVAL), ({"ldy": 71}, EINVAL), ({"xs": -1}, EINVAL),
    ({"ys": 2879}, EINVAL), ({"x": A + 1}, EALIGN), ({"y": B + 1}, EALIGN), ({"dtype": 1, "x": A + 2}, EALIGN), ({"ws": C + 64}, EALIGN),
    ({"size": 1000}, ERANGE), ({"batch": 70000}, ERANGE), ({"rows": 40000, "cols": 40000, "ldx": 40000, "ldy": 40000, "batch": 1}, ERANGE),
    ({"rows": 1 << 31, "batch": 1}, ERANGE), ({"xs": 1 << 62}, ERANGE),
])
def test_orthogonalize(lib, kw, want):
    check(lib, lambda **k: orth(lib, **k), want, **kw)


def test_nothing_to_do_launches_nothing(lib):
    before = lib.fake_launches()
    assert norm(lib, rows=0, x=None, y=None) == OK and norm(lib, cols=0, ldx=0, ldy=0, x=None, y=None) == OK
    assert grad(lib, cols=0, ldx=0, lddy=0, lddx=0) == OK and grad(lib, rows=0, dgamma=None, dbeta=None) == OK
    for kw in ({"batch": 0}, {"rows": 0}, {"cols": 0}):
        assert orth(lib, x=None, y=None, ws=None, size=0, **kw) == OK
    assert lib.fake_launches() == before


@pytest.mark.parametrize("kw,want", [
    ({}, OK), ({"dtype": 1}, OK), ({"mode": 1, "r0": 1, "begin": 64}, OK), ({"base": 64, "begin": 64}, OK), ({"src": A + 2, "begin": 3}, OK),
    ({"n_src": 0}, EINVAL), ({"n_src": 65}, ERANGE), ({"src": None}, EINVAL), ({"dtype": 2}, EINVAL), ({"base": 1}, EINVAL), ({"base": -1}, EINVAL),
    ({"div": 0.0}, EINVAL), ({"div": NAN}, EINVAL), ({"div": -2.0}, EINVAL), ({"r0": 2}, EINVAL), ({"r1": 3}, EINVAL), ({"end": 129}, EINVAL),
    ({"begin": 60, "r0": 1}, EINVAL), ({"m": None}, EINVAL), ({"u": None}, EINVAL), ({"mode": 2}, EINVAL), ({"mode": -1}, EINVAL), ({"hp": False}, EINVAL),
    ({"momentum": 1.0}, EINVAL), ({"momentum": -0.1}, EINVAL), ({"momentum": NAN}, EINVAL), ({"lr": INF}, EINVAL), ({"weight_decay": NAN}, EINVAL),
    ({"scale": INF}, EINVAL), ({"reserved": 1}, EINVAL), ({"nesterov": 2}, EINVAL), ({"src": A + 1}, EALIGN), ({"dtype": 1, "src": A + 2}, EALIGN),
    ({"m": B + 2}, EALIGN), ({"u": C + 1}, EALIGN),
])
def test_momentum(lib, zlib, kw, want):
    check(lib, lambda **k: momentum(lib, zlib, **k), want, **kw)


@pytest.mark.parametrize("kw,want", [
    ({}, OK), ({"mode": 1, "r0": 1, "begin": 70}, OK), ({"base": 5, "begin": 5}, OK), ({"o": None}, EINVAL), ({"base": 1}, EINVAL), ({"base": -3}, EINVAL),
    ({"w": None}, EINVAL), ({"out": None}, EINVAL), ({"mode": 5}, EINVAL), ({"hp": False}, EINVAL), ({"lr": NAN}, EINVAL), ({"weight_decay": INF}, EINVAL),
    ({"end": 1000}, EINVAL), ({"o": A + 1}, EALIGN), ({"w": B + 1}, EALIGN), ({"out": C + 1}, EALIGN),
])
def test_update(lib, zlib, kw, want):
    check(lib, lambda **k: update(lib, zlib, **k), want, **kw)


def test_empty_ranges(lib, zlib):
    before = lib.fake_launches()
    assert momentum(lib, zlib, begin=7, end=7) == OK and update(lib, zlib, begin=7, end=7) == OK
    assert lib.fake_launches() == before


def test_workspaces(lib):
    n = ctypes.c_int64(-1)
    for call, args in ((lib.zero_orthogonalize_workspace, (0, 5, 5)), (lib.zero_orthogonalize_workspace, (1, 0, 5)),
                       (lib.zero_layer_norm_grad_workspace, (0, 5)), (lib.zero_layer_norm_grad_workspace, (5, 0))):
        assert call(*args, ctypes.byref(n)) == OK and n.value == 0
    assert lib.zero_orthogonalize_workspace(3, 100, 200, ctypes.byref(n)) == OK
    assert n.value >= 3 * (100 * 200 * 8 + 100 * 100 * 4)
    assert lib.zero_layer_norm_grad_workspace(1000, 100, ctypes.byref(n)) == OK and n.value % (100 * 8) == 0 and n.value > 0
    for args in ((-1, 5, 5), (1, -5, 5), (1, 5, -5)):
        assert lib.zero_orthogonalize_workspace(*args, ctypes.byref(n)) == EINVAL
    assert lib.zero_orthogonalize_workspace(1, 5, 5, None) == EINVAL and lib.zero_layer_norm_grad_workspace(5, 5, None) == EINVAL
    assert lib.zero_orthogonalize_workspace(1, 40000, 40000, ctypes.byref(n)) == ERANGE
    assert lib.zero_orthogonalize_workspace(1 << 58, 4000, 4000, ctypes.byref(n)) == ERANGE
    assert lib.zero_layer_norm_grad_workspace(5, 1 << 40, ctypes.byref(n)) == ERANGE and lib.zero_layer_norm_grad_workspace(-5, 5, ctypes.byref(n)) == EINVAL


CALLS = {"norm": lambda lib, z: norm(lib), "norm gradient": lambda lib, z: grad(lib), "wide norm gradient": lambda lib, z: grad(lib, cols=12000, ldx=12000, lddy=12000, lddx=12000, size=1 << 26),
         "orthogonalize": lambda lib, z: orth(lib, rows=300, xs=21600, ys=21600), "small orthogonalize": lambda lib, z: orth(lib),
         "momentum": momentum, "update": update}


@pytest.mark.parametrize("call", CALLS)
@pytest.mark.parametrize("failing", ["cudaGetDevice", "cudaPointerGetAttributes", "cudaFuncSetAttribute", "cudaOccupancyMaxActiveClusters",
                                     "cudaOccupancyMaxActiveBlocksPerMultiprocessor", "cudaDeviceGetAttribute", "cudaLaunchKernelExC"])
def test_a_failed_runtime_call_leaves_no_error_behind(lib, zlib, call, failing):
    """As for the dense operators: a call that succeeds all the same leaves no error, one
    that fails says so by its code, once, and the next stands on its own."""
    run = CALLS[call]
    for nth in range(1, 12):
        lib.fake_fail(failing.encode(), nth)
        rc = run(lib, zlib)
        hit = lib.fake_seen() >= nth
        lib.fake_fail(b"", 0)
        assert lib.zero_status_check(None) == OK, (call, failing, nth, rc)
        assert rc == OK if not hit else rc in (OK, EINVAL, ECUDA)
        assert run(lib, zlib) == OK
        if not hit:
            break


def test_binding_checks(zlib):
    """What the binding itself refuses before any call (CPU tensors never reach the library)."""
    import torch
    x = torch.zeros(4, 8, dtype=torch.bfloat16)
    with pytest.raises(ValueError, match="CUDA"):
        zlib.zero_layer_norm(x, x)
    with pytest.raises(ValueError, match="matrix"):
        zlib.zero_layer_norm(x[0], x[0])
    with pytest.raises(ValueError, match="CUDA"):
        zlib.zero_orthogonalize(x, x)
    with pytest.raises(ValueError, match="batch"):
        zlib.zero_orthogonalize(x[0], x[0])
    with pytest.raises(ValueError, match="CUDA"):
        zlib.zero_muon_update(zlib.zero_layout([8], 1), x, 0, 0, 1, 0, 8, x.float(), x, 0, zlib.ZeroMuon.make())
