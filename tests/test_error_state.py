"""What a failed runtime call leaves behind.  The library's own objects are linked
over a runtime without a device (tests/c/fake_cudart.c) in which one chosen call
fails, so no GPU is needed and none sees a fault.  A dense operator whose call
succeeds all the same (another kernel took it) has to leave no error for
zero_status_check to blame on it, and one that fails reports that by its code,
once, and the next call stands on its own."""
import ctypes
import os
import shutil
import subprocess

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
A, B, C = 1 << 20, 2 << 20, 3 << 20   # never dereferenced


@pytest.fixture(scope="module")
def fake(zlib, tmp_path_factory):
    from zero_sharded_mixed_gb300 import build
    out = str(tmp_path_factory.mktemp("fake") / "libfake.so")
    cuda = os.path.dirname(os.path.dirname(shutil.which("nvcc") or "/usr/local/cuda/bin/nvcc"))
    own = [os.path.join(build.BUILD, os.path.splitext(n)[0] + ".o") for n in build.CUDA_SOURCES + build.HOST_SOURCES]
    obj = out[:-3] + ".o"
    subprocess.check_call(["gcc", "-O1", "-fPIC", "-w", "-I", os.path.join(cuda, "include"), "-c",
                           os.path.join(ROOT, "tests", "c", "fake_cudart.c"), "-o", obj])
    # -Bsymbolic: the objects' runtime calls stay inside, whatever runtime the process has
    subprocess.check_call(["g++", "-shared", "-Wl,-Bsymbolic", "-o", out, obj, *own])
    lib = ctypes.CDLL(out, mode=os.RTLD_LOCAL)
    real = zlib.load()
    for name in ("zero_linear", "zero_linear_grad_input", "zero_linear_grad_weight", "zero_dropout", "zero_dropout_grad", "zero_rope",
                 "zero_status_check"):
        getattr(lib, name).argtypes = getattr(real, name).argtypes
    lib.fake_fail.argtypes = [ctypes.c_char_p, ctypes.c_int]
    return lib


def _calls(zlib):
    plan, drop = zlib.zero_rope_plan(64), zlib.ZeroDropout.make(0.1, seed=1)
    return {
        "linear, few tiles and a long sum": lambda f: f.zero_linear(512, 1600, 6400, A, 6400, B, 6400, None, 0, None, None, 1600, None, 1600, C, 0, 1600, None),
        "linear, fp32": lambda f: f.zero_linear(512, 1600, 6400, A, 6400, B, 6400, None, 0, None, None, 1600, None, 1600, C, 1, 1600, None),
        "linear, one row": lambda f: f.zero_linear(1, 1600, 1600, A, 1600, B, 1600, None, 0, None, None, 1600, None, 1600, C, 0, 1600, None),
        "linear, large": lambda f: f.zero_linear(8192, 6400, 1600, A, 1600, B, 1600, None, 0, None, None, 6400, None, 6400, C, 0, 6400, None),
        "linear, off the grid": lambda f: f.zero_linear(77, 333, 129, A + 2, 129, B, 129, None, 0, None, None, 333, None, 333, C, 0, 333, None),
        "input gradient": lambda f: f.zero_linear_grad_input(512, 6400, 1600, A, 6400, B, 1600, 0, None, None, 1600, None, 1600, C, 0, 1600, None),
        "weight gradient": lambda f: f.zero_linear_grad_weight(8192, 512, 512, A, 512, B, 512, None, 512, C, 1, 512, None, C + (1 << 19), None),
        "dropout": lambda f: f.zero_dropout(333, 1600, A, 1600, 0, drop, None, 1600, B, 1600, None),
        "dropout, off the grid": lambda f: f.zero_dropout(333, 1601, A, 1601, 0, drop, None, 1601, B, 1601, None),
        "dropout gradient": lambda f: f.zero_dropout_grad(333, 1600, A, 1600, 0, drop, 0, None, 1600, B, 0, 1600, None, C, 0, None),
        "rotary": lambda f: f.zero_rope(plan, 8, 4, 64, A, 256, 64, B, 256, 64, 0, None, 0, 0, None),
    }


FAILING = ["cudaGetDevice", "cudaPointerGetAttributes", "cudaFuncSetAttribute", "cudaOccupancyMaxActiveClusters",
           "cudaOccupancyMaxActiveBlocksPerMultiprocessor", "cudaDeviceGetAttribute", "cudaLaunchKernelExC"]
CALLS = ["linear, few tiles and a long sum", "linear, fp32", "linear, one row", "linear, large", "linear, off the grid",
         "input gradient", "weight gradient", "dropout", "dropout, off the grid", "dropout gradient", "rotary"]


def test_the_fake_reports_errors(zlib, fake):
    call = _calls(zlib)["dropout"]
    assert call(fake) == 0 and fake.zero_status_check(None) == 0 and fake.fake_launches() >= 1
    fake.fake_fail(b"cudaStreamSynchronize", 1)
    assert fake.zero_status_check(None) == zlib.ZERO_ECUDA
    assert fake.zero_status_check(None) == 0
    fake.fake_fail(b"cudaLaunchKernelExC", 1)
    assert call(fake) == zlib.ZERO_ECUDA


def _apart(work):
    """work()'s numbers from a process of its own, in which the library keeps what it
    keeps from its first calls anew."""
    r, w = os.pipe()
    pid = os.fork()
    if pid == 0:
        try:
            os.write(w, " ".join(str(v) for v in work()).encode())
        finally:
            os._exit(0)
    os.close(w)
    with os.fdopen(r) as f:
        said = f.read()
    os.waitpid(pid, 0)
    return [int(v) for v in said.split()]


_swept = {}


def _sweep(zlib, fake, call, failing, first):
    """For every call of `failing` that the operator makes, on the library's first call
    or a later one: (which, the operator's answer, what it launched, the status after);
    an answer of None where the process ended.  Asked once for the tests below."""
    key = call, failing, first
    if key in _swept:
        return _swept[key]
    run = _calls(zlib)[call]

    def scenario(nth):
        if not first:
            run(fake)
        fake.fake_fail(failing.encode(), nth)
        before = fake.fake_launches()
        code, seen = run(fake), fake.fake_seen()
        fake.fake_fail(b"", 0)
        return code, seen, fake.fake_launches() - before, fake.zero_status_check(None)

    found = _swept[key] = []
    for nth in range(1, 64):
        code, seen, launched, status = _apart(lambda: scenario(nth)) or (None, nth, 0, 0)
        if seen < nth:
            assert code == 0
            return found
        found.append((nth, code, launched, status))
    raise AssertionError("no end")


@pytest.mark.filterwarnings("ignore:This process:DeprecationWarning")
@pytest.mark.parametrize("first", [True, False], ids=["first call", "later call"])
@pytest.mark.parametrize("failing", FAILING)
@pytest.mark.parametrize("call", CALLS)
def test_a_failed_question_is_answered(zlib, fake, call, failing, first):
    """By a code or by going on without it, and never by the end of the process."""
    for nth, code, launched, _ in _sweep(zlib, fake, call, failing, first):
        assert code in (0, zlib.ZERO_EINVAL, zlib.ZERO_ECUDA), (nth, code)
        assert code != 0 or launched > 0, nth


@pytest.mark.filterwarnings("ignore:This process:DeprecationWarning")
@pytest.mark.parametrize("first", [True, False], ids=["first call", "later call"])
@pytest.mark.parametrize("failing", FAILING)
@pytest.mark.parametrize("call", CALLS)
def test_no_error_is_left_behind(zlib, fake, call, failing, first):
    for nth, code, _, status in _sweep(zlib, fake, call, failing, first):
        assert status == 0, f"call {nth} of {failing} failed, the operator returned {code}, and its error stayed"
