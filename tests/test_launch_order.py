"""The dense operators' kernels are launched before their predecessors have ended and
wait inside (await_predecessor).  Data that a predecessor writes is not read-only for
such a kernel's lifetime, so none of its loads may take the read-only path
(ld.global.nc: __ldg, or a pointer promised with __restrict__), which may return a
stale line and which the compiler may move above the wait."""
import os
import re

import pytest

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "zero_sharded_mixed_gb300", "csrc")


def _code(name):
    """A source without its comments."""
    with open(os.path.join(CSRC, name)) as f:
        return re.sub(r"//[^\n]*|/\*.*?\*/", "", f.read(), flags=re.S)


def _dense_files():
    """Every source that launches or waits so, and the headers of these operators alone."""
    waits = [n for n in sorted(os.listdir(CSRC)) if re.search(r"\bawait_predecessor\(|\blaunch_dense\(", _code(n))]
    return sorted({*waits, "zero_dense.cuh", "zero_product.cuh", "zero_tensor.cuh"})


def test_the_files_are_found():
    assert {"zero_linear.cu", "zero_rows.cu", "zero_dropout.cu", "zero_rope.cu"} <= set(_dense_files())


@pytest.mark.parametrize("name", _dense_files())
def test_no_load_takes_the_read_only_path(name):
    # ld_stream_*: the step kernels' loads, which a build option turns into __ldg
    found = re.findall(r"__ldg\b|\bld\.global(?:\.\w+)*\.nc\b|__restrict__|\bld_stream_\w+", _code(name))
    assert not found, (name, sorted(set(found)))
