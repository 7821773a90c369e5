"""zero_status_check copies a status word of each kind of kernel that has bounded waits, about
9 us each: those of the layer norm's gradient and of the orthogonalisation only where they
have been called (CPU, over a runtime without a device)."""
import pytest

from tests.test_error_state import _apart, fake  # noqa: F401  (a fixture)
from tests.test_norm_muon_refusals import A, C, F, grad, lib, norm, orth  # noqa: F401  (a fixture)


def _copies(lib):  # noqa: F811
    lib.fake_fail(b"cudaMemcpyFromSymbol", 0)
    assert lib.zero_status_check(None) == 0
    return lib.fake_seen()


@pytest.mark.filterwarnings("ignore:This process:DeprecationWarning")
@pytest.mark.parametrize("calls,copies", [
    ([], 4),
    ([norm, grad], 4),                                                        # their copies are waited for without a limit
    ([lambda b: grad(b, cols=2001, lddy=2001, ldx=2001, lddx=2001)], 5),      # rows off the grid to several warps
    ([orth], 5),
    ([orth, lambda b: grad(b, cols=2001, lddy=2001, ldx=2001, lddx=2001)], 6),
])
def test_words(lib, calls, copies):  # noqa: F811
    def work():
        codes = [call(lib) for call in calls]
        return [max(codes, key=abs, default=0), _copies(lib), _copies(lib)]

    assert _apart(work) == [0, copies, copies]
