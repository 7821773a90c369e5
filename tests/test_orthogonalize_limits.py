"""The largest matrices that zero_orthogonalize takes, as the header states them (CPU)."""
import pytest

from zero_sharded_mixed_gb300 import binding as zb


@pytest.mark.parametrize("rows,cols", [(32768, 131064), (131071, 32768), (1, 1 << 30), ((1 << 29) - 1, 1), (3, 1 << 30), (32768, 32768), ((1 << 29) - 1, 8)])
def test_taken(rows, cols):
    """hi and lo of X twice at least."""
    assert zb.zero_orthogonalize_workspace(1, rows, cols) >= 8 * rows * cols


@pytest.mark.parametrize("rows,cols", [(32768, 131072), (131072, 32768), (32769, 32769), (4, 1 << 30), (1 << 30, 1), (1, (1 << 30) + 1), ((1 << 30) + 1, 1), (1 << 29, 8)])
def test_refused(rows, cols):
    with pytest.raises(zb.ZeroError) as e:
        zb.zero_orthogonalize_workspace(1, rows, cols)
    assert e.value.code == zb.ZERO_ERANGE
