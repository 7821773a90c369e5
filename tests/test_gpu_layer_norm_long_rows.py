"""Layer norm of rows of many million columns: sums of as many terms keep fp32's digits, also
where the terms are alike and each addition rounds the same way."""
import pytest
import torch

pytestmark = pytest.mark.gpu
BF, F32 = torch.bfloat16, torch.float32


@pytest.mark.parametrize("cols", [200_003, 30_000_001, 1 << 28])
@pytest.mark.parametrize("dtype", [BF, F32])
def test_equal_columns(zlib, cuda_device, cols, dtype):
    """Mean and deviation of one number: a sum of n terms in runs of 256 and of those by 512 threads
    is off by some (256 + n / 2^17 + 9) 2^-24 of itself at most, for 2^28 1.4e-4; the deviations
    from that mean correct it by as much of what is left, 2e-8, so that fp32's own 2^-24 and two
    more roundings remain: 2^-22.  Of y that is times rstd, at most 1 / sqrt(eps) = 316."""
    value = torch.tensor(1.1).to(dtype)
    x = torch.full((1, cols), float(value), dtype=dtype, device="cuda")
    y, mean, rstd = torch.empty_like(x), torch.empty(1, device="cuda"), torch.empty(1, device="cuda")
    zlib.zero_layer_norm(x, y, mean=mean, rstd=rstd)
    zlib.zero_status_check()
    v = float(value)
    assert abs(float(mean) - v) <= 2.0 ** -22 * v
    # the variance is 0, to (2^-22 v)^2 and what is left of the two sums' difference, 1.4e-4 of
    # (1.4e-4 v)^2: 4e-12 beside eps = 1e-5
    assert abs(float(rstd) * 1e-5 ** 0.5 - 1) <= 1e-6
    assert float(y.abs().max()) <= 2.0 ** -22 * v * 317


@pytest.mark.parametrize("cols", [30_000_001, 1 << 27])
def test_gradient_of_equal_columns(zlib, cuda_device, cols):
    """dy of one number: g - avg(g) is 0, to the average's rounding, (256 + n / 2^17 + 9) 2^-24 of
    it; x is 0 but for two columns, so that the other average is small and exact."""
    x = torch.zeros(1, cols, device="cuda")
    x[0, 0], x[0, 1] = 1.0, -1.0
    dy = torch.full_like(x, 1.1)
    mean, rstd = torch.zeros(1, device="cuda"), torch.ones(1, device="cuda")
    dx = torch.empty_like(x)
    zlib.zero_layer_norm_grad(dy, x, mean, rstd, dx)
    zlib.zero_status_check()
    assert float(dx.abs().max()) <= 1.1 * (256 + cols / 2 ** 17 + 9) * 2.0 ** -24
