"""zero_orthogonalize where a pair of CTAs has several tiles of each product: accumulators
used again, narrow tiles after full ones and beyond the pairs that had one tile less,
mirrored tiles of 128 and 256 columns, matrices from the last to the first.  (On 152 SMs
the shapes of test_gpu_orthogonalize give a pair at most two tiles of X' and one of A or B.)"""
import pytest
import torch

from tests.test_gpu_orthogonalize import BF, F32, _close, _run, _x

pytestmark = pytest.mark.gpu

# (batch, rows, columns): tiles a pair of A and B, of X', as planned for 76 pairs
WAVES = [
    (200, 256, 256),    # 2 to 3 full, 2 to 3
    (30, 512, 512),     # 2 to 3 of 128 columns, mirrored; 1 to 2
    (40, 512, 768),     # 1 to 2 of 256 columns, mirrored; 3 to 4
    (40, 768, 512),
    (300, 100, 333),    # 4 narrow alone; 7 to 8 of 192 columns
    (100, 260, 520),    # 1 to 2 full and 2 to 3 narrow, some beyond the lighter pairs; 7 to 8
    (40, 600, 520),     # 1 to 2 full and 2 narrow; 4 to 5
    (20, 832, 1000),    # mirrored full and narrow ones; 4 to 5
    (12, 1700, 900),    # fewer full ones than pairs; 4 to 5
    (10, 1100, 1700),   # a batch of many row tiles; 4 to 5
    (24, 600, 900),
    (500, 40, 64),
]


@pytest.mark.parametrize("shape", WAVES)
@pytest.mark.parametrize("dtype", [BF, F32])
def test_several_tiles_a_pair(zlib, cuda_device, shape, dtype):
    x = _x(shape, dtype, 13)
    y = _run(zlib, x.cuda())
    zlib.zero_status_check()
    _close(y, x)
    assert torch.equal(_run(zlib, x.cuda()), y)


def _whole(shape, dtype, seed):
    """Small whole numbers: their squares' sums are exact in any order.  (The norm is summed in
    parts whose number depends on the batch, a product's sums in one order for every tile.)"""
    g = torch.Generator().manual_seed(seed)
    return torch.randint(-8, 9, shape, generator=g).to(dtype)


@pytest.mark.parametrize("shape", [(40, 512, 768), (40, 600, 520), (20, 832, 1000), (12, 1700, 900)])
@pytest.mark.parametrize("dtype", [BF, F32])
def test_a_batch_and_its_matrices_alone(zlib, cuda_device, shape, dtype):
    """With the same norm to the bit, a matrix does not depend on the others or on its tiles."""
    x = _whole(shape, dtype, 17).cuda()
    y = _run(zlib, x)
    for i in (0, 1, shape[0] // 2, shape[0] - 1):
        assert torch.equal(_run(zlib, x[i]), y[i]), i


def test_matrices_of_a_block(zlib, cuda_device):
    """Twelve of 4800 x 1600, each as alone."""
    x = _whole((2, 4800, 1600), BF, 19).cuda()[[0, 1] * 6].contiguous()
    y = _run(zlib, x)
    one = [_run(zlib, x[i]) for i in (0, 1)]
    for i in range(12):
        assert torch.equal(y[i], one[i % 2]), i
    _close(one[0].unsqueeze(0), x[:1].cpu())
