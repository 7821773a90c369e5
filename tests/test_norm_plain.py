"""The 64-bit statements of layer norm and of the orthogonalised step against
differences, torch's own gradient and singular values (CPU)."""
import numpy as np
import pytest
import torch

from tests import norm_plain as npl


def _case(rows, cols, seed=0):
    g = torch.Generator().manual_seed(seed)
    return (torch.randn(rows, cols, generator=g, dtype=torch.float64) + 0.3, 1 + 0.2 * torch.randn(cols, generator=g, dtype=torch.float64),
            torch.randn(cols, generator=g, dtype=torch.float64), torch.randn(rows, cols, generator=g, dtype=torch.float64))


@pytest.mark.parametrize("shape", [(1, 1), (1, 5), (3, 8), (4, 33)])
def test_gradient_against_differences(shape):
    x, gamma, beta, dy = _case(*shape)
    eps, d = 1e-3, 1e-6

    def loss(x, gamma, beta):
        return (npl.layer_norm(x, gamma, beta, eps)[0] * dy).sum()

    _, mean, rstd, _ = npl.layer_norm(x, gamma, beta, eps)
    dx, dg, db = npl.layer_norm_grad(dy, x, mean, rstd, gamma)[:3]
    for value, grad, at in ((x, dx, 0), (gamma, dg, 1), (beta, db, 2)):
        flat = value.reshape(-1)
        for i in range(flat.numel()):
            args = [[x, gamma, beta], [x, gamma, beta]]
            for side, sign in zip(args, (1, -1)):
                moved = value.clone().reshape(-1)
                moved[i] += sign * d
                side[at] = moved.reshape(value.shape)
            diff = (loss(*args[0]) - loss(*args[1])) / (2 * d)
            # a central difference: d^2 times third derivatives (up to eps^-1.5), and rounding over d
            assert abs(float(diff) - float(grad.reshape(-1)[i])) < 1e-6


def test_gradient_against_torch():
    x, gamma, beta, dy = (t.requires_grad_() for t in _case(17, 40, 3))
    y = torch.nn.functional.layer_norm(x, (40,), gamma, beta, 1e-5)
    ref = torch.autograd.grad(y, (x, gamma, beta), dy.detach())
    with torch.no_grad():
        mine, mean, rstd, _ = npl.layer_norm(x, gamma, beta, 1e-5)
        got = npl.layer_norm_grad(dy, x, mean, rstd, gamma)[:3]
        assert torch.allclose(mine, y, rtol=1e-12, atol=1e-12)
        for a, b in zip(got, ref):
            assert torch.allclose(a, b, rtol=1e-10, atol=1e-12)


@pytest.mark.parametrize("shape", [(1, 1), (6, 6), (5, 12), (12, 5)])
def test_orthogonalized_matrix_has_the_singular_vectors(shape):
    g = torch.Generator().manual_seed(1)
    x = torch.randn(*shape, generator=g, dtype=torch.float64)
    u, s, vt = torch.linalg.svd(x, full_matrices=False)
    s = s / (x.norm() + 1e-7)
    a, b, c = npl.NS
    for _ in range(5):
        s = s * (a + b * s ** 2 + c * s ** 4)
    assert torch.allclose(npl.orthogonalize(x), u @ torch.diag(s) @ vt, rtol=1e-9, atol=1e-9)
    assert float(s.min()) > 0.6 and float(s.max()) < 1.3 or min(shape) > 1


@pytest.mark.parametrize("kind,limit", [("plain", 1.1e-3), ("tall", 1.1e-3), ("heavy", 1.1e-3), ("faint", 1.3e-3), ("few", 4e-3), ("one", 1e-3)])
def test_what_the_roundings_cost(kind, limit):
    """The iteration with the library's roundings against the exact one, by norm: about a
    thousandth, also where a few directions stand a thousand times above the rest; small
    matrices of that kind, whose few directions are rounded together, have the most."""
    g = torch.Generator().manual_seed(3)

    def normal(*shape):
        return torch.randn(*shape, generator=g, dtype=torch.float64)

    x = {"plain": lambda: normal(256, 384), "tall": lambda: normal(300, 64), "heavy": lambda: normal(200, 300) * torch.exp(normal(200, 1)),
         "faint": lambda: normal(384, 24) @ normal(24, 512) + 1e-3 * normal(384, 512), "few": lambda: normal(40, 2) @ normal(2, 100) + 1e-3 * normal(40, 100),
         "one": lambda: normal(1, 50)}[kind]().to(torch.bfloat16).double()
    ref = npl.orthogonalize(x)
    assert float((npl.orthogonalize_rounded(x, source_lo=False) - ref).norm() / ref.norm()) < limit


def test_elementwise_ends():
    f = np.float32
    m, u = npl.momentum([np.array([1, 2], f), np.array([3, 4], f)], 2.0, np.array([1, -1], f), 0.5, True)
    assert m.tolist() == [2.5, 2.5] and u.tolist() == [3.25, 4.25]
    assert npl.muon_update(np.array([2.0], f), np.array([1.0], f), 0.5, 0.5, 2.0).tolist() == [0.5]
