"""Layer norm with its gradient and the step by orthogonalised momentum, written out
in 64 bits (the two elementwise ends in 32, operation by operation).  Test
infrastructure; shares no code with the library."""
import numpy as np
import torch

NS = (3.4445, -4.7750, 2.0315)


def layer_norm(h, gamma, beta, eps):
    """h [rows, cols] float64: y, mean, rstd, xhat."""
    mean = h.mean(1)
    d = h - mean[:, None]
    rstd = 1.0 / torch.sqrt((d * d).mean(1) + eps)
    xhat = d * rstd[:, None]
    y = xhat if gamma is None else xhat * gamma
    return (y if beta is None else y + beta), mean, rstd, xhat


def layer_norm_grad(dy, x, mean, rstd, gamma):
    """dx, dgamma, dbeta and the magnitudes of what the first two are sums of."""
    xhat = (x - mean[:, None]) * rstd[:, None]
    g = dy if gamma is None else dy * gamma
    m1, m2 = g.mean(1, keepdim=True), (g * xhat).mean(1, keepdim=True)
    dx = rstd[:, None] * (g - m1 - xhat * m2)
    mag = rstd[:, None] * (g.abs() + g.abs().mean(1, keepdim=True) + xhat.abs() * (g * xhat).abs().mean(1, keepdim=True))
    return dx, (dy * xhat).sum(0), dy.sum(0), mag, (dy * xhat).abs().sum(0), dy.abs().sum(0)


def orthogonalize(x, steps=5, coefficients=NS, eps=1e-7):
    """x [..., rows, cols] float64."""
    a, b, c = coefficients
    n = x.square().sum((-2, -1), keepdim=True).sqrt() + eps
    x = torch.where(n == 0, torch.zeros_like(x), x / n)
    wide = x.shape[-2] <= x.shape[-1]
    for _ in range(steps):
        g = x @ x.mT if wide else x.mT @ x
        p = b * g + c * (g @ g)
        x = a * x + (p @ x if wide else x @ p)
    return x


def orthogonalize_rounded(x, steps=5, coefficients=NS, eps=1e-7, source_lo=True):
    """The same with the roundings that the library states: operands of products in
    fp16, X as two fp16 numbers hi + lo, products of hi alone, B's diagonal kept, which
    also stands for B in its product with lo.  Sums in 64 bits.  source_lo: whether the
    input has a lo (a bf16 one needs none)."""
    def half(t, scale):
        return (t * scale).float().half().double() / scale

    a, b, c = coefficients
    n = x.square().sum((-2, -1), keepdim=True).sqrt() + eps
    f, e = torch.frexp(n)
    x = x * torch.pow(2.0, -e.double())   # by a power of two; 1 / f goes into the first step
    s = torch.where(n == 0, torch.zeros_like(n), 1 / f)
    wide = x.shape[-2] <= x.shape[-1]
    for i in range(steps):
        hi = half(x, 2.0 ** 12)
        lo = half(x - hi, 2.0 ** 23) if i or source_lo else torch.zeros_like(x)
        g = half((hi @ hi.mT if wide else hi.mT @ hi) * s * s, 2.0 ** 10)
        p = b * g + c * (g @ g)
        q = half(p, 2.0 ** 10)
        d, r = p.diagonal(dim1=-2, dim2=-1), (p - q).diagonal(dim1=-2, dim2=-1)
        d, r = (d.unsqueeze(-1), r.unsqueeze(-1)) if wide else (d.unsqueeze(-2), r.unsqueeze(-2))
        x = s * ((a + r) * hi + (a + d) * lo + (q @ hi if wide else hi @ q))
        s = torch.ones_like(s)
    return x


def momentum(grads, divisor, m, mu, nesterov):
    """float32 arrays, every operation rounded on its own: the new m, and u before its cast."""
    f = np.float32
    s = np.zeros_like(m)
    for g in grads:
        s = (s + g).astype(f)
    g = (s / f(divisor)).astype(f)
    m = ((f(mu) * m).astype(f) + g).astype(f)
    return m, (g + (f(mu) * m).astype(f)).astype(f) if nesterov else m


def muon_update(w, o, lr, wd, scale):
    f = np.float32
    w = (w - ((f(lr) * f(wd)).astype(f) * w).astype(f)).astype(f)
    return (w - ((f(lr) * f(scale)).astype(f) * o).astype(f)).astype(f)
