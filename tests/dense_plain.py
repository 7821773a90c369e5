"""The dense operators (linear, dropout, rotary positions and their gradients)
written out in 64 bits, and the tolerances their kernels are held to.  Test
infrastructure; shares no code with the library."""
import math

import numpy as np
import torch

NONE, RELU, GELU, GELU_TANH, SILU = range(5)
ACTS = [NONE, RELU, GELU, GELU_TANH, SILU]


def philox4x32(counter, key, rounds=10):
    """Philox4x32 (Salmon et al., 2011) on numpy arrays of 32-bit words."""
    c, k, low = [np.asarray(x, np.uint64) for x in counter], [int(x) for x in key], np.uint64(0xFFFFFFFF)
    for _ in range(rounds):
        a, b = c[0] * np.uint64(0xD2511F53), c[2] * np.uint64(0xCD9E8D57)
        c = [(b >> np.uint64(32)) ^ c[1] ^ np.uint64(k[0]), b & low,
             (a >> np.uint64(32)) ^ c[3] ^ np.uint64(k[1]), a & low]
        k = [(k[0] + 0x9E3779B9) & 0xFFFFFFFF, (k[1] + 0xBB67AE85) & 0xFFFFFFFF]
    return c


def cut_of(p):
    return int(round(p * 65536))


def factor(rows, cols, p, seed=0, site=0, step=0):
    """[rows, cols] float64: what dropout multiplies with (0 where dropped)."""
    cut = cut_of(p)
    if cut == 0:
        return torch.ones(rows, cols, dtype=torch.float64)
    nb = -(-cols // 8)
    r, c = np.meshgrid(np.arange(rows), np.arange(nb), indexing="ij")
    w = philox4x32([c, r, np.full_like(c, site), np.full_like(c, step & 0xFFFFFFFF)], [seed & 0xFFFFFFFF, seed >> 32])
    halves = np.stack([h for x in w for h in (x & np.uint64(0xFFFF), x >> np.uint64(16))], axis=-1)
    keep = halves.reshape(rows, nb * 8)[:, :cols].astype(np.int64) >= cut
    # the factor itself is an fp32 number
    scale = float(np.float32(65536.0 / (65536 - cut))) if cut < 65536 else 0.0
    return torch.from_numpy(keep * scale)


def act(z, a):
    if a == RELU:
        return torch.where(z < 0, torch.zeros_like(z), z)
    if a == GELU:
        return z * 0.5 * torch.special.erfc(-z / math.sqrt(2))
    if a == GELU_TANH:
        return z * torch.sigmoid(2 * math.sqrt(2 / math.pi) * (z + 0.044715 * z ** 3))
    if a == SILU:
        return z * torch.sigmoid(z)
    return z


def slope(z, a):
    if a == RELU:
        return (z > 0).to(z.dtype)
    if a == GELU:
        return 0.5 * torch.special.erfc(-z / math.sqrt(2)) + z * torch.exp(-z * z / 2) / math.sqrt(2 * math.pi)
    if a == GELU_TANH:
        c = math.sqrt(2 / math.pi)
        s = torch.sigmoid(2 * c * (z + 0.044715 * z ** 3))
        return s + z * s * (1 - s) * 2 * c * (1 + 3 * 0.044715 * z * z)
    if a == SILU:
        s = torch.sigmoid(z)
        return s * (1 + z * (1 - s))
    return torch.ones_like(z)


# Tolerances.  A product of depth t summed in fp32 in any order, each addition
# rounded or cut (2^-23 relative at most), is within (t + 8) 2^-23 sum|a||b| of
# the exact one; the elementwise end adds a few more such steps on its own
# magnitude; the fast exponential and division are within 2^-19 of their values
# over the tested range; storing rounds by at most 2^-8 (bf16, 8 significant bits) or 2^-24 (fp32)
# of the value.  Slopes are at most 1.13, so an error of z grows by no more.
def eps_out(dtype):
    return 2.0 ** -8 if dtype == torch.bfloat16 else 2.0 ** -23


def tol_product(mag, depth, extra=0.0):
    return (depth + 8) * 2.0 ** -23 * mag + extra + 1e-30


def close(got, ref, tol, what=""):
    """Every element within tol (finite), the same infinities and NaNs."""
    got = got.double().cpu()
    ref, tol = ref.cpu(), (tol.cpu() if isinstance(tol, torch.Tensor) else torch.full_like(ref.cpu(), tol))
    assert got.shape == ref.shape
    fin = torch.isfinite(ref)
    assert torch.equal(torch.isnan(got), torch.isnan(ref)), f"{what}: NaNs differ"
    same = got[~fin & ~torch.isnan(ref)] == ref[~fin & ~torch.isnan(ref)]
    assert bool(same.all()), f"{what}: infinities differ"
    off = (got - ref).abs()[fin] - tol[fin]
    assert off.numel() == 0 or float(off.max()) <= 0, (
        f"{what}: {int((off > 0).sum())} of {off.numel()} past the tolerance, worst by {float(off.max()):.3e}")


# ---- rotary positions --------------------------------------------------------


def rope_theta(rot, base=10000.0, scaling=0, fac=1.0, context=0.0):
    """(frequencies, factor): NONE, LINEAR, NTK, YARN = 0..3."""
    if scaling == 2 and rot > 2:
        base = base * fac ** (rot / (rot - 2))
    th = np.array([base ** (-2.0 * i / rot) for i in range(rot // 2)])
    if scaling == 1:
        return th / fac, 1.0
    if scaling == 3:
        turns = context * th / (2 * math.pi)
        keep = np.clip((turns - 1) / (32 - 1), 0, 1)
        return th * keep + th / fac * (1 - keep), 0.1 * math.log(fac) + 1
    return th, 1.0


def rope(x, positions, rot, layout, theta, scale, inverse=False):
    """x [tokens, heads, dim] float64; layout 0 half, 1 interleaved."""
    # angles reduced with exact integer positions in extended precision
    ang = np.asarray(positions, np.longdouble)[:, None] * np.asarray(theta, np.longdouble)[None, :]
    ang = np.asarray(np.remainder(ang, 2 * np.longdouble(np.pi)), np.float64) if np.finfo(np.longdouble).nmant > 60 else np.asarray(ang, np.float64)
    c = torch.from_numpy(np.cos(ang) * scale)[:, None, :]
    s = torch.from_numpy(np.sin(ang) * scale)[:, None, :] * (-1 if inverse else 1)
    y = x.clone()
    h = rot // 2
    ia, ib = (slice(0, h), slice(h, rot)) if layout == 0 else (slice(0, rot, 2), slice(1, rot, 2))
    a, b = x[..., ia], x[..., ib]
    y[..., ia], y[..., ib] = a * c - b * s, b * c + a * s
    return y


# ---- placing inputs and outputs ------------------------------------------------


def inside(t, ld=None, shift=0, fill=float("nan")):
    """t (a CPU matrix) on the GPU as rows `ld` apart, `shift` elements into a
    buffer whose every other element is `fill`: what is read beside it shows.
    Returns (the view, the buffer)."""
    rows, cols = t.shape
    ld = cols if ld is None else ld
    buf = torch.full((shift + rows * ld + 64,), fill, dtype=t.dtype, device="cuda")
    view = buf[shift:shift + rows * ld].view(rows, ld)[:, :cols]
    view.copy_(t)
    return view, buf


SENTINEL = -77.0


def blank(rows, cols, dtype, ld=None, shift=0):
    """An output matrix inside a buffer of sentinels: (the view, a check that
    nothing outside the view was written)."""
    view, buf = inside(torch.full((rows, cols), SENTINEL, dtype=dtype), ld, shift, SENTINEL)

    def untouched():
        keep = view.clone()
        view.fill_(SENTINEL)
        ok = bool((buf == SENTINEL).all())
        view.copy_(keep)
        return ok

    return view, untouched
