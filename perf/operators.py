"""The dense operators of a training unit and what is measured of them.

Three operators, each with its gradient, that sit between the bf16 weights a
step gathers and the bf16 gradient buffer it reduces:

linear   y  = residual + D(act(x w^T + bias)),  pre = x w^T + bias kept for the gradient
         dz = D'(dy) act'(pre),  dx = dz w,  dw = acc + dz^T x,  db = sum over rows of dz
dropout  y  = residual + D(x),  dx = D'(dy)
rope     pairs of a head's first `rot` elements turned by position * frequency, and back

D keeps an element where its 16 random bits are at least round(65536 p), times
65536 / (65536 - round(65536 p)), and puts 0 elsewhere.  The bits come from the
counter-based generator Philox4x32-10 (Salmon, Moraes, Dror and Shaw, 2011): the
counter is (column / 8, row, site, step), the key the 64-bit seed, and its 128
bits serve eight neighbouring columns of a row, low halves first; no mask is stored.

`own` False: the plain forms below, elementary torch operations in 32 bits,
rounded once at the end.  `own` True: the framework's calls.
"""
import math

import numpy as np
import torch

own = False

DT = {"bf16": torch.bfloat16, "f32": torch.float32}
SEED = 0x1234_5678_9ABC


# --------------------------------------------------------------------------
# cases
# --------------------------------------------------------------------------


def _linear(name, m, k, n, bias=True, act="none", residual=False, p=0.0, pre=False, out="bf16", shift=0):
    return {"name": name, "op": "linear", "m": m, "k": k, "n": n, "bias": bias, "act": act,
            "residual": residual, "p": p, "pre": pre, "out": out, "shift": shift}


def _linear_grad(name, m, k, n, bias=True, act="none", p=0.0, out="bf16", acc=False, shift=0):
    return {"name": name, "op": "linear_grad", "m": m, "k": k, "n": n, "bias": bias, "act": act,
            "p": p, "out": out, "acc": acc, "shift": shift}


def _dropout(name, op, m, n, p, dtype="bf16", residual=False):
    return {"name": name, "op": op, "m": m, "n": n, "p": p, "dtype": dtype, "residual": residual}


def _rope(name, op, t, heads, dim, rot, layout="half", dtype="bf16", packed=0, most=0, scaling="none", factor=1.0):
    return {"name": name, "op": op, "t": t, "heads": heads, "dim": dim, "rot": rot, "layout": layout,
            "dtype": dtype, "packed": packed, "most": most, "scaling": scaling, "factor": factor}


def listed():
    return [
        # GPT-2 XL's query/key/value projection of one token: the smallest call, bound by its weights and by latency
        _linear("linear one token", 1, 1600, 4800),
        # GPT-2 XL's first feed-forward product over 8 sequences of 1024, its pre-activation kept for the gradient
        _linear("linear gpt2-xl fc", 8192, 1600, 6400, act="gelu_tanh", pre=True),
        # its second one: the end of a residual branch, with the model's dropout
        _linear("linear gpt2-xl proj", 8192, 6400, 1600, residual=True, p=0.1),
        # the tied head over one sequence: an odd number of columns, logits in 32 bits for the loss
        _linear("linear gpt2-xl head", 1024, 1600, 50257, bias=False, out="f32"),
        # the gradient of the first feed-forward product, into the bf16 gradient buffer
        _linear_grad("linear grad gpt2-xl fc", 8192, 1600, 6400, act="gelu_tanh"),
        # Llama-7B's down projection, a micro-batch of 2048 tokens added to the 32-bit accumulated gradient
        _linear_grad("linear grad llama-7b down", 2048, 11008, 4096, bias=False, out="f32", acc=True),
        # a small model whose tensors lie at odd places of the flat buffers: nothing is aligned
        _linear_grad("linear grad ragged", 333, 517, 1031, act="relu", p=0.25, shift=3),
        # GPT-2 XL's embedding or residual dropout over 8 sequences
        _dropout("dropout gpt2-xl residual", "dropout", 8192, 1600, 0.1, residual=True),
        # its gradient in 32 bits, rows of an odd length
        _dropout("dropout grad odd", "dropout_grad", 1021, 6401, 0.1, dtype="f32"),
        # queries and keys of one new token of Llama-7B
        _rope("rope one token", "rope", 1, 64, 128, 128),
        # queries and keys inside the packed projection of 4 sequences of 2048
        _rope("rope llama-7b packed", "rope", 8192, 64, 128, 128, packed=96),
        # the gradient at a stretched context: interleaved pairs, half of the head, positions up to 131072
        _rope("rope grad long", "rope_grad", 6001, 25, 64, 32, layout="interleaved", dtype="f32",
              most=131072, scaling="yarn", factor=16.0),
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def _size(rng, lo, hi):
    """A size of the range: as drawn, odd, or a multiple of 64 as widths most often are."""
    v = _log(rng, lo, hi)
    kind = rng.randrange(5)
    if kind == 0 or v < 64:
        return v
    return min(hi - 1 | 1, v | 1) if kind == 1 else v // 64 * 64


def draw(rng):
    op = rng.choice(["linear", "linear", "linear_grad", "linear_grad", "dropout", "dropout_grad", "rope", "rope_grad"])
    if op in ("linear", "linear_grad"):
        while True:
            m, k, n = _log(rng, 1, 8192), _size(rng, 48, 11008), _size(rng, 48, 50257)
            if m * k * n <= 1.5e11 / (2 if op == "linear_grad" else 1) and k * n <= 5e7 and m * n <= 5e7:
                break
        act = rng.choice(["none", "none", "relu", "gelu", "gelu_tanh", "silu"])
        p = rng.choice([0.0, 0.0, 0.1, 0.5])
        # 32-bit results: logits and the accumulated gradients of plain projections
        out = "f32" if rng.random() < 0.3 and (k if op == "linear" else m) <= 2048 and (op == "linear" or act == "none") else "bf16"
        shift = rng.choice([0, 0, 0, 0, 0, 8, 1, 5])
        if op == "linear":
            return _linear(None, m, k, n, rng.random() < 0.7, act, rng.random() < 0.5, p, act != "none" and rng.random() < 0.7, out, shift) | {"name": ""}
        return _linear_grad(None, m, k, n, rng.random() < 0.7, act, p, out, rng.random() < 0.5, shift) | {"name": ""}
    if op in ("dropout", "dropout_grad"):
        while True:
            m, n = _log(rng, 1, 65536), _size(rng, 1, 50257)
            if m * n <= 3e7:
                break
        return _dropout("", op, m, n, rng.choice([0.05, 0.1, 0.3, 0.5]), rng.choice(["bf16", "bf16", "f32"]), op == "dropout" and rng.random() < 0.5)
    dim = rng.choice([32, 64, 80, 128, 256])
    heads = rng.choice([1, 5, 8, 25, 32, 40, 64])
    rot = rng.choice([dim, dim, dim // 2, dim // 4])
    t = min(_log(rng, 1, 32768), 60_000_000 // (heads * dim))
    scaling = rng.choice(["none", "none", "linear", "ntk", "yarn"])
    return _rope("", op, t, heads, dim, rot, rng.choice(["half", "interleaved"]), rng.choice(["bf16", "bf16", "f32"]),
                 rng.choice([0, 0, heads + 8]), rng.choice([0, 4096, 131072]), scaling, 1.0 if scaling == "none" else rng.choice([2.0, 8.0, 32.0]))


def work(case):
    c = case
    if c["op"] in ("linear", "linear_grad"):
        m, k, n, o = c["m"], c["k"], c["n"], 4 if c["out"] == "f32" else 2
        if c["op"] == "linear":
            by = 2 * (m * k + n * k) + o * m * n + 2 * n * c["bias"] + o * m * n * c["residual"] + 2 * m * n * c["pre"]
            return {"bytes": by, "flops": 2 * m * n * k}
        by = 2 * (m * n + m * k + n * k) + 2 * m * k + o * n * k * (2 if c["acc"] else 1) + 2 * n * c["bias"] + 2 * m * n * (c["act"] != "none")
        return {"bytes": by, "flops": 4 * m * n * k}
    size = 4 if c["dtype"] == "f32" else 2
    if c["op"] in ("dropout", "dropout_grad"):
        return {"bytes": size * c["m"] * c["n"] * (3 if c["residual"] else 2), "flops": 2 * c["m"] * c["n"]}
    e = c["t"] * c["heads"] * c["dim"]
    return {"bytes": 2 * size * e + 8 * c["t"], "flops": 3 * c["t"] * c["heads"] * c["rot"]}


# --------------------------------------------------------------------------
# inputs
# --------------------------------------------------------------------------


def _frequencies(c, base=10000.0, context=4096.0):
    """Radians a position for each pair, and the factor on the turned elements: plain,
    interpolated (linear), with a larger base (ntk), or YaRN (Peng et al., 2023: by
    wavelength, interpolated where less than 1 turn fits the first context, kept
    where more than 32 do, and the 0.1 ln s + 1 temperature)."""
    rot, s = c["rot"], c["factor"]
    if c["scaling"] == "ntk" and rot > 2:
        base *= s ** (rot / (rot - 2))
    theta = np.array([base ** (-2.0 * i / rot) for i in range(rot // 2)])
    if c["scaling"] == "linear":
        return theta / s, 1.0
    if c["scaling"] == "yarn":
        keep = np.clip((context * theta / (2 * math.pi) - 1.0) / 31.0, 0.0, 1.0)
        return theta * (keep + (1.0 - keep) / s), 0.1 * math.log(s) + 1.0
    return theta, 1.0


def _placed(shape, shift, make):
    """A tensor that lies `shift` elements into a flat buffer, as a slice of gathered weights does."""
    n = math.prod(shape)
    flat = make(n + shift + 8)
    return flat[shift:shift + n].view(shape)


def prepare(case, seed):
    c = case
    dev = torch.device("cuda")
    g = torch.Generator(device=dev)
    g.manual_seed(int(seed) * 7919 + 17)
    bf = torch.bfloat16

    def normal(*shape, std=1.0, dtype=bf):
        return torch.randn(*shape, generator=g, device=dev).mul_(std).to(dtype)

    s = {"case": c, "step": int(seed) % 100003}
    if c["op"] in ("linear", "linear_grad"):
        m, k, n, shift, dt = c["m"], c["k"], c["n"], c["shift"], DT[c["out"]]
        s["x"] = normal(m, k)
        s["w"] = _placed((n, k), shift, lambda e: normal(e, std=0.02))
        s["bias"] = normal(n, std=0.1) if c["bias"] else None
        if c["op"] == "linear":
            s["residual"] = normal(m, n, dtype=dt) if c["residual"] else None
            s["pre"] = torch.empty(m, n, dtype=bf, device=dev) if c["pre"] else None
            s["y"] = torch.empty(m, n, dtype=dt, device=dev)
        else:
            s["dy"] = normal(m, n, std=1e-2)
            s["z"] = normal(m, n) if c["act"] != "none" else None
            s["acc"] = normal(n, k, std=1e-2, dtype=dt) if c["acc"] else None
            s["dz"] = torch.empty(m, n, dtype=bf, device=dev) if c["act"] != "none" or c["p"] else None
            s["dx"] = torch.empty(m, k, dtype=bf, device=dev)
            s["dw"] = _placed((n, k), shift, lambda e: torch.empty(e, dtype=dt, device=dev))
            s["db"] = torch.empty(n, dtype=dt, device=dev) if c["bias"] else None
    elif c["op"] in ("dropout", "dropout_grad"):
        dt = DT[c["dtype"]]
        s["x"] = normal(c["m"], c["n"], dtype=dt)
        s["residual"] = normal(c["m"], c["n"], dtype=dt) if c["residual"] else None
        s["y"] = torch.empty(c["m"], c["n"], dtype=dt, device=dev)
    else:
        t, h, d, dt = c["t"], c["heads"], c["dim"], DT[c["dtype"]]
        s["x"] = normal(t, max(h, c["packed"]), d, dtype=dt)[:, :h]
        s["y"] = torch.empty(t, h, d, dtype=dt, device=dev)
        most = c["most"]
        s["at"] = (torch.randint(0, most, (t,), generator=g, device=dev) if most
                   else torch.arange(t, device=dev) % 2048 + int(seed) % 1000)
        theta, s["scale"] = _frequencies(c)
        s["theta"] = torch.from_numpy(theta).to(dev)
    if own:  # the small handles that a program makes once
        import zero_sharded_mixed_gb300 as zero
        s["zero"] = zero
        if c["op"].startswith("rope"):
            layout, scaling = (getattr(zero, "ZERO_ROPE_" + c[key].upper()) for key in ("layout", "scaling"))
            s["plan"] = zero.zero_rope_plan(c["rot"], layout=layout, base=10000.0, scaling=scaling, factor=c["factor"], context=4096)
        else:
            s["act"] = getattr(zero, "ZERO_ACT_" + c.get("act", "none").upper())
            s["drop"] = zero.ZeroDropout.make(c["p"], seed=SEED, site=7, step=s["step"]) if c["p"] else None
    return s


# --------------------------------------------------------------------------
# the framework's calls
# --------------------------------------------------------------------------


def _run_own(s):
    c, zero = s["case"], s["zero"]
    if c["op"] == "linear":
        zero.zero_linear(s["x"], s["w"], s["y"], bias=s["bias"], act=s["act"], residual=s["residual"], drop=s["drop"], pre=s["pre"])
        return [s["y"], s["pre"]]
    if c["op"] == "linear_grad":
        dz, db = s["dy"], s["db"]
        if s["dz"] is not None:
            dz, db = s["dz"], None
            zero.zero_dropout_grad(s["dy"], dz, drop=s["drop"], act=s["act"], pre=s["z"], db=s["db"])
        zero.zero_linear_grad_input(dz, s["w"], s["dx"])
        zero.zero_linear_grad_weight(dz, s["x"], s["dw"], db=db, acc=s["acc"])
        return [s["dx"], s["dw"], s["db"]]
    if c["op"] == "dropout":
        zero.zero_dropout(s["x"], s["y"], s["drop"], residual=s["residual"])
    elif c["op"] == "dropout_grad":
        zero.zero_dropout_grad(s["x"], s["y"], drop=s["drop"])
    else:
        zero.zero_rope(s["plan"], s["x"], s["y"], positions=s["at"], inverse=c["op"] == "rope_grad")
    return s["y"]


# --------------------------------------------------------------------------
# the plain forms
# --------------------------------------------------------------------------


def _halves(rows, cols, step, dev):
    """The 16 random bits of every element, [rows, cols], as int32 values."""
    c0 = torch.arange((cols + 7) // 8, device=dev).expand(rows, -1)
    c1 = torch.arange(rows, device=dev)[:, None].expand_as(c0)
    c2, c3 = torch.full_like(c0, 7), torch.full_like(c0, step)
    k0, k1, low = SEED & 0xFFFFFFFF, SEED >> 32, 0xFFFFFFFF
    for r in range(10):  # ten rounds of two 32 x 32 -> 64 bit products
        p0, p1 = c0 * 0xD2511F53, c2 * 0xCD9E8D57
        c0, c1, c2, c3 = ((p1 >> 32) & low) ^ c1 ^ k0, p1 & low, ((p0 >> 32) & low) ^ c3 ^ k1, p0 & low
        k0, k1 = (k0 + 0x9E3779B9) & low, (k1 + 0xBB67AE85) & low
    words = torch.stack([c0, c1, c2, c3], dim=-1)
    bits = torch.stack([words & 0xFFFF, words >> 16], dim=-1).to(torch.int32)
    return bits.reshape(rows, -1)[:, :cols]


def _drop(v, p, step):
    if not p:
        return v
    cut = round(p * 65536)
    scale = 65536 / (65536 - cut) if cut < 65536 else 0.0
    return torch.where(_halves(v.shape[0], v.shape[1], step, v.device) >= cut, v * scale, 0.0)


def _act(z, act):
    if act == "relu":
        return torch.where(z < 0, 0.0, z)
    if act == "silu":
        return z / (1 + torch.exp(-z))
    if act == "gelu":
        return 0.5 * z * (1 + torch.erf(z * 0.5 ** 0.5))
    if act == "gelu_tanh":
        return 0.5 * z * (1 + torch.tanh((2 / math.pi) ** 0.5 * (z + 0.044715 * z * z * z)))
    return z


def _act_slope(z, act):
    if act == "relu":
        return (z > 0).float()
    if act == "silu":
        e = 1 / (1 + torch.exp(-z))
        return e * (1 + z * (1 - e))
    if act == "gelu":
        return 0.5 * (1 + torch.erf(z * 0.5 ** 0.5)) + z * torch.exp(-0.5 * z * z) * (0.5 / math.pi) ** 0.5
    u = torch.tanh((2 / math.pi) ** 0.5 * (z + 0.044715 * z * z * z))
    return 0.5 * (1 + u) + 0.5 * z * (1 - u * u) * (2 / math.pi) ** 0.5 * (1 + 3 * 0.044715 * z * z)


def _turn(x, cos, sin, rot, layout):
    x, rest = x[..., :rot], x[..., rot:]
    a, b = (x[..., :rot // 2], x[..., rot // 2:]) if layout == "half" else (x[..., 0::2], x[..., 1::2])
    a, b = a * cos - b * sin, b * cos + a * sin
    turned = torch.cat([a, b], dim=-1) if layout == "half" else torch.stack([a, b], dim=-1).flatten(-2)
    return torch.cat([turned, rest], dim=-1)


def run(state):
    s = state
    if own:
        return _run_own(s)
    c = s["case"]
    if c["op"] == "linear":
        dt = DT[c["out"]]
        z = s["x"].float() @ s["w"].float().t()
        if s["bias"] is not None:
            z = z + s["bias"].float()
        y = _drop(_act(z, c["act"]), c["p"], s["step"])
        if s["residual"] is not None:
            y = y + s["residual"].float()
        return [y.to(dt), z.to(torch.bfloat16) if s["pre"] is not None else None]
    if c["op"] == "linear_grad":
        dt = DT[c["out"]]
        dz = _drop(s["dy"].float(), c["p"], s["step"])
        if c["act"] != "none":
            dz = dz * _act_slope(s["z"].float(), c["act"])
        if dt == torch.float32 and s["dz"] is not None:
            dz = dz.to(torch.bfloat16).float()  # the operators' interface: dz is a bf16 tensor
        dx, dw = dz @ s["w"].float(), dz.t() @ s["x"].float()
        if s["acc"] is not None:
            dw = dw + s["acc"].float()
        return [dx.to(torch.bfloat16), dw.to(dt), dz.sum(0).to(dt) if c["bias"] else None]
    if c["op"] in ("dropout", "dropout_grad"):
        y = _drop(s["x"].float(), c["p"], s["step"])
        return (y if s["residual"] is None else y + s["residual"].float()).to(s["x"].dtype)
    # the turn of a position in 2^-64ths of a circle, whose products wrap where the circle does
    steps = torch.round(s["theta"] * (2.0 ** 64 / (2 * math.pi))).to(torch.int64)
    angle = ((s["at"][:, None] * steps[None, :]) >> 32).float() * (2 * math.pi / 2.0 ** 32)
    cos, sin = (torch.cos(angle) * s["scale"])[:, None], (torch.sin(angle) * s["scale"])[:, None]
    return _turn(s["x"].float(), cos, sin if c["op"] == "rope" else -sin, c["rot"], c["layout"]).to(s["x"].dtype)


# --------------------------------------------------------------------------
# the definitions in 64 bits
# --------------------------------------------------------------------------


def _kept(rows, cols, p, step, dev):
    """[rows, cols]: what D multiplies with, in 64 bits (0 where an element is dropped)."""
    cut = int(round(p * 65536))
    u = np.uint64
    nb = (cols + 7) // 8
    ctr = [np.broadcast_to(np.arange(nb, dtype=u), (rows, nb)), np.broadcast_to(np.arange(rows, dtype=u)[:, None], (rows, nb)),
           np.full((rows, nb), 7, u), np.full((rows, nb), step, u)]
    key, low = [SEED & 0xFFFFFFFF, SEED >> 32], u(0xFFFFFFFF)
    for _ in range(10):
        a, b = ctr[0] * u(0xD2511F53), ctr[2] * u(0xCD9E8D57)
        ctr = [(b >> u(32)) ^ ctr[1] ^ u(key[0]), b & low, (a >> u(32)) ^ ctr[3] ^ u(key[1]), a & low]
        key = [(key[0] + 0x9E3779B9) & 0xFFFFFFFF, (key[1] + 0xBB67AE85) & 0xFFFFFFFF]
    kept = np.empty((rows, nb, 8), np.float32)
    for j in range(8):
        kept[:, :, j] = ((ctr[j // 2] >> u(16 * (j % 2))) & u(0xFFFF)) >= u(cut)
    k = torch.from_numpy(kept.reshape(rows, nb * 8)[:, :cols]).to(dev).double()
    return k * (65536.0 / (65536 - cut)) if cut < 65536 else k * 0.0


def exact(case, seed):
    c, s = case, prepare(case, seed)
    if c["op"] in ("linear", "linear_grad"):
        m, n, act, dev = c["m"], c["n"], c["act"], s["x"].device
        x, w = s["x"].double(), s["w"].double()
        keep = _kept(m, n, c["p"], s["step"], dev) if c["p"] else 1.0
        z = (torch.einsum("mk,nk->mn", x, w) + (s["bias"].double() if c["bias"] else 0.0)) if c["op"] == "linear" else None
        if c["op"] == "linear_grad" and act != "none":
            z = s["z"].double()
        if z is not None:
            f = z.detach().requires_grad_(c["op"] == "linear_grad")
            cdf = {"none": 1.0, "relu": (f > 0).double(), "silu": torch.sigmoid(f) if act == "silu" else 0,
                   "gelu": torch.special.ndtr(f) if act == "gelu" else 0,
                   "gelu_tanh": torch.sigmoid(math.sqrt(8 / math.pi) * (f + 0.044715 * f ** 3)) if act == "gelu_tanh" else 0}[act]
            a = f * cdf
        if c["op"] == "linear":
            y = a * keep + (s["residual"].double() if c["residual"] else 0.0)
            return [y, z if c["pre"] else None]
        dz = s["dy"].double() * keep
        if act != "none":
            dz, = torch.autograd.grad(a, f, dz)
        if c["out"] == "f32" and s["dz"] is not None:
            # 32-bit sums over the dz that is handed on in bf16: its rounding is no
            # part of the definition, so they have no exact value at their precision
            return [torch.einsum("mn,nk->mk", dz, w), None, None]
        dw = torch.einsum("mn,mk->nk", dz, x) + (s["acc"].double() if c["acc"] else 0.0)
        return [torch.einsum("mn,nk->mk", dz, w), dw, dz.sum(dim=0) if c["bias"] else None]
    if c["op"] in ("dropout", "dropout_grad"):
        y = s["x"].double() * _kept(c["m"], c["n"], c["p"], s["step"], s["x"].device)
        return y + s["residual"].double() if c["residual"] else y
    back = -1.0 if c["op"] == "rope_grad" else 1.0
    theta, scale = _frequencies(c)
    angle = back * s["at"].cpu().numpy().astype(np.float64)[:, None] * theta[None, :]
    turn = torch.from_numpy(scale * np.exp(1j * angle)).to(s["x"].device)[:, None, :]
    y = s["x"].double()
    h = c["rot"] // 2
    first, second = (slice(0, h), slice(h, 2 * h)) if c["layout"] == "half" else (slice(0, 2 * h, 2), slice(1, 2 * h, 2))
    z = torch.complex(y[..., first].contiguous(), y[..., second].contiguous()) * turn
    y = y.clone()
    y[..., first], y[..., second] = z.real, z.imag
    return y
