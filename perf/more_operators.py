"""The operators of a unit's norms and of its orthogonalised update, and what is measured of them.

layer_norm       h = x + residual (kept in x's type), y = (h - mean) rstd gamma + beta, with the
                 mean of a row of h and rstd = 1 / sqrt(variance + eps) kept for the gradient
layer_norm_grad  with xhat = (x - mean) rstd and g = dy gamma:
                 dx = residual + rstd (g - mean(g) - xhat mean(g xhat)),
                 dgamma = acc + sum over rows of dy xhat, dbeta = acc + sum over rows of dy
momentum         g = the mean of the ranks' gradients, m = mu m + g, u = g + mu m in bf16
orthogonalize    X = U / (|U| + eps) by the Frobenius norm, then five times
                 X = a X + (b A + c A A) X with A = X X^T (of the shorter side): the singular
                 values go to about 1, the singular vectors stay (a quintic Newton-Schulz iteration)
update           w = w - lr wd w - lr scale o in 32 bits, and its bf16 weights

The last three are one step of the Muon optimizer (Jordan et al., 2024) under ZeRO: the ranks'
gradients reduced into the owners' momentum, the gathered momentum orthogonalised matrix by
matrix, the owners' master weights moved and cast into the gathered weights.

`own` False: the plain forms below, elementary torch operations in 32 bits, rounded once at the
end.  `own` True: the framework's calls.
"""
import math

import torch

own = False

DT = {"bf16": torch.bfloat16, "f32": torch.float32}
EPS = 1e-5                                  # of the norms
NS = (3.4445, -4.7750, 2.0315)              # the quintic's coefficients
NS_STEPS, NS_EPS = 5, 1e-7
MU, LR, WD = 0.95, 0.02, 0.01


# --------------------------------------------------------------------------
# cases
# --------------------------------------------------------------------------


def _norm(name, rows, cols, dtype="bf16", out="bf16", residual=True, affine=True, shift=0):
    return {"name": name, "op": "layer_norm", "rows": rows, "cols": cols, "dtype": dtype, "out": out,
            "residual": residual, "affine": affine, "shift": shift}


def _norm_grad(name, rows, cols, dtype="bf16", weights="bf16", residual=True, acc=False, shift=0):
    return {"name": name, "op": "layer_norm_grad", "rows": rows, "cols": cols, "dtype": dtype,
            "weights": weights, "residual": residual, "acc": acc, "shift": shift}


def _flat(name, op, n, ranks, skip=0, src="bf16"):
    return {"name": name, "op": op, "n": n, "ranks": ranks, "skip": skip, "src": src}


def _orth(name, batch, rows, cols, dtype="bf16", shift=0):
    return {"name": name, "op": "orthogonalize", "batch": batch, "rows": rows, "cols": cols, "dtype": dtype, "shift": shift}


def listed():
    return [
        # the norm of one new token's 32-bit residual stream, GPT-2 XL's width: the smallest call, all latency
        _norm("layer norm one token", 1, 1600, dtype="f32", residual=False),
        # the norm after a branch of GPT-2 XL over 8 sequences of 1024: the branch joins the stream in the same pass
        _norm("layer norm gpt2-xl", 8192, 1600),
        # its gradient, joined with the stream's, and the gain's and shift's gradients into the bf16 gradient buffer
        _norm_grad("layer norm grad gpt2-xl", 8192, 1600),
        # odd rows in 32 bits, gradients added to the accumulated ones, weights at an odd place of the flat buffers
        _norm_grad("layer norm grad odd", 1021, 6401, dtype="f32", weights="f32", residual=False, acc=True, shift=3),
        # the momentum of one GPT-2 XL block's matrices over 8 ranks
        _flat("momentum gpt2-xl block", "momentum", 12 * 1600 * 1600, 8),
        # an odd range of a small model's buffer, from the accumulated 32-bit gradient
        _flat("momentum odd range", "momentum", 1000003, 2, skip=4801, src="f32"),
        # a small block's square projection: fifteen dependent products of next to nothing
        _orth("orthogonalize small", 1, 256, 256),
        # three small layers' matrices at odd places of the flat buffer
        _orth("orthogonalize ragged", 3, 517, 333, shift=3),
        # the query/key/value projections of 12 of GPT-2 XL's blocks, taller than wide
        _orth("orthogonalize gpt2-xl qkv", 12, 4800, 1600),
        # one Llama-7B down projection: the largest call
        _orth("orthogonalize llama-7b down", 1, 4096, 11008),
        # the weights of one GPT-2 XL block's matrices after it
        _flat("update gpt2-xl block", "update", 12 * 1600 * 1600, 8),
        # and an odd range of a small model's
        _flat("update odd range", "update", 1000003, 2, skip=4801),
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
    op = rng.choice(["layer_norm", "layer_norm_grad", "layer_norm_grad", "momentum", "update",
                     "orthogonalize", "orthogonalize", "orthogonalize"])
    if op in ("layer_norm", "layer_norm_grad"):
        while True:
            rows, cols = _log(rng, 1, 65536), _size(rng, 48, 16384)
            if rows * cols <= 3e7:
                break
        dtype, shift = rng.choice(["bf16", "bf16", "f32"]), rng.choice([0, 0, 0, 8, 1, 5])
        residual = rng.random() < 0.6
        if op == "layer_norm":
            return _norm("", rows, cols, dtype, rng.choice(["bf16", dtype]), residual, rng.random() < 0.8, shift)
        return _norm_grad("", rows, cols, dtype, rng.choice(["bf16", "f32"]), residual, rng.random() < 0.5, shift)
    if op in ("momentum", "update"):
        n = _log(rng, 1000, 30_000_000)
        src = "f32" if op == "momentum" and rng.random() < 0.3 else "bf16"
        return _flat("", op, n, rng.choice([1, 2, 4, 8]), rng.choice([0, 0, 64, 77]), src)
    while True:
        batch, rows, cols = _log(rng, 1, 24), _size(rng, 16, 11008), _size(rng, 16, 11008)
        if batch * _flops(rows, cols) <= 2.4e12 and batch * rows * cols <= 1e8:
            break
    return _orth("", batch, rows, cols, rng.choice(["bf16", "bf16", "f32"]), rng.choice([0, 0, 0, 8, 1, 3]))


def _flops(rows, cols):
    """Of one orthogonalised matrix: a symmetric product of two factors needs half of its multiplications."""
    s, t = min(rows, cols), max(rows, cols)
    return NS_STEPS * (s * s * t + s * s * s + 2 * s * s * t)


def work(case):
    c = case
    if c["op"] == "layer_norm":
        e, size = c["rows"] * c["cols"], DT[c["dtype"]].itemsize
        return {"bytes": e * (size * (3 if c["residual"] else 1) + DT[c["out"]].itemsize) + 8 * c["rows"] + (4 * c["cols"] if c["affine"] else 0),
                "flops": 8 * e}
    if c["op"] == "layer_norm_grad":
        e, size = c["rows"] * c["cols"], DT[c["dtype"]].itemsize
        vectors = c["cols"] * (2 + DT[c["weights"]].itemsize * (4 if c["acc"] else 2))
        return {"bytes": e * (2 + size * (3 if c["residual"] else 2)) + 8 * c["rows"] + vectors, "flops": 14 * e}
    if c["op"] == "momentum":
        return {"bytes": c["n"] * (8 + 2 + (4 if c["src"] == "f32" else 2 * c["ranks"])), "flops": c["n"] * (4 + c["ranks"])}
    if c["op"] == "update":
        return {"bytes": 12 * c["n"], "flops": 4 * c["n"]}
    e = c["batch"] * c["rows"] * c["cols"]
    return {"bytes": e * (DT[c["dtype"]].itemsize + 2), "flops": c["batch"] * _flops(c["rows"], c["cols"])}


# --------------------------------------------------------------------------
# inputs
# --------------------------------------------------------------------------


def _placed(shape, shift, make):
    """A tensor that lies `shift` elements into a flat buffer, as a slice of the weights does."""
    n = math.prod(shape)
    return make(n + shift + 8)[shift:shift + n].view(shape)


def _buffer(c):
    """Elements of the flat buffers around a range of n: whole shards of the ranks, multiples of 8."""
    most = c["skip"] + c["n"]
    return (-(-most // c["ranks"]) + 7) // 8 * 8 * c["ranks"]


def prepare(case, seed):
    c = case
    dev = torch.device("cuda")
    g = torch.Generator(device=dev)
    g.manual_seed(int(seed) * 7919 + 29)
    bf, f32 = torch.bfloat16, torch.float32

    def normal(*shape, std=1.0, dtype=bf):
        return torch.randn(*shape, generator=g, device=dev).mul_(std).to(dtype)

    s = {"case": c}
    if c["op"] == "layer_norm":
        rows, cols, dt, shift = c["rows"], c["cols"], DT[c["dtype"]], c["shift"]
        s["x"] = normal(rows, cols, dtype=dt)
        s["residual"] = normal(rows, cols, std=3.0, dtype=dt) if c["residual"] else None
        # a stream of transformer blocks: rows have a mean of their own
        s["x"] += normal(rows, 1, std=0.5, dtype=dt)
        s["gamma"] = _placed((cols,), shift, lambda e: normal(e, std=0.2) + 1) if c["affine"] else None
        s["beta"] = _placed((cols,), shift, lambda e: normal(e, std=0.1)) if c["affine"] else None
        s["sum"] = torch.empty(rows, cols, dtype=dt, device=dev) if c["residual"] else None
        s["y"] = torch.empty(rows, cols, dtype=DT[c["out"]], device=dev)
        s["mean"], s["rstd"] = torch.empty(rows, device=dev), torch.empty(rows, device=dev)
    elif c["op"] == "layer_norm_grad":
        rows, cols, dt, wt, shift = c["rows"], c["cols"], DT[c["dtype"]], DT[c["weights"]], c["shift"]
        s["x"] = normal(rows, cols, std=2.0, dtype=dt) + normal(rows, 1, std=0.5, dtype=dt)
        s["dy"] = normal(rows, cols, std=1e-2)
        s["residual"] = normal(rows, cols, std=1e-2, dtype=dt) if c["residual"] else None
        s["gamma"] = _placed((cols,), shift, lambda e: normal(e, std=0.2) + 1)
        # what the forward pass kept
        x = s["x"].double()
        mean = x.mean(1)
        s["mean"], s["rstd"] = mean.float(), (x.sub_(mean[:, None]).square_().mean(1) + EPS).rsqrt().float()
        s["dx"] = torch.empty(rows, cols, dtype=dt, device=dev)
        for name in ("dgamma", "dbeta"):
            s[name] = _placed((cols,), shift, lambda e: torch.empty(e, dtype=wt, device=dev))
            s[name + "_acc"] = normal(cols, std=1e-2, dtype=wt) if c["acc"] else None
    elif c["op"] == "momentum":
        p = _buffer(c)
        s["grads"] = ([normal(p, std=1e-3, dtype=f32)] if c["src"] == "f32"
                      else [normal(p, std=1e-3) for _ in range(c["ranks"])])
        s["m"] = normal(p, std=5e-3, dtype=f32)
        s["u"] = torch.zeros(p, dtype=bf, device=dev)
    elif c["op"] == "update":
        p = _buffer(c)
        s["o"] = normal(p, std=0.02)
        s["w"] = normal(p, std=0.02, dtype=f32)
        s["out"] = s["w"].to(bf)
    else:
        b, rows, cols, dt, shift = c["batch"], c["rows"], c["cols"], DT[c["dtype"]], c["shift"]
        # a momentum's spectrum: some directions of a few tokens stand far above the rest
        r = max(1, min(rows, cols) // 16)
        strong = torch.linspace(2.0, 0.2, r, device=dev)[:, None] * normal(b, r, cols, dtype=f32)
        x = torch.bmm(normal(b, rows, r, dtype=f32), strong) / math.sqrt(r) + normal(b, rows, cols, dtype=f32)
        s["x"] = _placed((b, rows, cols), shift, lambda e: torch.empty(e, dtype=dt, device=dev)).copy_(x * 1e-3)
        s["y"] = _placed((b, rows, cols), shift, lambda e: torch.empty(e, dtype=bf, device=dev))
    if own:  # the small handles and workspaces that a program makes once
        import zero_sharded_mixed_gb300 as zero
        s["zero"] = zero
        if c["op"] == "layer_norm_grad":
            s["workspace"] = torch.empty(zero.zero_layer_norm_grad_workspace(c["rows"], c["cols"]), dtype=torch.uint8, device=dev)
        elif c["op"] == "orthogonalize":
            s["workspace"] = torch.empty(zero.zero_orthogonalize_workspace(c["batch"], c["rows"], c["cols"]), dtype=torch.uint8, device=dev)
        elif c["op"] in ("momentum", "update"):
            s["layout"] = zero.zero_layout([c["skip"] + c["n"]], c["ranks"])
            s["hp"] = zero.ZeroMuon.make(lr=LR, momentum=MU, weight_decay=WD, scale=0.2)
    return s


# --------------------------------------------------------------------------
# the framework's calls
# --------------------------------------------------------------------------


def _run_own(s):
    c, zero = s["case"], s["zero"]
    if c["op"] == "layer_norm":
        zero.zero_layer_norm(s["x"], s["y"], gamma=s["gamma"], beta=s["beta"], eps=EPS, residual=s["residual"], sum=s["sum"],
                             mean=s["mean"], rstd=s["rstd"])
        return [s["y"], s["sum"], s["mean"], s["rstd"]]
    if c["op"] == "layer_norm_grad":
        zero.zero_layer_norm_grad(s["dy"], s["x"], s["mean"], s["rstd"], s["dx"], gamma=s["gamma"], residual=s["residual"],
                                  dgamma=s["dgamma"], dbeta=s["dbeta"], dgamma_acc=s["dgamma_acc"], dbeta_acc=s["dbeta_acc"],
                                  workspace=s["workspace"])
        return [s["dx"], s["dgamma"], s["dbeta"]]
    if c["op"] == "momentum":
        code = zero.ZERO_F32 if c["src"] == "f32" else zero.ZERO_BF16
        zero.zero_reduce_scatter_momentum(s["layout"], s["grads"], code, 0, float(c["ranks"]), 0, c["ranks"], c["skip"], c["skip"] + c["n"],
                                          s["m"], s["u"], zero.ZERO_OUT_FULL, s["hp"])
        return [s["m"], s["u"]]
    if c["op"] == "update":
        zero.zero_muon_update(s["layout"], s["o"], 0, 0, c["ranks"], c["skip"], c["skip"] + c["n"], s["w"], s["out"],
                              zero.ZERO_OUT_FULL, s["hp"])
        return [s["w"], s["out"]]
    zero.zero_orthogonalize(s["x"], s["y"], steps=NS_STEPS, coefficients=NS, eps=NS_EPS, workspace=s["workspace"])
    return s["y"]


# --------------------------------------------------------------------------
# the plain forms
# --------------------------------------------------------------------------


def run(state):
    s = state
    if own:
        return _run_own(s)
    c = s["case"]
    if c["op"] == "layer_norm":
        h = s["x"].float()
        total = None
        if s["residual"] is not None:
            total = (h + s["residual"].float()).to(DT[c["dtype"]])
            h = total.float()
        mean = h.mean(1, keepdim=True)
        h = h - mean
        rstd = 1 / torch.sqrt((h * h).mean(1, keepdim=True) + EPS)
        y = h * rstd
        if s["gamma"] is not None:
            y = y * s["gamma"].float() + s["beta"].float()
        return [y.to(DT[c["out"]]), total, mean[:, 0], rstd[:, 0]]
    if c["op"] == "layer_norm_grad":
        rstd = s["rstd"][:, None]
        xhat = (s["x"].float() - s["mean"][:, None]) * rstd
        dy = s["dy"].float()
        g = dy * s["gamma"].float()
        dx = rstd * (g - g.mean(1, keepdim=True) - xhat * (g * xhat).mean(1, keepdim=True))
        if s["residual"] is not None:
            dx = dx + s["residual"].float()
        sums = [(dy * xhat).sum(0), dy.sum(0)]
        if c["acc"]:
            sums = [a + s[name].float() for a, name in zip(sums, ("dgamma_acc", "dbeta_acc"))]
        return [dx.to(DT[c["dtype"]])] + [a.to(DT[c["weights"]]) for a in sums]
    if c["op"] == "momentum":
        part = slice(c["skip"], c["skip"] + c["n"])
        total = torch.zeros(c["n"], device=s["m"].device)
        for grad in s["grads"]:
            total = total + grad[part].float()
        g = total / float(c["ranks"])
        m = MU * s["m"][part] + g
        s["m"][part] = m
        s["u"][part] = (g + MU * m).to(torch.bfloat16)
        return [s["m"], s["u"]]
    if c["op"] == "update":
        part = slice(c["skip"], c["skip"] + c["n"])
        w = s["w"][part]
        w = w - LR * WD * w - (LR * 0.2) * s["o"][part].float()
        s["w"][part] = w
        s["out"][part] = w.to(torch.bfloat16)
        return [s["w"], s["out"]]
    x = s["x"].float()
    tall = c["rows"] > c["cols"]
    if tall:
        x = x.transpose(1, 2)
    x = x / (x.double().square().sum((1, 2), keepdim=True).sqrt().float() + NS_EPS)
    for _ in range(NS_STEPS):
        a = x @ x.transpose(1, 2)
        x = NS[0] * x + (NS[1] * a + NS[2] * (a @ a)) @ x
    return (x.transpose(1, 2) if tall else x).to(torch.bfloat16).contiguous()


# --------------------------------------------------------------------------
# the definitions in 64 bits
# --------------------------------------------------------------------------


def exact(case, seed):
    c = case
    if c["op"] == "orthogonalize" and c["batch"] * _flops(c["rows"], c["cols"]) > 4e12:
        return None
    s = prepare(case, seed)
    if c["op"] == "layer_norm":
        h, total = s["x"].double(), None
        if c["residual"]:
            total = h + s["residual"].double()
            h = total.to(s["x"].dtype).double()  # what is normalised is the sum as it is kept
        var, mean = torch.var_mean(h, dim=1, correction=0)
        rstd = (var + EPS).pow(-0.5)
        y = torch.einsum("rc,r->rc", h - mean[:, None], rstd)
        if c["affine"]:
            y = torch.addcmul(s["beta"].double(), y, s["gamma"].double())
        return [y, total, mean, rstd]
    if c["op"] == "layer_norm_grad":
        x = s["x"].double().requires_grad_()
        gamma = s["gamma"].double().requires_grad_()
        beta = torch.zeros_like(gamma).requires_grad_()
        var, mean = torch.var_mean(x, dim=1, correction=0, keepdim=True)
        y = (x - mean) * (var + EPS).pow(-0.5) * gamma + beta
        grads = list(torch.autograd.grad(y, (x, gamma, beta), s["dy"].double()))
        for i, name in enumerate(("residual", "dgamma_acc", "dbeta_acc")):
            if s[name] is not None:
                grads[i] = grads[i] + s[name].double()
        return grads
    if c["op"] == "momentum":
        a, b = c["skip"], c["skip"] + c["n"]
        g = torch.stack([t[a:b].double() for t in s["grads"]]).sum(0).div_(c["ranks"])
        m, u = s["m"].double(), s["u"].double()
        m[a:b].mul_(MU).add_(g)
        u[a:b] = torch.add(g, m[a:b], alpha=MU)
        return [m, u]
    if c["op"] == "update":
        a, b = c["skip"], c["skip"] + c["n"]
        w, out = s["w"].double(), s["out"].double()
        w[a:b].mul_(1 - LR * WD).add_(s["o"][a:b].double(), alpha=-LR * 0.2)
        out[a:b] = w[a:b]
        return [w, out]
    out = torch.empty(s["x"].shape, dtype=torch.float64, device=s["x"].device)
    for i in range(c["batch"]):
        x = s["x"][i].double()
        x /= torch.linalg.matrix_norm(x) + NS_EPS
        wide = c["rows"] <= c["cols"]
        for _ in range(NS_STEPS):
            gram = torch.einsum("ik,jk->ij", x, x) if wide else torch.einsum("ki,kj->ij", x, x)
            poly = NS[2] * gram  # Horner's rule: a + (b + c A) A
            poly.diagonal().add_(NS[1])
            poly = poly @ gram
            poly.diagonal().add_(NS[0])
            x = poly @ x if wide else x @ poly
        out[i] = x
    return out
