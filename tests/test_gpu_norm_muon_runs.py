"""The norms and the orthogonalised step as a program runs them: one after the other
without synchronisation, on two streams at once, captured and replayed on new inputs, and
on matrices whose rows lie further apart than 32 bits count."""
import pytest
import torch

from tests import dense_plain as dp
from tests import norm_plain as npl

pytestmark = pytest.mark.gpu
BF, F32 = torch.bfloat16, torch.float32


class Unit:
    """Norm, product, gradient of both: the buffers of one pass.  dt: of the residual stream."""

    def __init__(self, zlib, rows, d, n, seed, dt=BF):
        g = torch.Generator(device="cuda").manual_seed(seed)
        new = lambda *s, dt=BF: torch.empty(*s, dtype=dt, device="cuda")   # noqa: E731
        rnd = lambda *s: torch.randn(*s, generator=g, device="cuda").to(BF)   # noqa: E731
        self.z, self.x, self.r, self.w, self.gamma, self.beta, self.dy = zlib, rnd(rows, d).to(dt), rnd(rows, d).to(dt), rnd(n, d) * 0.05, 1 + rnd(d) * 0.1, rnd(d), rnd(rows, n)
        self.s, self.h, self.y, self.dh, self.dx = new(rows, d, dt=dt), new(rows, d), new(rows, n), new(rows, d), new(rows, d, dt=dt)
        self.mean, self.rstd, self.dg, self.db, self.dw = new(rows, dt=F32), new(rows, dt=F32), new(d), new(d), new(n, d)
        self.ws = new(zlib.zero_layer_norm_grad_workspace(rows, d), dt=torch.uint8)
        self.o, self.ows = new(n, d), new(zlib.zero_orthogonalize_workspace(1, n, d), dt=torch.uint8)

    def run(self):
        z = self.z
        z.zero_layer_norm(self.x, self.h, self.gamma, self.beta, residual=self.r, sum=self.s, mean=self.mean, rstd=self.rstd)
        z.zero_linear(self.h, self.w, self.y)
        z.zero_linear_grad_weight(self.dy, self.h, self.dw)
        z.zero_linear_grad_input(self.dy, self.w, self.dh)
        z.zero_layer_norm_grad(self.dh, self.s, self.mean, self.rstd, self.dx, self.gamma, residual=self.r, dgamma=self.dg, dbeta=self.db,
                               workspace=self.ws)
        z.zero_orthogonalize(self.dw, self.o, workspace=self.ows)

    def out(self):
        return [t.clone() for t in (self.s, self.h, self.y, self.dw, self.dh, self.dx, self.dg, self.db, self.o, self.mean, self.rstd)]


def test_chain_against_64_bits(zlib, cuda_device):
    u = Unit(zlib, 300, 200, 264, 1)
    u.run()
    zlib.zero_status_check()
    # each call on what the calls before it left, within its own tolerances
    h = u.s.cpu().double()
    ref, mean, rstd, xhat = npl.layer_norm(h, u.gamma.cpu().double(), u.beta.cpu().double(), 1e-5)
    dp.close(u.h, ref, 2.0 ** -17 * (xhat.abs() + 1) * u.gamma.cpu().double().abs() + dp.eps_out(BF) * ref.abs() + 2.0 ** -23 * u.beta.cpu().double().abs())
    dx, dg, db, mag, mg, mb = npl.layer_norm_grad(u.dh.cpu().double(), h, u.mean.cpu().double(), u.rstd.cpu().double(), u.gamma.cpu().double())
    r = u.r.cpu().double()
    dp.close(u.dx, dx + r, 2.0 ** -17 * mag + 2.0 ** -23 * (dx.abs() + r.abs()) + dp.eps_out(BF) * (dx + r).abs())
    for got, want, m in ((u.dg, dg, mg), (u.db, db, mb)):
        dp.close(got, want, 364 * 2.0 ** -24 * m + dp.eps_out(BF) * want.abs())
    from tests.test_gpu_orthogonalize import _close
    _close(u.o, u.dw.cpu())


@pytest.mark.parametrize("dt", [BF, F32])
def test_two_streams_at_once(zlib, cuda_device, dt):
    units = [Unit(zlib, 500 + 77 * i, 320, 200, i, dt) for i in range(2)]
    refs = []
    for u in units:
        u.run()
        torch.cuda.synchronize()
        refs.append(u.out())
    streams = [torch.cuda.Stream() for _ in units]
    torch.cuda.synchronize()
    for _ in range(8):
        for u, s in zip(units, streams):
            with torch.cuda.stream(s):
                u.run()
    torch.cuda.synchronize()
    for u, ref in zip(units, refs):
        assert all(torch.equal(a, b) for a, b in zip(u.out(), ref))
    # a stream given by hand
    units[0].z.zero_layer_norm(units[0].x, units[0].h, units[0].gamma, units[0].beta, residual=units[0].r, sum=units[0].s, stream=streams[1])
    torch.cuda.synchronize()
    assert torch.equal(units[0].h, refs[0][1])


@pytest.mark.parametrize("dt", [BF, F32])
@pytest.mark.parametrize("d", [256, 257])
def test_captured_and_replayed(zlib, cuda_device, d, dt):
    u, other = Unit(zlib, 700, d, 129, 3, dt), Unit(zlib, 700, d, 129, 4, dt)
    want = []
    for v in (u, other):
        v.run()
        torch.cuda.synchronize()
        want.append(v.out())
    inputs = [[t.clone() for t in (v.x, v.r, v.w, v.gamma, v.beta, v.dy)] for v in (u, other)]
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        u.run()
    for i in (1, 0, 1, 1, 0):
        for t, new in zip((u.x, u.r, u.w, u.gamma, u.beta, u.dy), inputs[i]):
            t.copy_(new)
        graph.replay()
        assert all(torch.equal(a, b) for a, b in zip(u.out(), want[i])), i
    zlib.zero_status_check()


def test_rows_and_matrices_far_apart(zlib, cuda_device):
    """Rows 2^31 + 8 elements apart, matrices 2^32 + 1: offsets that pass 32 bits."""
    g = torch.Generator().manual_seed(0)
    ld = 2 ** 31 + 8
    buf = torch.zeros(2 * ld + 4096, dtype=BF, device="cuda")
    for cols in (1600, 1601):
        x = buf.as_strided((3, cols), (ld, 1))
        host = torch.randn(3, cols, generator=g).to(BF)
        x.copy_(host)
        close_by = host.cuda()
        y, ref = torch.empty(3, cols, dtype=BF, device="cuda"), torch.empty(3, cols, dtype=BF, device="cuda")
        mean, rstd = torch.empty(3, device="cuda"), torch.empty(3, device="cuda")
        zlib.zero_layer_norm(x, y, mean=mean, rstd=rstd)
        zlib.zero_layer_norm(close_by, ref)
        assert torch.equal(y, ref)
        zlib.zero_layer_norm(close_by, x)   # and written there
        assert torch.equal(x, ref)
        x.copy_(host)
        dy = torch.randn(3, cols, generator=g).to(BF).cuda()
        zlib.zero_layer_norm_grad(dy, x, mean, rstd, y)
        zlib.zero_layer_norm_grad(dy, close_by, mean, rstd, ref)
        assert torch.equal(y, ref)
    ws = torch.empty(zlib.zero_orthogonalize_workspace(2, 3, 700), dtype=torch.uint8, device="cuda")
    host = torch.randn(2, 3, 700, generator=g).to(BF)
    for far in (buf.as_strided((2, 3, 700), (2 ** 32 + 1, 701, 1)), buf.as_strided((2, 2, 700), (701, ld, 1))):
        b, rows, cols = far.shape
        near = host[:, :rows].contiguous().cuda()
        far.copy_(near)
        y, ref = torch.empty_like(near), torch.empty_like(near)
        zlib.zero_orthogonalize(far, y, workspace=ws)
        zlib.zero_orthogonalize(near, ref, workspace=ws)
        assert torch.equal(y, ref)
        if b == 2 and rows == 3:
            zlib.zero_orthogonalize(far, far, workspace=ws)
            assert torch.equal(far, ref)
