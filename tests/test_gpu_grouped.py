"""Products grouped by expert and the expert MLP's training passes on the GPU,
against the definitions in 64 bits.

Tolerances.  A product of two bf16 values is exact in fp32, so a sum of n of
them is off by at most n * V * sum |terms| with V = 2^-23 (V, not 2^-24: the
matrix unit may truncate), plus half a step of the output's type (bf16 2^-8,
fp32 2^-24, relative).  s = sigmoid(g) from the hardware's exponential of
g * log2(e), an addition and a division is off by at most (|g| + 6) V
relative.  From there:

  a  = g s u                 rel. (|g| + 8) V, plus the sums' errors through |da/dg| <= 1.1 |u| and |da/du| = |g| s
  dg = da u s (1 + g (1-s))  |da u s| ((|g| + 10) V (1 + |g|) (1 + s)), plus the sum's error times the factor
  du = da g s                rel. (|g| + 8) V, plus the sum's error times |g s|

each then rounded to bf16 (2^-8), and these errors pass through the next
product's absolute values."""
import pytest
import torch

from combine_routing_preprocess_amd import Dispatcher
from gpu_util import DEV, log

pytestmark = pytest.mark.gpu
BF, F32, F64 = torch.bfloat16, torch.float32, torch.float64
V = 2.0 ** -23
HALF = {BF: 2.0 ** -8, F32: 2.0 ** -24}


class Case:
    """Rows of given counts per expert (top-1 routing of shuffled tokens); rows that hold no copy are NaN."""

    def __init__(self, counts, H=64, pad=1, seed=0, capacity=None, out_rows=0, extra_empty=3):
        self.g = torch.Generator().manual_seed(seed)
        idx = torch.cat([torch.full((c,), e) for e, c in enumerate(counts)] + [torch.full((extra_empty,), -1)])
        idx = idx[torch.randperm(len(idx), generator=self.g)].to(torch.int32)[:, None].contiguous()
        self.E = len(counts)
        self.d = Dispatcher(len(idx), H, self.E, 1, route_fmt="dense_i32", pad_multiple=pad, capacity=capacity,
                            out_rows=out_rows, device=DEV)
        self.d.preprocess(idx.to(DEV))
        torch.cuda.synchronize()
        self.R = self.d.R
        off, kept = self.d.seg_off.tolist(), self.d.kept.tolist()
        self.rows_of = [torch.arange(o, min(o + k, self.R)) if o < self.R else torch.arange(0)
                        for o, k in zip(off[:-1], kept)]
        self.live = torch.zeros(self.R, dtype=torch.bool)
        for r in self.rows_of:
            self.live[r] = True

    def rows(self, width, std=1.0):
        t = (torch.randn(self.R, width, generator=self.g) * std).to(BF)
        t[~self.live] = float("nan")
        return t

    def weight(self, n, m, std=None):
        return (torch.randn(self.E, n, m, generator=self.g) * (std or m ** -0.5)).to(BF)


def _within(got, want, tol, what):
    """tol: bound of the error before the rounding to got's type."""
    got = got.double().cpu()
    tol = tol + HALF[BF if what[1] == BF else F32] * (want.abs() + tol) + 1e-37
    bad = ~((got - want).abs() <= tol)
    assert not bool(bad.any()), (what, int(bad.sum()), float(((got - want).abs() / tol).nan_to_num(nan=1e9).max()),
                                 bad.nonzero()[:4].tolist())


def _product(x, w):
    """x @ w and the bound of its fp32 sums' error, in 64 bits."""
    return x @ w, x.shape[1] * V * (x.abs() @ w.abs())


COUNTS = [[1], [0, 0, 5], [33, 1, 0, 128, 129], [300, 7, 64], [0, 257, 0, 2, 511], [16] * 9, [0, 0]]
SIZES = [(8, 8), (64, 128), (72, 40), (264, 1016), (520, 256), (1032, 136)]


@pytest.mark.parametrize("transpose", [False, True])
@pytest.mark.parametrize("N,M", SIZES)
@pytest.mark.parametrize("ci", range(len(COUNTS)))
def test_product(ci, N, M, transpose):
    log("grouped product", COUNTS[ci], N, M, transpose)
    c = Case(COUNTS[ci], pad=(1, 4, 16)[ci % 3], seed=ci + N)
    x, w = c.rows(N if transpose else M), c.weight(N, M)
    out = torch.full((c.R, M if transpose else N), 7.0, dtype=BF, device=DEV)
    got = c.d.grouped_product(x.to(DEV), w.to(DEV), transpose=transpose, out=out)
    torch.cuda.synchronize()
    assert got is out
    for e, r in enumerate(c.rows_of):
        we = w[e].double()
        want, tol = _product(x[r].double(), we if transpose else we.T)
        _within(got[r.to(DEV)], want, tol, ("product", BF, e))
    assert bool((got[~c.live.to(DEV)] == 7.0).all())          # rows without a copy are left as they were


@pytest.mark.parametrize("out_dtype", [BF, F32])
@pytest.mark.parametrize("accumulate", [False, True])
@pytest.mark.parametrize("N,M", SIZES)
@pytest.mark.parametrize("ci", range(len(COUNTS)))
def test_weight_grad(ci, N, M, out_dtype, accumulate):
    log("grouped weight grad", COUNTS[ci], N, M, out_dtype, accumulate)
    c = Case(COUNTS[ci], pad=(4, 1, 16)[ci % 3], seed=100 + ci + M)
    g, x = c.rows(N), c.rows(M)
    before = (torch.randn(c.E, N, M, generator=c.g) * 4).to(out_dtype)
    out = before.clone().to(DEV)
    c.d.grouped_weight_grad(g.to(DEV), x.to(DEV), out=out, accumulate=accumulate)
    torch.cuda.synchronize()
    for e, r in enumerate(c.rows_of):
        want, tol = _product(g[r].double().T, x[r].double())
        if accumulate:
            want = want + before[e].double()
            tol = tol + 2.0 ** -24 * (want.abs() + tol)
        _within(out[e], want, tol, ("weight grad", out_dtype, e))


def _swiglu_bounds(g, u, dg, du):
    """a = silu(g) u and its bound where g and u are off by dg and du."""
    s = torch.sigmoid(g)
    a = g * s * u
    return a, 1.1 * (u.abs() + du) * dg + (g * s).abs() * du + (g.abs() + 8) * V * a.abs()


def _keep_reference(c, x, w1, w2, F, e):
    r = c.rows_of[e]
    h, dh = _product(x[r].double(), w1[e].double().T)
    a, da = _swiglu_bounds(h[:, :F], h[:, F:], dh[:, :F], dh[:, F:])
    da = da + 2.0 ** -8 * (a.abs() + da)                      # a in bf16
    y, dy = _product(a, w2[e].double().T)
    return h, dh, y, dy + da @ w2[e].double().abs().T


MLP = [([33, 1, 0, 70], 64, 40), ([5, 300, 129], 264, 128), ([1], 8, 8), ([0, 64, 128, 3, 17], 136, 520),
       ([140, 0, 9], 512, 264)]


@pytest.mark.parametrize("counts,H,F", MLP)
def test_mlp_keep(counts, H, F):
    log("mlp keep", counts, H, F)
    c = Case(counts, H=H, pad=4, seed=H + F)
    x, w1, w2 = c.rows(H), c.weight(2 * F, H), c.weight(H, F)
    h = torch.full((c.R, 2 * F), 7.0, dtype=BF, device=DEV)
    out = torch.full((c.R, H), 7.0, dtype=BF, device=DEV)
    c.d.grouped_mlp_keep(x.to(DEV), w1.to(DEV), w2.to(DEV), h=h, out=out)
    torch.cuda.synchronize()
    for e, r in enumerate(c.rows_of):
        hw, dh, y, dy = _keep_reference(c, x, w1, w2, F, e)
        _within(h[r.to(DEV)], hw, dh, ("h", BF, e))
        _within(out[r.to(DEV)], y, dy, ("y", BF, e))
    dead = ~c.live.to(DEV)
    assert bool((h[dead] == 7.0).all()) and bool((out[dead] == 7.0).all())


def _backward_reference(gy, x, h, w1, w2, F):
    """(value, bound before its last rounding) of grad_perm, grad_w1, grad_w2 for one expert."""
    gy, x, h, w1, w2 = (t.double() for t in (gy, x, h, w1, w2))
    g, u = h[:, :F], h[:, F:]
    s = torch.sigmoid(g)
    da, dda = _product(gy, w2)
    f = u * s * (1 + g * (1 - s))
    hg, hu, a = da * f, da * g * s, g * s * u
    tg = f.abs() * dda + (da.abs() + dda) * (u * s).abs() * (g.abs() + 10) * V * (1 + g.abs()) * (1 + s)
    tu = (g * s).abs() * (dda + (da.abs() + dda) * (g.abs() + 8) * V)
    gh, tgh = torch.cat((hg, hu), 1), torch.cat((tg, tu), 1)
    tgh = tgh + 2.0 ** -8 * (gh.abs() + tgh)
    ta = (g.abs() + 8) * V * a.abs()
    ta = ta + 2.0 ** -8 * (a.abs() + ta)
    gx, tx = _product(gh, w1)
    g1, t1 = _product(gh.T, x)
    g2, t2 = _product(gy.T, a)
    return (gx, tx + tgh @ w1.abs()), (g1, t1 + tgh.T @ x.abs()), (g2, t2 + gy.abs().T @ ta)


@pytest.mark.parametrize("dtype,accumulate", [(BF, False), (F32, False), (F32, True)])
@pytest.mark.parametrize("counts,H,F", MLP)
def test_mlp_backward(counts, H, F, dtype, accumulate):
    log("mlp backward", counts, H, F, dtype, accumulate)
    c = Case(counts, H=H, pad=4, seed=7 + H + F)
    x, gy, h, w1, w2 = c.rows(H), c.rows(H), c.rows(2 * F), c.weight(2 * F, H), c.weight(H, F)
    h[c.rows_of[-1][:1]] *= 20                                  # saturated gates
    out = torch.full((c.R, H), 7.0, dtype=BF, device=DEV)
    b1 = torch.randn(w1.shape, generator=c.g).to(dtype)
    b2 = torch.randn(w2.shape, generator=c.g).to(dtype)
    g1, g2 = b1.clone().to(DEV), b2.clone().to(DEV)
    got = c.d.grouped_mlp_backward(gy.to(DEV), x.to(DEV), h.to(DEV), w1.to(DEV), w2.to(DEV), grad_perm=out,
                                   grad_w1=g1, grad_w2=g2, accumulate=accumulate)
    torch.cuda.synchronize()
    assert got[0] is out and got[1] is g1 and got[2] is g2
    for e, r in enumerate(c.rows_of):
        rx, r1, r2 = _backward_reference(gy[r], x[r], h[r], w1[e], w2[e], F)
        _within(out[r.to(DEV)], *rx, ("grad_perm", BF, e))
        for name, t, before, (want, tol) in (("grad_w1", g1, b1, r1), ("grad_w2", g2, b2, r2)):
            if accumulate:
                want = want + before[e].double()
                tol = tol + 2.0 ** -24 * (want.abs() + tol)
            _within(t[e], want, tol, (name, dtype, e))
    assert bool((out[~c.live.to(DEV)] == 7.0).all())


def test_mlp_backward_against_differences():
    """The change of sum(y * gy) along random directions of x, w1 and w2, in 64 bits by central differences, against
    the kernels' gradients; each gradient may be off by its bound, summed over the direction's absolute values.  The
    differences' own error: relative 1e-6 of the largest term (step 1e-4, third derivatives of order one)."""
    counts, H, F = [40, 0, 25], 72, 56
    c = Case(counts, H=H, seed=3)
    x, gy, w1, w2 = c.rows(H), c.rows(H), c.weight(2 * F, H), c.weight(H, F)
    hd = torch.zeros(c.R, 2 * F)
    for e, r in enumerate(c.rows_of):
        hd[r] = (x[r].double() @ w1[e].double().T).float()
    h = hd.to(BF)                                               # what the forward keeps: h rounded
    gx, g1, g2 = (t.double().cpu() for t in c.d.grouped_mlp_backward(*(t.to(DEV) for t in (gy, x, h, w1, w2)),
                                                                     grad_dtype=F32))

    def loss(dx, d1, d2, t):
        total = 0.0
        for e, r in enumerate(c.rows_of):
            # h's rounding is held fixed: the gradient is that of the function around the kept h
            w = w1[e].double()
            hh = h[r].double() + ((x[r].double() + t * dx[r]) @ (w + t * d1[e]).T - x[r].double() @ w.T)
            a = torch.sigmoid(hh[:, :F]) * hh[:, :F] * hh[:, F:]
            total = total + ((a @ (w2[e].double() + t * d2[e]).T) * gy[r].double()).sum()
        return total

    bounds = [_backward_reference(gy[r], x[r], h[r], w1[e], w2[e], F) for e, r in enumerate(c.rows_of)]
    zero = [torch.zeros(c.R, H, dtype=F64), torch.zeros(w1.shape, dtype=F64), torch.zeros(w2.shape, dtype=F64)]
    for k in range(3):
        dirs = [z.clone() for z in zero]
        dirs[k] = torch.randn(dirs[k].shape, generator=c.g, dtype=F64)
        slope = (loss(*dirs, 1e-4) - loss(*dirs, -1e-4)) / 2e-4
        got, allowed, size = 0.0, 0.0, 0.0
        for e, r in enumerate(c.rows_of):
            grad, v = (gx[r], dirs[0][r]) if k == 0 else (g1[e], dirs[1][e]) if k == 1 else (g2[e], dirs[2][e])
            want, tol = bounds[e][k]
            got = got + (grad * v).sum()
            allowed += float(((tol + (2.0 ** -8 if k == 0 else 2.0 ** -24) * (want.abs() + tol)) * v.abs()).sum())
            size += float((want * v).abs().sum())
        assert abs(float(got - slope)) <= allowed + 1e-6 * size, (k, float(got), float(slope), allowed)


def test_fused_backward_is_its_parts():
    """grouped_mlp_backward's products are those of the single calls, bit for bit."""
    counts, H, F = [33, 0, 140], 136, 72
    c = Case(counts, H=H, pad=4, seed=11)
    dv = [t.to(DEV) for t in (c.rows(H), c.rows(H), c.rows(2 * F), c.weight(2 * F, H), c.weight(H, F))]
    gy, x, h, w1, w2 = dv
    scratch = c.d.alloc_mlp_backward_scratch(F)
    gx, g1, g2 = c.d.grouped_mlp_backward(*dv, scratch=scratch)
    torch.cuda.synchronize()
    gh = scratch[:c.R * 4 * F].view(BF).view(c.R, 2 * F)
    at = (c.R * 4 * F + 255) // 256 * 256
    act = scratch[at:at + c.R * 2 * F].view(BF).view(c.R, F)
    live = c.live.to(DEV)
    assert torch.equal(gx[live], c.d.grouped_product(gh, w1, transpose=True)[live])
    assert torch.equal(g1, c.d.grouped_weight_grad(gh, x)) and torch.equal(g2, c.d.grouped_weight_grad(gy, act))
    only_x = c.d.grouped_mlp_backward(*dv, want_weights=False)
    only_w = c.d.grouped_mlp_backward(*dv, want_rows=False)
    assert only_x[1] is None and only_x[2] is None and only_w[0] is None
    assert torch.equal(only_x[0][live], gx[live]) and torch.equal(only_w[1], g1) and torch.equal(only_w[2], g2)


def test_capacity_and_out_rows_bound_the_rows():
    """Copies over capacity and rows beyond out_rows take no part."""
    c = Case([50, 3, 90], capacity=40, seed=5)
    assert [len(r) for r in c.rows_of] == [40, 3, 40]
    t = Case([50, 3, 90], out_rows=100, seed=6)
    assert sum(len(r) for r in t.rows_of) == 100
    for k in (c, t):
        x, w, g = k.rows(40), k.weight(72, 40), k.rows(72)
        y = k.d.grouped_product(x.to(DEV), w.to(DEV))
        gw = k.d.grouped_weight_grad(g.to(DEV), x.to(DEV), out_dtype=F32)
        for e, r in enumerate(k.rows_of):
            _within(y[r.to(DEV)], *_product(x[r].double(), w[e].double().T), ("y", BF, e))
            _within(gw[e], *_product(g[r].double().T, x[r].double()), ("gw", F32, e))


def test_non_finite_values_stay_in_their_row_and_expert():
    c = Case([70, 40, 5], seed=9)
    x, w, g = c.rows(136), c.weight(72, 136), c.rows(72)
    bad = int(c.rows_of[1][3])
    x[bad, 7] = float("inf")
    y = c.d.grouped_product(x.to(DEV), w.to(DEV)).cpu()
    gw = c.d.grouped_weight_grad(g.to(DEV), x.to(DEV)).cpu()
    ok = c.live.clone()
    ok[bad] = False
    assert bool(y[ok].isfinite().all()) and not bool(y[bad].isfinite().any())
    assert bool(gw[0].isfinite().all()) and bool(gw[2].isfinite().all())
    assert bool(gw[1][:, :7].isfinite().all()) and bool(gw[1][:, 8:].isfinite().all())
    assert not bool(gw[1][:, 7].isfinite().any())


def test_calls_repeat_bit_for_bit_on_two_streams_and_in_graphs():
    counts, H, F = [200, 0, 31, 129], 264, 136
    c = Case(counts, H=H, pad=4, seed=13)
    dv = [t.to(DEV) for t in (c.rows(H), c.rows(H), c.weight(2 * F, H), c.weight(H, F))]
    x, gy, w1, w2 = dv
    torch.cuda.synchronize()

    def step(bufs):
        y, h = c.d.grouped_mlp_keep(x, w1, w2, h=bufs["h"], scratch=bufs["s"], out=bufs["y"])
        c.d.grouped_mlp_backward(gy, x, h, w1, w2, grad_perm=bufs["gx"], grad_w1=bufs["g1"], grad_w2=bufs["g2"],
                                 scratch=bufs["b"])

    def room():
        new = lambda *s: torch.zeros(s, dtype=BF, device=DEV)
        return dict(h=new(c.R, 2 * F), y=new(c.R, H), gx=new(c.R, H), g1=new(*w1.shape), g2=new(*w2.shape),
                    s=c.d.alloc_mlp_scratch(F), b=c.d.alloc_mlp_backward_scratch(F))

    names = ("h", "y", "gx", "g1", "g2")
    want = room()
    step(want)
    torch.cuda.synchronize()
    a, b = room(), room()
    sa, sb = torch.cuda.Stream(), torch.cuda.Stream()
    sa.wait_stream(torch.cuda.current_stream())
    sb.wait_stream(torch.cuda.current_stream())
    for st, bufs in ((sa, a), (sb, b)):
        with torch.cuda.stream(st):
            step(bufs)
    torch.cuda.synchronize()
    for n in names:
        assert torch.equal(a[n], want[n]) and torch.equal(b[n], want[n]), n
    graph, gb = torch.cuda.CUDAGraph(), room()
    with torch.cuda.graph(graph):
        step(gb)
    for _ in range(3):
        for n in names:
            gb[n].fill_(0 if n != "g1" else 5)
        graph.replay()
        torch.cuda.synchronize()
        for n in names:
            assert torch.equal(gb[n], want[n]), n
        step(a)                                                # eager work between the replays
        torch.cuda.synchronize()


def test_weights_beyond_32_bit_offsets():
    """E * N * M = 2.3e9 elements: the last expert's offsets pass 2^31 elements and 2^32 bytes."""
    E, N, M = 34, 8200, 8200
    counts = [0] * (E - 2) + [3, 40]
    c = Case(counts, seed=21)
    w = torch.zeros((E, N, M), dtype=BF, device=DEV)
    w[E - 1].normal_(0, M ** -0.5)
    x, g = c.rows(M).to(DEV), c.rows(N).to(DEV)
    y = c.d.grouped_product(x, w)
    yt = c.d.grouped_product(g, w, transpose=True)
    gw = c.d.grouped_weight_grad(g, x, out=w.clone())
    torch.cuda.synchronize()
    r = c.rows_of[E - 1].to(DEV)
    wd, xd, gd = w[E - 1].double(), x[r].double(), g[r].double()
    for got, (want, tol) in ((y[r], _product(xd, wd.T)), (yt[r], _product(gd, wd)), (gw[E - 1], _product(gd.T, xd))):
        _within(got, want.cpu(), tol.cpu(), ("large", BF))
    assert bool((y[c.rows_of[E - 2].to(DEV)] == 0).all()) and bool((gw[0] == 0).all())


def test_many_experts():
    """More experts than a workgroup has threads, most of them empty."""
    counts = [(i * 7) % 5 if i % 3 == 0 else 0 for i in range(1000)] + [260]
    c = Case(counts, seed=23)
    x, w, g = c.rows(40), c.weight(24, 40), c.rows(24)
    y = c.d.grouped_product(x.to(DEV), w.to(DEV)).cpu()
    gw = c.d.grouped_weight_grad(g.to(DEV), x.to(DEV)).cpu()
    for e, r in enumerate(c.rows_of):
        _within(y[r], *_product(x[r].double(), w[e].double().T), ("y", BF, e))
        _within(gw[e], *_product(g[r].double().T, x[r].double()), ("gw", BF, e))
