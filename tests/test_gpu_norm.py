"""Layer norm and its backward pass on the GPU against the formulas in 64 bits.

Tolerances, with u = 2^-24 (an fp32 rounding) and n the depth of a row's sums
(a lane adds up to 8 * NC elements, 6 butterfly levels, up to 16 parts, plus
the few operations around them): a sum of H terms is off by at most
n * u * sum |terms|.  The centred elements and their square sum carry no
rounding of the row's offset (the mean is held as m + delta), so

  y      (n + 16) u (|xh| + 1) |w| + 4 u |b|                   + half a step of y's type
  gx     u r ((4 + n) mean|g| + 4 |g| + (n + 8) |xh| mean|g xh|) + half a step of gx's type
  gw, gb (rows per workgroup + groups + partials / 8 + 16) u sum |terms|

with xh and r taken from the fp32 mean and rstd that the call is given in the
backward pass (their own rounding is an input, not an error)."""
import numpy as np
import pytest
import torch

from combine_routing_preprocess_amd import layer_norm, layer_norm_backward
from combine_routing_preprocess_amd import _abi as A
from gpu_util import DEV, log

pytestmark = pytest.mark.gpu
U = 2.0 ** -24
HALF = {torch.bfloat16: 2.0 ** -8, torch.float32: 2.0 ** -24}
BF, F32 = torch.bfloat16, torch.float32


def _depth(H):
    groups = (H + 511) // 512
    nc = 1 if groups <= 16 else 2 if groups <= 32 else 4
    return 8 * nc + 6 + 16


def _inputs(T, H, xt, wt, seed, offset=0.0, bias=True, weight=True):
    g = torch.Generator().manual_seed(seed)
    x = (torch.randn(T, H, generator=g) * torch.exp(0.5 * torch.randn(T, 1, generator=g)) + offset).to(xt)
    w = (1.0 + 0.3 * torch.randn(H, generator=g)).to(wt) if weight else None
    b = (0.2 * torch.randn(H, generator=g)).to(wt) if bias else None
    return x, w, b


def _dev(*ts):
    return [None if t is None else t.to(DEV) for t in ts]


def _f64(t, fill, H):
    return torch.full((H,), fill, dtype=torch.float64) if t is None else t.double()


def _check_forward(x, w, b, eps, y, mean, rstd):
    T, H = x.shape
    xd, wd, bd = x.double(), _f64(w, 1.0, H), _f64(b, 0.0, H)
    mu = xd.mean(1)
    d = xd - mu[:, None]
    r = 1.0 / torch.sqrt((d * d).mean(1) + eps)
    xh = d * r[:, None]
    n = _depth(H)
    want = xh * wd + bd
    tol = (n + 16) * U * (xh.abs() + 1) * wd.abs() + 4 * U * bd.abs()
    tol = tol + HALF[y.dtype] * (want.abs() + tol)
    err = (y.double().cpu() - want).abs()
    assert bool((err <= tol).all()), (float((err / tol).max()), err.argmax())
    sd = d.abs().mean(1)
    assert bool(((mean.double().cpu() - mu).abs() <= U * mu.abs() + n * U * sd + 1e-300).all())
    assert bool(((rstd.double().cpu() - r).abs() <= (n + 8) * U * r).all())


SHAPES = [(1, 1), (1, 7168), (3, 7), (5, 64), (17, 130), (9, 513), (64, 1000), (70, 4097), (300, 1024), (33, 8192),
          (6, 8200), (2, 16385), (2, 32768), (1030, 520), (0, 64)]


@pytest.mark.parametrize("xt,yt,wt", [(BF, BF, BF), (F32, BF, F32), (F32, F32, F32), (BF, F32, BF)])
@pytest.mark.parametrize("T,H", SHAPES)
def test_forward(T, H, xt, yt, wt):
    log("layer norm", T, H, xt, yt, wt)
    x, w, b = _inputs(T, H, xt, wt, 100 + T + H)
    xd, wd, bd = _dev(x, w, b)
    y, mean, rstd = layer_norm(xd, wd, bd, 1e-5, out_dtype=yt)
    torch.cuda.synchronize()
    assert y.dtype == yt and tuple(y.shape) == (T, H)
    _check_forward(x, w, b, 1e-5, y, mean, rstd)


@pytest.mark.parametrize("weight,bias", [(True, False), (False, True), (False, False)])
def test_forward_without_parameters(weight, bias):
    x, w, b = _inputs(37, 776, F32, F32, 5, weight=weight, bias=bias)
    xd, wd, bd = _dev(x, w, b)
    y, mean, rstd = layer_norm(xd, wd, bd)
    _check_forward(x, w, b, 1e-5, y, mean, rstd)


@pytest.mark.parametrize("H", [96, 1537, 7168, 20000])
def test_forward_offset_far_larger_than_spread(H):
    x, w, b = _inputs(11, H, F32, F32, 6, offset=1.0e4)
    xd, wd, bd = _dev(x, w, b)
    y, mean, rstd = layer_norm(xd, wd, bd)
    _check_forward(x, w, b, 1e-5, y, mean, rstd)


def test_forward_writes_only_its_rows_and_columns():
    T, H = 13, 77
    x, w, b = _inputs(T, H, BF, F32, 7)
    xd, wd, bd = _dev(x, w, b)
    room = torch.full(((T + 2) * H + 64,), 3.0, dtype=BF, device=DEV)
    out = room[32:32 + T * H].view(T, H)          # 64 bytes in: 16-byte aligned
    layer_norm(xd, wd, bd, out=out)
    torch.cuda.synchronize()
    assert bool((room[:32] == 3.0).all()) and bool((room[32 + T * H:] == 3.0).all())


def test_constant_rows_and_non_finite_rows():
    H = 640
    x = torch.randn(6, H, generator=torch.Generator().manual_seed(8))
    x[1] = 2.5            # no spread: xh = 0, rstd = 1 / sqrt(eps)
    x[2, 100] = float("nan")
    x[3, 639] = float("inf")
    y, mean, rstd = layer_norm(x.to(DEV))
    y, mean, rstd = y.cpu(), mean.cpu(), rstd.cpu()
    assert bool((y[1] == 0).all()) and abs(float(rstd[1]) * 1e-5 ** 0.5 - 1) < 1e-6
    assert bool(torch.isnan(y[2]).all()) and bool(torch.isnan(rstd[2])) and bool(torch.isnan(y[3]).all())
    keep = [0, 4, 5]      # the other rows are not touched by these
    _check_forward(x[keep], None, None, 1e-5, y[keep], mean[keep], rstd[keep])


def _check_backward(x, w, gy, mean, rstd, gx, gw, gb):
    T, H = x.shape
    m, r = mean.double().cpu()[:, None], rstd.double().cpu()[:, None]
    xh = (x.double() - m) * r
    gyd = gy.double()
    g = gyd * _f64(w, 1.0, H)
    want = r * (g - g.mean(1, keepdim=True) - xh * (g * xh).mean(1, keepdim=True))
    n = _depth(H)
    tol = U * r * ((4 + n) * g.abs().mean(1, keepdim=True) + 4 * g.abs()
                   + (n + 8) * xh.abs() * (g * xh).abs().mean(1, keepdim=True))
    tol = tol + HALF[gx.dtype] * (want.abs() + tol)
    err = (gx.double().cpu() - want).abs()
    assert bool((err <= tol).all()), float((err / tol).max())
    if gw is None:
        return
    nsum = T / 256 + 16 + 32 + 16
    for got, terms in ((gw, gyd * xh), (gb, gyd)):
        err = (got.double().cpu() - terms.sum(0)).abs()
        assert bool((err <= nsum * U * terms.abs().sum(0)).all()), float(err.max())


@pytest.mark.parametrize("xt,yt,wt", [(BF, BF, F32), (F32, BF, BF), (F32, F32, F32), (BF, F32, F32)])
@pytest.mark.parametrize("T,H", SHAPES + [(5000, 96), (700, 2056)])
def test_backward(T, H, xt, yt, wt):
    log("layer norm backward", T, H, xt, yt, wt)
    x, w, b = _inputs(T, H, xt, wt, 200 + T + H)
    gy = torch.randn(T, H, generator=torch.Generator().manual_seed(T * 7 + H)).to(yt)
    xd, wd, bd, gd = _dev(x, w, b, gy)
    _, mean, rstd = layer_norm(xd, wd, bd)
    gx, gw, gb = layer_norm_backward(gd, xd, mean, rstd, wd)
    torch.cuda.synchronize()
    assert gx.dtype == xt
    _check_backward(x, w, gy, mean, rstd, gx, gw, gb)
    again = layer_norm_backward(gd, xd, mean, rstd, wd)      # fixed order: bit for bit
    for p, q in zip((gx, gw, gb), again):
        assert torch.equal(p, q)


def test_backward_without_weight_and_parameter_gradients():
    x, _, _ = _inputs(40, 300, BF, F32, 9, weight=False, bias=False)
    gy = torch.randn(40, 300, generator=torch.Generator().manual_seed(10))
    xd, gd = _dev(x, gy)
    _, mean, rstd = layer_norm(xd)
    gx, gw, gb = layer_norm_backward(gd, xd, mean, rstd, want_params=False)
    assert gw is None and gb is None
    _check_backward(x, None, gy, mean, rstd, gx, None, None)


def test_backward_agrees_with_differences():
    """d/dt of sum(gy * norm(x + t v)) in 64 bits against <gx, v>, and the
    same for the parameters."""
    T, H = 4, 96
    x, w, b = _inputs(T, H, F32, F32, 11)
    g = torch.Generator().manual_seed(12)
    gy, v = torch.randn(T, H, generator=g), torch.randn(T, H, generator=g)
    vw, vb = torch.randn(H, generator=g), torch.randn(H, generator=g)

    def loss(t):
        xd = x.double() + t * v.double()
        d = xd - xd.mean(1, keepdim=True)
        y = d / torch.sqrt((d * d).mean(1, keepdim=True) + 1e-5) * (w.double() + t * vw.double()) \
            + b.double() + t * vb.double()
        return float((y * gy.double()).sum())

    xd, wd, bd, gd = _dev(x, w, b, gy)
    _, mean, rstd = layer_norm(xd, wd, bd)
    gx, gw, gb = (t.double().cpu() for t in layer_norm_backward(gd, xd, mean, rstd, wd))
    terms = [gx * v.double(), gw * vw.double(), gb * vb.double()]
    got = sum(float(t.sum()) for t in terms)
    size = sum(float(t.abs().sum()) for t in terms)
    step = 1e-5
    want = (loss(step) - loss(-step)) / (2 * step)
    # central differences: step^2 times a third derivative of the order of the
    # terms, plus 2^-52 |loss| / step; the kernel adds (n + 16) u of the terms
    assert abs(got - want) <= size * (100 * step ** 2 + 64 * U) + 2.0 ** -50 * abs(loss(0.0)) / step


def test_graph_replay_and_other_stream():
    T, H = 100, 1000
    x, w, b = _inputs(T, H, F32, F32, 13)
    gy = torch.randn(T, H, generator=torch.Generator().manual_seed(14)).to(BF)
    xd, wd, bd, gd = _dev(x, w, b, gy)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        first = layer_norm(xd, wd, bd, out_dtype=BF)
        second = layer_norm_backward(gd, xd, first[1], first[2], wd)
    torch.cuda.synchronize()
    _check_forward(x, w, b, 1e-5, *first)
    _check_backward(x, w, gy, first[1], first[2], *second)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        y, mean, rstd = layer_norm(xd, wd, bd, out_dtype=BF)
        grads = layer_norm_backward(gd, xd, mean, rstd, wd)
    for k in range(3):
        xd.copy_((x * (1 + k)).to(DEV))
        want = layer_norm(xd, wd, bd, out_dtype=BF)
        want_g = layer_norm_backward(gd, xd, want[1], want[2], wd)
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        for p, q in zip((y, mean, rstd) + tuple(grads), tuple(want) + tuple(want_g)):
            assert torch.equal(p, q)


def test_offsets_past_two_to_the_31_elements():
    T, H = 300_001, 7168
    x = torch.empty((T, H), dtype=BF, device=DEV)
    tail = _inputs(9, H, BF, F32, 15)[0]
    x[:8].zero_()
    x[-9:] = tail.to(DEV)
    y, mean, rstd = layer_norm(x, out=torch.empty_like(x))
    torch.cuda.synchronize()
    _check_forward(tail, None, None, 1e-5, y[-9:], mean[-9:], rstd[-9:])
    assert bool((y[:8] == 0).all())
