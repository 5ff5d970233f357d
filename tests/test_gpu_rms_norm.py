"""RMS norm with the residual's addition and 8-bit rows, and its backward pass,
on the GPU against the formulas in 64 bits.

Tolerances, with u = 2^-24 and n the most operations a term of a row's sum
passes through (a lane adds up to 8 * 4 elements, or H / 256 of them one by
one, 6 levels between lanes, up to 16 parts):  t = x + residual carries u |t|,
its mean square (n + 3) u relative, so

  rstd    (n / 2 + 8) u relative
  y       (n / 2 + 12) u |y|                                   + half a step of its type
  codes   |code * scale - y| <= half an e4m3 step of y (2^-4 |y|, or half the
          smallest subnormal, 2^-10 scale) + the error above + 2 u |y|
  scale   (n / 2 + 13) u relative
  grad    u (|grad_total| + r ((n + 8) |xh| mean|q xh| + 6 |q|) + 2 |grad|) + half a step
  weight  (rows that one lane adds + 256 + 16) u sum |terms|"""
import pytest
import torch

from combine_routing_preprocess_amd import Dispatcher, rms_norm, rms_norm_backward
from gpu_util import DEV, log

pytestmark = pytest.mark.gpu
U = 2.0 ** -24
HALF = {torch.bfloat16: 2.0 ** -8, torch.float32: 2.0 ** -24}
BF, F32 = torch.bfloat16, torch.float32


def _depth(H):
    return max(32, (H + 255) // 256) + 6 + 16


def _dev(*ts):
    return [None if t is None else t.to(DEV) for t in ts]


def _inputs(T, H, xt, rt, wt, seed):
    g = torch.Generator().manual_seed(seed)
    size = torch.exp(0.5 * torch.randn(T, 1, generator=g))
    x = (torch.randn(T, H, generator=g) * size).to(xt)
    r = None if rt is None else (torch.randn(T, H, generator=g) * size).to(rt)
    w = None if wt is None else (1 + 0.3 * torch.randn(H, generator=g)).to(wt)
    return x, r, w, g


def _reference(x, r, w, eps):
    t = x.double() if r is None else x.double() + r.double()
    rs = 1 / torch.sqrt((t * t).mean(1) + eps)
    y = t * rs[:, None]
    return t, rs, y if w is None else y * w.double()


def _check(got, x, r, w, eps):
    H = x.shape[1]
    t, rs, y = _reference(x, r, w, eps)
    n = _depth(H)
    assert bool(((got.rstd.double().cpu() - rs).abs() <= (n / 2 + 8) * U * rs).all())
    err = (n / 2 + 12) * U * y.abs()
    if got.out is not None:
        tol = err + HALF[got.out.dtype] * (y.abs() + err)
        assert bool(((got.out.double().cpu() - y).abs() <= tol).all())
    if got.total is not None:
        tol = U * t.abs() + HALF[got.total.dtype] * (1 + U) * t.abs()
        assert bool(((got.total.double().cpu() - t).abs() <= tol).all())
    if got.codes is not None:
        sc = got.scales.double().cpu()
        top = y.view(len(y), H // 128, 128).abs().amax(2)
        want = torch.where(top > 0, top / 448, 1.0)
        assert bool(((sc - want).abs() <= (n / 2 + 13) * U * want).all())
        full = sc.repeat_interleave(128, 1)
        value = got.codes.view(torch.float8_e4m3fn).float().double().cpu() * full
        tol = torch.maximum(2.0 ** -4 * y.abs(), 2.0 ** -10 * full) * (1 + 2.0 ** -10) + err + 2 * U * y.abs()
        assert bool(((value - y).abs() <= tol).all())


SHAPES = [(1, 1), (1, 7168), (3, 7), (17, 130), (9, 513), (64, 1000), (70, 4097), (300, 1024), (33, 8192), (6, 8200),
          (2, 16385), (2, 32768), (1030, 520), (0, 64), (2600, 64)]


@pytest.mark.parametrize("xt,rt,yt,wt", [(BF, BF, BF, BF), (BF, F32, BF, F32), (F32, F32, F32, BF), (BF, None, F32, None),
                                         (F32, BF, BF, BF)])
@pytest.mark.parametrize("T,H", SHAPES)
def test_forward(T, H, xt, rt, yt, wt):
    log("rms norm", T, H, xt, rt, yt, wt)
    x, r, w, _ = _inputs(T, H, xt, rt, wt, T + H)
    xd, rd, wd = _dev(x, r, w)
    got = rms_norm(xd, wd, 1e-6, residual=rd, out_dtype=yt)
    torch.cuda.synchronize()
    assert got.codes is None and got.scales is None and (got.total is None) == (r is None)
    _check(got, x, r, w, 1e-6)


@pytest.mark.parametrize("both", [False, True])
@pytest.mark.parametrize("xt,rt", [(BF, BF), (F32, None), (BF, F32), (F32, BF)])
@pytest.mark.parametrize("T,H", [(1, 128), (1, 7168), (65, 512), (33, 1408), (5, 16384), (3, 32768), (700, 256), (0, 128),
                                 (17, 8320)])
def test_forward_in_8_bits(T, H, xt, rt, both):
    log("rms norm fp8", T, H, xt, rt, both)
    x, r, w, _ = _inputs(T, H, xt, rt, BF, T + H)
    if T > 2:
        x[1] = 0
        if r is not None:
            r[1] = 0
        x[2, :128] *= 1e-3
    xd, rd, wd = _dev(x, r, w)
    got = rms_norm(xd, wd, 1e-6, residual=rd, want_rows=both, quantize=True)
    torch.cuda.synchronize()
    assert (got.out is not None) == both and got.codes.dtype == torch.float8_e4m3fn
    _check(got, x, r, w, 1e-6)
    if T > 2:
        assert bool((got.scales[1] == 1).all()) and bool((got.codes.view(torch.uint8)[1] & 127 == 0).all())


def test_total_may_be_an_input():
    x, r, w, _ = _inputs(300, 1032, BF, BF, F32, 4)
    xd, rd, wd = _dev(x, r, w)
    want = rms_norm(xd, wd, residual=rd)
    r2 = rd.clone()
    a = rms_norm(xd, wd, residual=r2, total=r2)
    x2 = xd.clone()
    b = rms_norm(x2, wd, residual=rd, total=x2)
    for got in (a, b):
        assert torch.equal(got.total, want.total) and torch.equal(got.out, want.out)
    assert a.total is r2 and b.total is x2
    plain = rms_norm(xd, wd, total=torch.empty_like(xd))       # without a residual: a copy
    assert torch.equal(plain.total, xd)


def test_non_finite_rows_and_no_eps():
    H = 640
    x = torch.randn(6, H, generator=torch.Generator().manual_seed(8))
    x[1] = 0.0
    x[2, 300] = float("nan")
    x[3, 639] = float("inf")
    x[4] *= 1e-30
    got = rms_norm(x.to(DEV), quantize=True)
    y, sc = got.out.cpu(), got.scales.cpu()
    assert bool((y[1] == 0).all()) and bool(y[2].isnan().all()) and bool(sc[2].isnan().all())
    assert bool(y[3, 639].isnan()) and bool((y[3, :639] == 0).all()) and bool(sc[3, 4].isnan())
    assert bool((sc[3, :4] == 1).all()) and bool(y[[0, 4, 5]].isfinite().all())
    zero = rms_norm(x[:2].to(DEV), eps=0.0)
    assert bool(zero.out[1].isnan().all()) and bool(zero.rstd[1].isinf()) and bool(zero.out[0].isfinite().all())


def test_writes_only_its_rows():
    T, H = 13, 77
    x, r, w, _ = _inputs(T, H, BF, BF, F32, 7)
    xd, rd, wd = _dev(x, r, w)
    rooms = [torch.full(((T + 2) * H + 64,), 3.0, dtype=BF, device=DEV) for _ in range(2)]
    out, total = (m[32:32 + T * H].view(T, H) for m in rooms)   # 64 bytes in: 16-byte aligned
    rms_norm(xd, wd, residual=rd, out=out, total=total)
    torch.cuda.synchronize()
    for m in rooms:
        assert bool((m[:32] == 3.0).all()) and bool((m[32 + T * H:] == 3.0).all())


@pytest.mark.parametrize("tt,yt,wt,with_total", [(BF, BF, F32, True), (F32, BF, BF, True), (F32, F32, None, False),
                                                 (BF, F32, BF, False)])
@pytest.mark.parametrize("T,H", SHAPES)
def test_backward(T, H, tt, yt, wt, with_total):
    log("rms backward", T, H, tt, yt, wt)
    t, _, w, g = _inputs(T, H, tt, None, wt, 50 + T + H)
    gy = torch.randn(T, H, generator=g).to(yt)
    gt = torch.randn(T, H, generator=g).to(tt) if with_total else None
    rstd = (1 / torch.sqrt((t.double() ** 2).mean(1) + 1e-6)).float()
    td, wd, gyd, gtd, rd = _dev(t, w, gy, gt, rstd)
    grad, gw = rms_norm_backward(gyd, td, rd, wd, grad_total=gtd)
    torch.cuda.synchronize()
    r = rstd.double()[:, None]
    xh, q = t.double() * r, gy.double() * (1.0 if w is None else w.double())
    want = r * (q - xh * (q * xh).mean(1, keepdim=True)) + (0.0 if gt is None else gt.double())
    n = _depth(H)
    tol = U * ((0.0 if gt is None else gt.double().abs()) + 2 * want.abs()
               + r * ((n + 8) * xh.abs() * (q * xh).abs().mean(1, keepdim=True) + 6 * q.abs()))
    tol = tol + HALF[tt] * (want.abs() + tol) + 1e-300
    assert grad.dtype == tt and bool(((grad.double().cpu() - want).abs() <= tol).all())
    terms = gy.double() * xh
    bound = (T + 256 + 16) * U * terms.abs().sum(0) + 1e-300
    assert bool(((gw.double().cpu() - terms.sum(0)).abs() <= bound).all())
    alone, none = rms_norm_backward(gyd, td, rd, wd, grad_total=gtd, want_weight=False)
    assert none is None and torch.equal(alone, grad)
    if with_total:
        same, gw2 = rms_norm_backward(gyd, td, rd, wd, grad_total=gtd, out=gtd)
        assert same is gtd and torch.equal(gtd, grad) and torch.equal(gw2, gw)      # in place, and bit for bit


def test_backward_against_differences():
    """Central differences of the formula in 64 bits along random directions of t and w (step 1e-5, own error 1e-6 of
    the largest term) against the kernel's gradients in fp32, each off by at most its bound."""
    T, H = 7, 300
    t, _, w, g = _inputs(T, H, F32, None, F32, 77)
    gy, gt = torch.randn(T, H, generator=g), torch.randn(T, H, generator=g)
    td, wd, gyd, gtd = _dev(t, w, gy, gt)
    f = rms_norm(td, wd)
    grad, gw = (v.double().cpu() for v in rms_norm_backward(gyd, td, f.rstd, wd, grad_total=gtd))

    def loss(tt, ww):
        return (_reference(tt, None, ww, 1e-6)[2] * gy.double()).sum() + (tt.double() * gt.double()).sum()

    n = _depth(H)
    for k in range(2):
        v = torch.randn((T, H) if k == 0 else (H,), generator=g, dtype=torch.float64)
        step = 1e-5
        up = loss(t.double() + step * v, w) if k == 0 else loss(t, w.double() + step * v)
        down = loss(t.double() - step * v, w) if k == 0 else loss(t, w.double() - step * v)
        got = ((grad if k == 0 else gw) * v).sum()
        # rstd is the kernel's, off by (n / 2 + 8) u; gradients are off by a few n u of sums of their terms
        size = float((grad.abs() * v.abs()).sum()) if k == 0 else float(
            ((gy.double() * t.double() * f.rstd.double().cpu()[:, None]).abs().sum(0) * v.abs()).sum())
        spread = 4 * (n + T + 300) * U * (size + float(gy.abs().sum()))
        assert abs(float(got - (up - down) / (2 * step))) <= spread + 1e-6 * size


def test_streams_and_graphs():
    x, r, w, g = _inputs(515, 1032, BF, BF, F32, 31)
    gy = torch.randn(515, 1032, generator=g).to(BF)
    xd, rd, wd, gyd = _dev(x, r, w, gy)

    def step():
        f = rms_norm(xd, wd, residual=rd)
        return (f.out, f.total, f.rstd) + rms_norm_backward(gyd, f.total, f.rstd, wd)

    want = step()
    torch.cuda.synchronize()
    st = torch.cuda.Stream()
    st.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(st):
        other = step()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        held = step()
    for _ in range(3):
        for t in held:
            t.zero_()
        graph.replay()
        torch.cuda.synchronize()
        for a, b, c in zip(want, other, held):
            assert torch.equal(a, b) and torch.equal(a, c)
        step()
        torch.cuda.synchronize()


@pytest.mark.parametrize("payload", ["bf16", "fp8"])
def test_layer_with_rms_norm_is_its_parts(payload):
    """layer(rms=..., residual=...) against the same calls one by one, bit for bit."""
    T, H, E, K, F = 96, 256, 8, 2, 128
    x, r, w, g = _inputs(T, H, BF, BF, BF, 41)
    rw = torch.randn(E, H, generator=g).to(DEV) * H ** -0.5
    xd, rd, wd = _dev(x, r, w)
    if payload == "bf16":
        ws = [(torch.randn(s, generator=g) * 0.05).to(BF).to(DEV) for s in ((E, 2 * F, H), (E, H, F))]
        kw = {}
    else:
        ws = [torch.randint(0, 120, s, generator=g, dtype=torch.uint8).to(DEV) for s in ((E, 2 * F, H), (E, H, F))]
        kw = dict(w1_scales=torch.full((E, 2 * F // 128, H // 128), 1e-3, device=DEV),
                  w2_scales=torch.full((E, H // 128, F // 128), 1e-3, device=DEV))
    router = lambda rows: rows.float() @ rw.T
    gate = dict(score="sigmoid", normalize=True)
    d = Dispatcher(T, H, E, K, payload=payload, device=DEV)
    r1 = rd.clone()
    got = d.layer(xd, None, None, *ws, rms=(wd, 1e-5), residual=r1, router=router, gate=gate, **kw)
    n = rms_norm(xd, wd, 1e-5, residual=rd, out_dtype=BF, quantize=payload == "fp8")
    e = Dispatcher(T, H, E, K, payload=payload, device=DEV)
    routing, probs = e.gate(router(n.out), **gate)
    perm, _, _, _, ps = e.dispatch(n.out if payload == "bf16" else n.codes, routing, probs, x_scales=n.scales)
    want = e.combine(e.grouped_mlp(perm, *ws, perm_scales=ps, **kw))
    torch.cuda.synchronize()
    assert torch.equal(got, want) and torch.equal(r1, n.total) and bool(got.isfinite().all())
    with pytest.raises(ValueError, match="exclude"):
        d.layer(xd, None, None, *ws, rms=(wd,), norm=(wd, wd), router=router, **kw)
    with pytest.raises(ValueError, match="residual needs rms"):
        d.layer(xd, None, None, *ws, residual=rd, router=router, **kw)
