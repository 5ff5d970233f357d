"""Refusals of the grouped products, the expert MLP's training passes and the
RMS norm: every call here is turned away by host checks, with nothing enqueued
and no GPU needed."""
import ctypes as C

import pytest
import torch

from combine_routing_preprocess_amd import Dispatcher, rms_norm, rms_norm_backward
from combine_routing_preprocess_amd import _abi as A
from combine_routing_preprocess_amd import api

BF, F32 = torch.bfloat16, torch.float32


def _p(v):
    return None if v is None else C.c_void_p(v)


# addresses that nothing reads, 2^40 apart
X, Y, Z, W, V, S, G, Q = ((i + 1) << 40 for i in range(8))


def _handle(routed=True, **kw):
    base = dict(T=100, H=256, E=8, K=2)
    base.update(kw)
    desc = api.make_desc(**base)
    L = A.lib()
    n = L.moe_workspace_bytes(C.byref(desc))
    buf = (C.c_uint8 * (n + 256))()
    h = A.MoeHandle()
    assert L.moe_handle_init(C.byref(desc), C.c_void_p((C.addressof(buf) + 255) // 256 * 256), n, C.byref(h)) == 0
    h.state = 1 if routed else 0
    return h, buf


def _product(h, N=64, M=128, tr=0, rows=X, w=W, out=Y):
    return A.lib().moe_grouped_product(C.byref(h), N, M, tr, _p(rows), _p(w), _p(out), None)


def _wgrad(h, N=64, M=128, dt=A.BF16, acc=0, grad=Z, rows=X, out=Y):
    return A.lib().moe_grouped_weight_grad(C.byref(h), N, M, dt, acc, _p(grad), _p(rows), _p(out), None)


SIZES = [(dict(N=0), A.MOE_ESHAPE), (dict(N=-8), A.MOE_ESHAPE), (dict(N=12), A.MOE_ESHAPE), (dict(M=4), A.MOE_ESHAPE),
         (dict(M=A.GROUPED_MAX + 8), A.MOE_ESHAPE), (dict(N=A.GROUPED_MAX, M=A.GROUPED_MAX), A.MOE_ESHAPE)]


@pytest.mark.parametrize("kw,status", SIZES + [
    (dict(rows=None), A.MOE_EINVAL), (dict(w=None), A.MOE_EINVAL), (dict(out=None), A.MOE_EINVAL),
    (dict(rows=X + 8), A.MOE_EALIGN), (dict(w=W + 2), A.MOE_EALIGN), (dict(out=Y + 4), A.MOE_EALIGN),
    (dict(out=X), A.MOE_EINVAL), (dict(out=W + 16), A.MOE_EINVAL), (dict(out=X + 200 * 128 * 2 - 16), A.MOE_EINVAL),
    (dict(out=X + 200 * 64 * 2 - 16, tr=1), A.MOE_EINVAL),
])
def test_product_refusals(kw, status):
    h, _buf = _handle()
    assert _product(h, **kw) == status


@pytest.mark.parametrize("kw,status", SIZES + [
    (dict(dt=A.FP8E4M3_B128), A.MOE_EDTYPE), (dict(dt=9), A.MOE_EDTYPE),
    (dict(rows=None), A.MOE_EINVAL), (dict(grad=None), A.MOE_EINVAL), (dict(out=None), A.MOE_EINVAL),
    (dict(grad=Z + 8), A.MOE_EALIGN), (dict(rows=X + 2), A.MOE_EALIGN), (dict(out=Y + 8), A.MOE_EALIGN),
    (dict(out=X), A.MOE_EINVAL), (dict(out=Z + 32, acc=1), A.MOE_EINVAL),
    (dict(rows=Y + 8 * 64 * 128 * 4 - 16, dt=A.F32), A.MOE_EINVAL),
])
def test_weight_grad_refusals(kw, status):
    h, _buf = _handle()
    assert _wgrad(h, **kw) == status


def test_handles_without_metadata_or_stale_are_refused():
    h, _buf = _handle(routed=False)
    assert _product(h) == A.MOE_ESTALE and _wgrad(h) == A.MOE_ESTALE and _keep(h) == A.MOE_ESTALE
    assert _backward(h) == A.MOE_ESTALE
    h.state = 1
    h.epoch += 1
    assert _product(h) == A.MOE_ESTALE and _wgrad(h) == A.MOE_ESTALE and _keep(h) == A.MOE_ESTALE
    assert _backward(h) == A.MOE_ESTALE
    L = A.lib()
    assert L.moe_grouped_product(None, 64, 64, 0, None, None, None, None) == A.MOE_EINVAL
    assert L.moe_grouped_mlp_keep(None, 64, None, None, None, None, 0, None, None, None) == A.MOE_EINVAL


def _keep(h, F=128, perm=X, w1=W, w2=V, scratch=S, nbytes=1 << 30, hh=Y, out=Z):
    return A.lib().moe_grouped_mlp_keep(C.byref(h), F, _p(perm), _p(w1), _p(w2), _p(scratch), nbytes, _p(hh), _p(out),
                                        None)


def _backward(h, F=128, dt=A.BF16, acc=0, gy=Y, perm=X, hh=Z, w1=W, w2=V, scratch=S, nbytes=1 << 30, gx=G, g1=Q,
              g2=Q + (1 << 36)):
    return A.lib().moe_grouped_mlp_backward(C.byref(h), F, dt, acc, _p(gy), _p(perm), _p(hh), _p(w1), _p(w2),
                                            _p(scratch), nbytes, _p(gx), _p(g1), _p(g2), None)


@pytest.mark.parametrize("kw,status", [
    (dict(F=0), A.MOE_ESHAPE), (dict(F=-8), A.MOE_ESHAPE), (dict(F=12), A.MOE_ESHAPE), (dict(F=4), A.MOE_ESHAPE),
    (dict(F=40000), A.MOE_ESHAPE), (dict(perm=None), A.MOE_EINVAL), (dict(w1=None), A.MOE_EINVAL),
    (dict(w2=None), A.MOE_EINVAL), (dict(scratch=None), A.MOE_EINVAL), (dict(hh=None), A.MOE_EINVAL),
    (dict(scratch=S + 8), A.MOE_EALIGN), (dict(hh=Z + 4), A.MOE_EALIGN),
    (dict(nbytes=200 * 128 * 2 - 1), A.MOE_ENOSPC), (dict(scratch=W), A.MOE_EINVAL), (dict(scratch=X), A.MOE_EINVAL),
])
def test_mlp_refusals(kw, status):
    h, _buf = _handle()
    assert _keep(h, **kw) == status
    assert _backward(h, **kw) == status


def test_mlp_refusals_of_their_own():
    h, _buf = _handle()
    assert _keep(h, hh=X) == A.MOE_EINVAL and _keep(h, out=None) == A.MOE_EINVAL and _keep(h, out=X) == A.MOE_EINVAL and _keep(h, out=Y) == A.MOE_EINVAL
    assert _backward(h, gy=None) == A.MOE_EINVAL and _backward(h, dt=A.INT4_G128) == A.MOE_EDTYPE
    assert _backward(h, gx=X) == A.MOE_EINVAL and _backward(h, g1=W) == A.MOE_EINVAL
    assert _backward(h, g2=Q) == A.MOE_EINVAL and _backward(h, g1=S + 64) == A.MOE_EINVAL
    assert _backward(h, g1=Q + 8) == A.MOE_EALIGN and _backward(h, gx=G + 2) == A.MOE_EALIGN
    f = A.lib().moe_mlp_backward_scratch_bytes
    assert f(C.byref(h), 128) >= 200 * 3 * 128 * 2 and f(C.byref(h), 0) == 0 and f(C.byref(h), 12) == 0
    assert f(None, 128) == 0 and _backward(h, nbytes=f(C.byref(h), 128) - 1) == A.MOE_ENOSPC
    odd, _b2 = _handle(H=264)
    assert _keep(odd, F=A.GROUPED_MAX) == A.MOE_ESHAPE


def _rms(T=4, H=128, xt=A.BF16, rt=A.BF16, yt=A.BF16, wt=A.F32, x=X, r=Y, w=W, eps=1e-6, y=Z, q=None, sc=None, t=V,
         rstd=S):
    return A.lib().moe_rms_norm(T, H, xt, rt, yt, wt, _p(x), _p(r), _p(w), eps, _p(y), _p(q), _p(sc), _p(t), _p(rstd),
                                None)


@pytest.mark.parametrize("kw,status", [
    (dict(T=-1), A.MOE_ESHAPE), (dict(H=0), A.MOE_ESHAPE), (dict(H=A.NORM_MAX_H + 1), A.MOE_ESHAPE),
    (dict(xt=A.FP8E4M3_B128), A.MOE_EDTYPE), (dict(rt=7), A.MOE_EDTYPE), (dict(yt=9), A.MOE_EDTYPE),
    (dict(wt=A.INT4_G128), A.MOE_EDTYPE), (dict(eps=-1.0), A.MOE_EINVAL), (dict(eps=float("nan")), A.MOE_EINVAL),
    (dict(eps=float("inf")), A.MOE_EINVAL), (dict(x=None), A.MOE_EINVAL), (dict(y=None), A.MOE_EINVAL),
    (dict(q=G), A.MOE_EINVAL), (dict(sc=G), A.MOE_EINVAL), (dict(q=G, sc=Q, H=64), A.MOE_ESHAPE),
    (dict(x=X + 8), A.MOE_EALIGN), (dict(r=Y + 2), A.MOE_EALIGN), (dict(w=W + 4), A.MOE_EALIGN),
    (dict(t=V + 8), A.MOE_EALIGN), (dict(q=G + 8, sc=Q), A.MOE_EALIGN), (dict(q=G, sc=Q + 2), A.MOE_EALIGN),
    (dict(rstd=S + 1), A.MOE_EALIGN), (dict(y=X), A.MOE_EINVAL), (dict(y=Y), A.MOE_EINVAL), (dict(y=V), A.MOE_EINVAL),
    (dict(t=X + 16), A.MOE_EINVAL), (dict(t=Y + 16), A.MOE_EINVAL), (dict(t=X, rt=A.F32), A.MOE_EINVAL),
    (dict(q=Z, sc=G), A.MOE_EINVAL), (dict(rstd=X), A.MOE_EINVAL), (dict(q=G, sc=V), A.MOE_EINVAL),
])
def test_rms_norm_refusals(kw, status):
    assert _rms(**kw) == status


def _rms_back(T=4, H=128, tt=A.BF16, yt=A.BF16, wt=A.F32, gy=X, t=Y, rstd=Z, w=W, gt=V, g=G, gw=Q, scratch=S,
              nbytes=None):
    if nbytes is None:
        nbytes = A.lib().moe_rms_norm_backward_scratch_bytes(T, H)
    return A.lib().moe_rms_norm_backward(T, H, tt, yt, wt, _p(gy), _p(t), _p(rstd), _p(w), _p(gt), _p(g), _p(gw),
                                         _p(scratch), nbytes, None)


@pytest.mark.parametrize("kw,status", [
    (dict(T=-1), A.MOE_ESHAPE), (dict(H=0), A.MOE_ESHAPE), (dict(tt=7), A.MOE_EDTYPE), (dict(yt=3), A.MOE_EDTYPE),
    (dict(gy=None), A.MOE_EINVAL), (dict(t=None), A.MOE_EINVAL), (dict(rstd=None), A.MOE_EINVAL),
    (dict(g=None), A.MOE_EINVAL), (dict(scratch=None), A.MOE_EINVAL), (dict(nbytes=10), A.MOE_ENOSPC),
    (dict(g=G + 2), A.MOE_EALIGN), (dict(gt=V + 4), A.MOE_EALIGN), (dict(scratch=S + 8), A.MOE_EALIGN),
    (dict(gw=Q + 4), A.MOE_EALIGN), (dict(g=X), A.MOE_EINVAL), (dict(g=Y), A.MOE_EINVAL), (dict(g=V + 16), A.MOE_EINVAL),
    (dict(gw=G), A.MOE_EINVAL), (dict(scratch=X), A.MOE_EINVAL),
])
def test_rms_norm_backward_refusals(kw, status):
    assert _rms_back(**kw) == status


def test_rms_scratch_sizing():
    f = A.lib().moe_rms_norm_backward_scratch_bytes
    assert f(-1, 8) == 0 and f(4, 0) == 0 and f(4, A.NORM_MAX_H + 1) == 0 and f(0, 8) > 0


def test_binding_refusals():
    x = torch.zeros(4, 128, dtype=BF)
    with pytest.raises(ValueError, match="current GPU"):
        rms_norm(x)
    with pytest.raises(ValueError, match="needs quantize"):
        rms_norm(x, want_rows=False)
    with pytest.raises(ValueError, match="multiple of 128"):
        rms_norm(x[:, :64].contiguous(), quantize=True)
    with pytest.raises(ValueError, match="need quantize"):
        rms_norm(x, scales=torch.zeros(4, 1))
    with pytest.raises(ValueError, match="need want_rows"):
        rms_norm(x, want_rows=False, quantize=True, out=x)
    with pytest.raises(ValueError, match="residual must be"):
        rms_norm(x, residual=x[:3])
    with pytest.raises(ValueError, match="total must be"):
        rms_norm(x, residual=x, total=x.float())
    with pytest.raises(ValueError, match="weight must be"):
        rms_norm(x, torch.zeros(64))
    with pytest.raises(ValueError, match="contiguous"):
        rms_norm(torch.zeros(128, 4, dtype=BF).T)
    rstd = torch.zeros(4)
    with pytest.raises(ValueError, match="grad_total must be"):
        rms_norm_backward(x, x, rstd, grad_total=x.float())
    with pytest.raises(ValueError, match="want_weight"):
        rms_norm_backward(x, x, rstd, want_weight=False, grad_weight=torch.zeros(128))
    with pytest.raises(ValueError, match="fewer than"):
        rms_norm_backward(x, x, rstd, scratch=torch.zeros(8, dtype=torch.uint8))
    with pytest.raises(ValueError, match="current GPU"):
        rms_norm_backward(x, x, rstd)
    d = Dispatcher(16, 64, 4, 2, device="cpu")
    rows, w, w1, w2 = (torch.zeros(s, dtype=BF) for s in ((d.R, 64), (4, 40, 64), (4, 80, 64), (4, 64, 40)))
    for call, match in [
        (lambda: d.grouped_product(rows, w.float()), "w must be bf16"),
        (lambda: d.grouped_product(rows, w[:3]), "w must be bf16"),
        (lambda: d.grouped_product(rows[:5], w), "rows must be"),
        (lambda: d.grouped_product(rows, w, transpose=True), "rows must be"),
        (lambda: d.grouped_product(rows, w, out=rows), "out must be"),
        (lambda: d.grouped_product(rows, w.transpose(1, 2).contiguous().transpose(1, 2)), "contiguous"),
        (lambda: d.grouped_product(rows, w), "current GPU"),
        (lambda: d.grouped_weight_grad(rows, rows.float()), "rows must be"),
        (lambda: d.grouped_weight_grad(rows, rows, accumulate=True), "needs out"),
        (lambda: d.grouped_weight_grad(rows, rows, out=w), "out must be"),
        (lambda: d.grouped_weight_grad(rows, rows), "current GPU"),
        (lambda: d.grouped_mlp_keep(rows, w, w2), "w2 must be"),
        (lambda: d.grouped_mlp_keep(rows, w1, w2, h=rows), "h must be"),
        (lambda: d.grouped_mlp_keep(rows, w1, w2), "current GPU"),
        (lambda: d.grouped_mlp_backward(rows, rows, rows, w1, w2), "h must be"),
        (lambda: d.grouped_mlp_backward(rows, rows, torch.zeros(d.R, 80, dtype=BF), w1, w2, accumulate=True),
         "accumulate needs"),
        (lambda: d.grouped_mlp_backward(rows, rows, torch.zeros(d.R, 80, dtype=BF), w1, w2, grad_w1=w1.float(),
                                        grad_w2=w2), "grad_w2 must be"),
        (lambda: d.grouped_mlp_backward(rows, rows, torch.zeros(d.R, 80, dtype=BF), w1, w2, want_weights=False,
                                        grad_w1=w1), "want_weights"),
        (lambda: d.grouped_mlp_backward(rows, rows, torch.zeros(d.R, 80, dtype=BF), w1, w2,
                                        scratch=torch.zeros(64, dtype=torch.uint8)), "fewer than"),
        (lambda: d.grouped_mlp_backward(rows, rows, torch.zeros(d.R, 80, dtype=BF), w1, w2), "current GPU"),
    ]:
        with pytest.raises(ValueError, match=match):
            call()
