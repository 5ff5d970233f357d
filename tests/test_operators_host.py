"""Refusals of the layer norm, the gate and the 4-bit weights: every call here
is turned away by host checks, with nothing enqueued and no GPU needed."""
import ctypes as C

import pytest
import torch

from combine_routing_preprocess_amd import Dispatcher, layer_norm, layer_norm_backward
from combine_routing_preprocess_amd import _abi as A
from combine_routing_preprocess_amd import api

BF, F32 = torch.bfloat16, torch.float32


def _p(v):
    return None if v is None else C.c_void_p(v)


X, Y, Z, W = 1 << 40, 2 << 40, 3 << 40, 4 << 40      # addresses that nothing reads


def _norm(T=4, H=16, xt=A.BF16, yt=A.BF16, wt=A.F32, x=X, w=W, b=None, eps=1e-5, y=Y, mean=Z, rstd=Z):
    return A.lib().moe_layer_norm(T, H, xt, yt, wt, _p(x), _p(w), _p(b), eps, _p(y), _p(mean), _p(rstd), None)


@pytest.mark.parametrize("kw,status", [
    (dict(T=-1), A.MOE_ESHAPE), (dict(H=0), A.MOE_ESHAPE), (dict(H=A.NORM_MAX_H + 1), A.MOE_ESHAPE),
    (dict(xt=A.FP8E4M3_B128), A.MOE_EDTYPE), (dict(yt=9), A.MOE_EDTYPE), (dict(wt=A.INT4_G128), A.MOE_EDTYPE),
    (dict(eps=-1e-5), A.MOE_EINVAL), (dict(eps=float("nan")), A.MOE_EINVAL), (dict(eps=float("inf")), A.MOE_EINVAL),
    (dict(x=None), A.MOE_EINVAL), (dict(y=None), A.MOE_EINVAL), (dict(x=X + 8), A.MOE_EALIGN),
    (dict(w=W + 4), A.MOE_EALIGN), (dict(b=W + 2), A.MOE_EALIGN), (dict(mean=Z + 2), A.MOE_EALIGN),
    (dict(y=X), A.MOE_EINVAL), (dict(y=X + 64), A.MOE_EINVAL),           # overlaps x
])
def test_layer_norm_refusals(kw, status):
    assert _norm(**kw) == status


def _norm_backward(T=4, H=16, xt=A.BF16, yt=A.BF16, wt=A.F32, gy=W, x=X, mean=Z, rstd=Z, w=None, gx=Y, gw=Z, gb=Z,
                   scratch=Z, nbytes=None):
    if nbytes is None:
        nbytes = A.lib().moe_layer_norm_backward_scratch_bytes(T, H)
    return A.lib().moe_layer_norm_backward(T, H, xt, yt, wt, _p(gy), _p(x), _p(mean), _p(rstd), _p(w), _p(gx), _p(gw),
                                           _p(gb), _p(scratch), nbytes, None)


@pytest.mark.parametrize("kw,status", [
    (dict(T=-1), A.MOE_ESHAPE), (dict(H=0), A.MOE_ESHAPE), (dict(xt=7), A.MOE_EDTYPE),
    (dict(gy=None), A.MOE_EINVAL), (dict(mean=None), A.MOE_EINVAL), (dict(rstd=None), A.MOE_EINVAL),
    (dict(gx=None), A.MOE_EINVAL), (dict(scratch=None), A.MOE_EINVAL), (dict(nbytes=10), A.MOE_ENOSPC),
    (dict(gx=Y + 2), A.MOE_EALIGN), (dict(scratch=Z + 8), A.MOE_EALIGN), (dict(gw=Z + 4), A.MOE_EALIGN),
    (dict(gx=X), A.MOE_EINVAL), (dict(gx=W), A.MOE_EINVAL),
])
def test_layer_norm_backward_refusals(kw, status):
    assert _norm_backward(**kw) == status


def test_layer_norm_scratch_sizing():
    f = A.lib().moe_layer_norm_backward_scratch_bytes
    assert f(-1, 8) == 0 and f(4, 0) == 0 and f(4, A.NORM_MAX_H + 1) == 0
    assert f(0, 8) > 0
    assert f(8192, 7168) >= 256 * 2 * 7168 * 4


def _handle(**kw):
    base = dict(T=100, H=256, E=8, K=2)
    base.update(kw)
    desc = api.make_desc(**base)
    L = A.lib()
    n = L.moe_workspace_bytes(C.byref(desc))
    buf = (C.c_uint8 * (n + 256))()
    h = A.MoeHandle()
    assert L.moe_handle_init(C.byref(desc), C.c_void_p((C.addressof(buf) + 255) // 256 * 256), n, C.byref(h)) == 0
    return h, buf


def test_gate_refusals():
    L = A.lib()
    h, _buf = _handle()

    def gate(z=X, dt=A.F32, bias=None, score=0, scale=1.0, r=Y, p=Z):
        return L.moe_gate(C.byref(h), _p(z), dt, _p(bias), score, 0, scale, _p(r), _p(p), None)

    def back(g=W, z=X, dt=A.F32, r=Y, score=0, scale=1.0, out=Z):
        return L.moe_gate_backward(C.byref(h), _p(g), _p(z), dt, _p(r), score, 0, scale, _p(out), None)

    assert gate(dt=A.FP8E4M3_B128) == A.MOE_EDTYPE and back(dt=A.INT4_G128) == A.MOE_EDTYPE
    assert gate(score=2) == A.MOE_EINVAL and back(score=-1) == A.MOE_EINVAL
    assert gate(scale=float("inf")) == A.MOE_EINVAL and back(scale=float("nan")) == A.MOE_EINVAL
    assert gate(z=None) == A.MOE_EINVAL and gate(r=None) == A.MOE_EINVAL and gate(p=None) == A.MOE_EINVAL
    assert back(g=None) == A.MOE_EINVAL and back(out=None) == A.MOE_EINVAL
    assert gate(z=X + 8) == A.MOE_EALIGN and gate(r=Y + 2) == A.MOE_EALIGN and gate(p=Z + 1) == A.MOE_EALIGN
    assert gate(bias=W + 2) == A.MOE_EALIGN and back(out=Z + 4) == A.MOE_EALIGN
    h.epoch += 1                                     # a re-initialised workspace
    assert gate() == A.MOE_ESTALE and back() == A.MOE_ESTALE


def test_int4_refusals_at_the_c_entry():
    L = A.lib()
    h, _buf = _handle()
    h.state = 1

    def mlp(hh, F=128, s1=Z, s2=Z, w1=X, w2=X, nbytes=1 << 40):
        return L.moe_grouped_swiglu_mlp(C.byref(hh), F, A.INT4_G128, _p(X), None, _p(w1), _p(s1), _p(w2), _p(s2),
                                        _p(Y), nbytes, _p(W), None)

    assert mlp(h, F=64) == A.MOE_ESHAPE and mlp(h, F=0) == A.MOE_ESHAPE
    assert mlp(h, nbytes=16) == A.MOE_ENOSPC
    assert L.moe_mlp_scratch_bytes(C.byref(h), 128, A.INT4_G128) == 2 * h.desc.out_rows * 128
    assert L.moe_mlp_scratch_bytes(C.byref(h), 100, A.INT4_G128) == 0
    assert mlp(h, s2=None) == A.MOE_EINVAL and mlp(h, s2=Z + 2) == A.MOE_EALIGN and mlp(h, w2=X + 4) == A.MOE_EALIGN
    odd, _b2 = _handle(H=200)
    odd.state = 1
    assert mlp(odd) == A.MOE_ESHAPE
    fp8, _b3 = _handle(payload="fp8")
    fp8.state = 1
    assert mlp(fp8) == A.MOE_EDTYPE                  # the rows stay bf16
    assert L.moe_grouped_fc2_fp8out(C.byref(h), 128, A.INT4_G128, _p(X), _p(Z), _p(Y), 1 << 40, _p(W), _p(Z),
                                    None) in (A.MOE_EUNSUPPORTED, A.MOE_EHIP)


def _cpu(**kw):
    base = dict(T=8, H=256, E=4, K=2)
    base.update(kw)
    return Dispatcher(base.pop("T"), base.pop("H"), base.pop("E"), base.pop("K"), device="cpu", **base)


def test_binding_refuses_bad_norm_arguments():
    x = torch.zeros(4, 16, dtype=BF)
    with pytest.raises(ValueError, match="T,H"):
        layer_norm(torch.zeros(16))
    with pytest.raises(ValueError, match="x must be"):
        layer_norm(torch.zeros(4, 16, dtype=torch.float16))
    with pytest.raises(ValueError, match="contiguous"):
        layer_norm(torch.zeros(16, 4, dtype=BF).t())
    with pytest.raises(ValueError, match="weight"):
        layer_norm(x, torch.zeros(15))
    with pytest.raises(ValueError, match="share their dtype"):
        layer_norm(x, torch.zeros(16), torch.zeros(16, dtype=BF))
    with pytest.raises(ValueError, match="out must be"):
        layer_norm(x, out=torch.zeros(4, 16, dtype=torch.float16))
    with pytest.raises(ValueError, match="out must be"):
        layer_norm(x, out_dtype=torch.float16)
    with pytest.raises(ValueError, match="mean"):
        layer_norm(x, mean=torch.zeros(3))
    with pytest.raises(ValueError, match="current GPU"):
        layer_norm(x)
    stat = torch.zeros(4)
    with pytest.raises(ValueError, match="grad_y"):
        layer_norm_backward(torch.zeros(4, 15, dtype=BF), x, stat, stat)
    with pytest.raises(ValueError, match="rstd"):
        layer_norm_backward(x, x, stat, torch.zeros(4, dtype=BF))
    with pytest.raises(ValueError, match="out must be"):
        layer_norm_backward(x, x, stat, stat, out=torch.zeros(4, 16))
    with pytest.raises(ValueError, match="fewer than"):
        layer_norm_backward(x, x, stat, stat, scratch=torch.zeros(8, dtype=torch.uint8))
    with pytest.raises(ValueError, match="want_params"):
        layer_norm_backward(x, x, stat, stat, want_params=False, grad_bias=torch.zeros(16))
    with pytest.raises(ValueError, match="current GPU"):
        layer_norm_backward(x, x, stat, stat)


def test_binding_refuses_bad_gate_arguments():
    d = _cpu()
    z = torch.zeros(8, 4)
    with pytest.raises(ValueError, match="logits"):
        d.gate(torch.zeros(8, 5))
    with pytest.raises(ValueError, match="logits"):
        d.gate(z.half())
    with pytest.raises(ValueError, match="contiguous"):
        d.gate(torch.zeros(4, 8).t())
    with pytest.raises(ValueError, match="score"):
        d.gate(z, score="tanh")
    with pytest.raises(ValueError, match="bias"):
        d.gate(z, torch.zeros(4, dtype=BF))
    with pytest.raises(ValueError, match="routing"):
        d.gate(z, routing=torch.zeros(8, 2, dtype=torch.int32))
    with pytest.raises(ValueError, match="probs"):
        d.gate(z, probs=torch.zeros(8, 3))
    with pytest.raises(ValueError, match="current GPU"):
        d.gate(z)
    r = torch.zeros(8, 2, dtype=torch.int16)
    with pytest.raises(ValueError, match="probs"):
        d.gate_backward(torch.zeros(8, 4), z, r)
    with pytest.raises(ValueError, match="out must be"):
        d.gate_backward(torch.zeros(8, 2), z, r, out=torch.zeros(8, 4, dtype=BF))
    with pytest.raises(ValueError, match="current GPU"):
        d.gate_backward(torch.zeros(8, 2), z, r)


def test_binding_tells_int4_from_fp8_and_refuses_bad_shapes():
    d = _cpu()
    d.h.state = 1
    E, H, F = 4, 256, 128
    w1, s1 = torch.zeros(E, 2 * F, H // 2, dtype=torch.uint8), torch.zeros(E, 2 * F, H // 128)
    w2, s2 = torch.zeros(E, H, F // 2, dtype=torch.uint8), torch.zeros(E, H, F // 128)
    assert d._check_w1(w1, s1) == (F, "int4") and d._check_w2(w2, s2) == (F, "int4")
    f1, g1 = torch.zeros(E, 2 * F, H, dtype=torch.uint8), torch.zeros(E, 2 * F // 128, H // 128)
    f2, g2 = torch.zeros(E, H, F, dtype=torch.uint8), torch.zeros(E, H // 128, F // 128)
    assert d._check_w1(f1, g1) == (F, "fp8") and d._check_w2(f2, g2) == (F, "fp8")
    perm = torch.zeros(d.R, H, dtype=BF)
    with pytest.raises(ValueError, match="4-bit w1"):
        d.grouped_mlp(perm, f1, w2, w1_scales=s1, w2_scales=s2)        # unpacked width
    with pytest.raises(ValueError, match="w1_scales"):
        d.grouped_mlp(perm, w1, w2, w1_scales=torch.zeros(E, 2 * F, 3), w2_scales=s2)
    with pytest.raises(ValueError, match="w2_scales"):
        d.grouped_mlp(perm, w1, w2, w1_scales=s1, w2_scales=s2.double())
    with pytest.raises(ValueError, match="share the FFN width"):
        d.grouped_mlp(perm, w1, f2, w1_scales=s1, w2_scales=g2)        # mixed weight types
    with pytest.raises(ValueError, match="w1 must be"):
        d.grouped_mlp(perm, w1, w2)                                    # no scales: not known as 4-bit
    with pytest.raises(ValueError, match="multiples of 128"):
        d._check_w2(torch.zeros(E, H, 32, dtype=torch.uint8), torch.zeros(E, H, 1))
    with pytest.raises(ValueError, match="scratch"):
        d.grouped_mlp(perm, w1, w2, w1_scales=s1, w2_scales=s2, scratch=torch.zeros(8, dtype=torch.uint8))
    with pytest.raises(ValueError, match="decode layer takes fp8"):
        d.decode_fused_fp8(torch.zeros(8, H, dtype=BF), w1, w2, s1, s2, scratch=perm, expert_out=perm, out=perm)
    with pytest.raises(ValueError, match="current GPU"):
        d.grouped_mlp(perm, w1, w2, w1_scales=s1, w2_scales=s2)


def test_layer_refuses_mixed_routing_arguments():
    d = _cpu()
    x = torch.zeros(8, 256, dtype=BF)
    r = torch.zeros(8, 2, dtype=torch.int16)
    with pytest.raises(ValueError, match="gate needs a router"):
        d.layer(x, r, None, None, None, gate=dict(score="sigmoid"))
    with pytest.raises(ValueError, match="come from the router"):
        d.layer(x, r, None, None, None, router=lambda rows: rows)
