"""An expert MLP without rows (no tokens, or a capacity of 0) is a valid call
that launches nothing: its checks pass without a GPU, with null rows, for
every weight type."""
import ctypes as C

import pytest
import torch

from combine_routing_preprocess_amd import Dispatcher
from combine_routing_preprocess_amd import _abi as A
from combine_routing_preprocess_amd import api

W, S = 1 << 40, 2 << 40      # addresses that nothing reads


def _handle(**kw):
    base = dict(T=0, H=256, E=4, K=2)
    base.update(kw)
    desc = api.make_desc(**base)
    L = A.lib()
    n = L.moe_workspace_bytes(C.byref(desc))
    buf = (C.c_uint8 * (n + 256))()
    h = A.MoeHandle()
    assert L.moe_handle_init(C.byref(desc), C.c_void_p((C.addressof(buf) + 255) // 256 * 256), n, C.byref(h)) == 0
    h.state = 1
    return h, buf


@pytest.mark.parametrize("shape", [dict(T=0), dict(T=9, capacity=0)])
@pytest.mark.parametrize("wdtype,scales", [(A.BF16, None), (A.FP8E4M3_B128, S), (A.INT4_G128, S)])
def test_mlp_without_rows_is_valid(shape, wdtype, scales):
    L = A.lib()
    h, _buf = _handle(**shape)
    assert h.desc.out_rows == 0
    need = L.moe_mlp_scratch_bytes(C.byref(h), 128, wdtype)
    assert 0 < need <= 256
    args = (C.byref(h), 128, wdtype)
    scratch = C.c_void_p(3 << 40)
    assert L.moe_grouped_swiglu_mlp(*args, None, None, W, scales, W, scales, scratch, need, None, None) == A.MOE_OK
    assert L.moe_grouped_fc1_swiglu(*args, None, None, W, scales, scratch, need, None) == A.MOE_OK
    assert L.moe_grouped_fc2(*args, W, scales, scratch, need, None, None) == A.MOE_OK
    # what is wrong without rows is still refused
    assert L.moe_grouped_fc1_swiglu(*args, None, None, None, scales, scratch, need, None) == A.MOE_EINVAL
    assert L.moe_grouped_fc1_swiglu(*args, None, None, W, scales, scratch, need - 1, None) == A.MOE_ENOSPC
    bad = 100                                      # no multiple of 128
    assert L.moe_grouped_fc1_swiglu(C.byref(h), bad, wdtype, None, None, W, scales, scratch, need,
                                    None) == A.MOE_ESHAPE


def test_rows_quantised_on_dispatch_may_be_none_too():
    L = A.lib()
    h, _buf = _handle(payload="fp8")
    need = L.moe_mlp_scratch_bytes(C.byref(h), 128, A.FP8E4M3_B128)
    scratch = C.c_void_p(3 << 40)
    assert L.moe_grouped_fc1_swiglu(C.byref(h), 128, A.FP8E4M3_B128, None, None, W, S, scratch, need,
                                    None) == A.MOE_OK
    full, _b2 = _handle(T=3, payload="fp8")        # rows there, their scales missing: the entry whose host checks run
    assert L.moe_grouped_swiglu_mlp_noalloc(C.byref(full), 128, A.FP8E4M3_B128, W, None, W, S, W, S, W,
                                            None) == A.MOE_EINVAL       # before it looks for a GPU


@pytest.mark.parametrize("wdtype", ["bf16", "fp8", "int4"])
def test_binding_takes_a_scratch_for_no_rows(wdtype):
    d = Dispatcher(0, 256, 4, 2, device="cpu")
    scratch = d.alloc_mlp_scratch(128, wdtype)
    d._check_scratch(scratch, 128, wdtype)
    if wdtype != "bf16":
        with pytest.raises(ValueError, match="invalid FFN width"):
            d._check_scratch(torch.zeros(256, dtype=torch.uint8), 100, wdtype)
