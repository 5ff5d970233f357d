"""The gate refuses outputs that overlap its inputs or each other; the gradient
alone may take the logits' place."""
import ctypes as C

import pytest

from combine_routing_preprocess_amd import _abi as A
from combine_routing_preprocess_amd import api

T, E, K = 100, 8, 2
Z, R, P, B, G, O = (i << 40 for i in range(1, 7))       # addresses that nothing reads


@pytest.fixture(params=["dense_i16", "dense_i32", "sparse_bool"])
def handle(request):
    desc = api.make_desc(T=T, H=256, E=E, K=K, route_fmt=request.param)
    L = A.lib()
    n = L.moe_workspace_bytes(C.byref(desc))
    buf = (C.c_uint8 * (n + 256))()
    h = A.MoeHandle()
    assert L.moe_handle_init(C.byref(desc), C.c_void_p((C.addressof(buf) + 255) // 256 * 256), n, C.byref(h)) == 0
    wide = E if request.param == "sparse_bool" else K
    return h, buf, T * wide * {"dense_i16": 2, "dense_i32": 4, "sparse_bool": 1}[request.param], T * wide * 4


def test_gate_refuses_overlaps(handle):
    h, _buf, nr, np_ = handle

    def gate(z=Z, bias=B, r=R, p=P):
        return A.lib().moe_gate(C.byref(h), z, A.F32, bias, 0, 0, 1.0, r, p, None)

    last = 16 * ((T * E * 4 - 1) // 16)                  # the logits' last aligned 16 bytes
    for bad in (dict(r=Z), dict(p=Z), dict(r=Z + last), dict(p=Z + last), dict(r=P), dict(p=R + 4), dict(r=B),
                dict(p=B + 4), dict(z=R + 16 * ((nr - 1) // 16)), dict(r=P + 16 * ((np_ - 1) // 16))):
        assert gate(**bad) == A.MOE_EINVAL, bad


def test_gate_backward_refuses_overlaps(handle):
    h, _buf, nr, np_ = handle

    def back(g=G, z=Z, r=R, out=O):
        return A.lib().moe_gate_backward(C.byref(h), g, z, A.BF16, r, 0, 0, 1.0, out, None)

    for bad in (dict(out=Z + 16), dict(z=O + 16), dict(out=G), dict(out=R), dict(g=O + 4),
                dict(out=R + 16 * ((nr - 1) // 16)), dict(out=G + 16 * ((np_ - 1) // 16))):
        assert back(**bad) == A.MOE_EINVAL, bad
