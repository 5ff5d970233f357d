"""The grouped products and the expert MLP's training passes of no tokens at all:
nothing is read, rows are left as they were, weights' gradients become zeros or,
added up, stay."""
import pytest
import torch

from combine_routing_preprocess_amd import Dispatcher
from gpu_util import DEV, log

pytestmark = pytest.mark.gpu
BF, F32 = torch.bfloat16, torch.float32
H, E, K, F = 72, 5, 2, 40


@pytest.mark.parametrize("route_fmt", ["dense_i16", "dense_i32", "sparse_bool"])
@pytest.mark.parametrize("pad,out_rows", [(1, 0), (16, 0), (1, 40)])
def test_no_tokens(pad, out_rows, route_fmt):
    log("no tokens", pad, out_rows, route_fmt)
    d = Dispatcher(0, H, E, K, pad_multiple=pad, out_rows=out_rows, route_fmt=route_fmt, device=DEV)
    kind = dict(dense_i16=torch.int16, dense_i32=torch.int32, sparse_bool=torch.uint8)[route_fmt]
    d.ws.fill_(0xff)                                        # metadata of an earlier use: counts and offsets of -1
    d.preprocess(torch.empty((0, E if route_fmt == "sparse_bool" else K), dtype=kind, device=DEV))
    rows = lambda width, v: torch.full((d.R, width), v, dtype=BF, device=DEV)
    nan = float("nan")
    w1, w2 = torch.ones((E, 2 * F, H), dtype=BF, device=DEV), torch.ones((E, H, F), dtype=BF, device=DEV)
    out, back = rows(2 * F, 7.0), rows(H, 7.0)
    d.grouped_product(rows(H, nan), w1, out=out)
    d.grouped_product(rows(2 * F, nan), w1, transpose=True, out=back)
    y, h = rows(H, 7.0), rows(2 * F, 7.0)
    d.grouped_mlp_keep(rows(H, nan), w1, w2, out=y, h=h)
    for t in (out, back, y, h):
        assert t.shape[0] == d.R and bool((t == 7.0).all())
    for dtype in (BF, F32):
        fresh = d.grouped_weight_grad(rows(2 * F, nan), rows(H, nan), out=torch.full((E, 2 * F, H), nan, dtype=dtype, device=DEV))
        added = d.grouped_weight_grad(rows(2 * F, nan), rows(H, nan), accumulate=True,
                                      out=torch.full((E, 2 * F, H), 3.0, dtype=dtype, device=DEV))
        assert bool((fresh == 0).all()) and bool((added == 3.0).all())
        for accumulate in (False, True):
            g1, g2 = torch.full(w1.shape, 3.0, dtype=dtype, device=DEV), torch.full(w2.shape, 3.0, dtype=dtype, device=DEV)
            gx = rows(H, 7.0)
            d.grouped_mlp_backward(rows(H, nan), rows(H, nan), rows(2 * F, nan), w1, w2, grad_perm=gx, grad_w1=g1,
                                   grad_w2=g2, accumulate=accumulate)
            want = 3.0 if accumulate else 0.0
            assert bool((g1 == want).all()) and bool((g2 == want).all()) and bool((gx == 7.0).all())
