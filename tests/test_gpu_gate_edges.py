"""The gate at the ends of its ranges.  Oracle and tolerances are those of
test_gpu_gate."""
import pytest
import torch

from combine_routing_preprocess_amd import Dispatcher
from gpu_util import DEV, log
from test_gpu_gate import BF, F32, _compare, _oracle

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("fmt", ["dense_i32", "sparse_bool"])
@pytest.mark.parametrize("E,K", [(12, 4), (96, 80)])        # a slot per lane, and slots with the experts' lanes
@pytest.mark.parametrize("dtype", [F32, BF])
def test_large_scale_over_a_small_sum(E, K, fmt, dtype):
    """Chosen sigmoids that sum to some 1e-274, scaled by 3e38: the weights
    are shares of 3e38 and finite, though 3e38 / 1e-274 is no 64-bit number."""
    log("gate large scale", E, K, fmt, dtype)
    z = (-630.0 - 0.5 * torch.rand(5, E, generator=torch.Generator().manual_seed(E))).to(dtype)
    z[1] = -596.0                                 # a sum of some 1e-258, and one above it
    z[2] = -580.0
    d = Dispatcher(5, 64, E, K, route_fmt=fmt, device=DEV)
    routing, probs = d.gate(z.to(DEV), score="sigmoid", normalize=True, scale=3e38)
    torch.cuda.synchronize()
    assert bool(torch.isfinite(probs).all())
    scale = float(torch.tensor(3e38, dtype=F32))
    idx, w = _oracle(z.double().numpy(), K, None, "sigmoid", True, scale)
    _compare(d, fmt, routing, probs, idx, w, E)


@pytest.mark.parametrize("fmt", ["dense_i16", "sparse_bool"])
@pytest.mark.parametrize("E,K", [(60, 4), (256, 8), (160, 96), (1000, 6)])
@pytest.mark.parametrize("score,normalize", [("softmax", False), ("softmax", True), ("sigmoid", False),
                                             ("sigmoid", True)])
@pytest.mark.parametrize("dtype", [F32, BF])
def test_gradient_in_the_logits_place(E, K, fmt, score, normalize, dtype):
    """The same bits as into a tensor of its own."""
    log("gate backward in place", E, K, fmt, score, normalize, dtype)
    T = 70
    gen = torch.Generator().manual_seed(E + K)
    z = (2 * torch.randn(T, E, generator=gen)).to(dtype).to(DEV)
    d = Dispatcher(T, 64, E, K, route_fmt=fmt, device=DEV)
    kw = dict(score=score, normalize=normalize, scale=2.5)
    routing, probs = d.gate(z, **kw)
    g = torch.randn(probs.shape, generator=gen).to(DEV)
    want = d.gate_backward(g, z, routing, **kw)
    got = d.gate_backward(g, z, routing, out=z, **kw)
    torch.cuda.synchronize()
    assert got is z and torch.equal(got, want)
