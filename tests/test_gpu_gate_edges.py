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


@pytest.mark.parametrize("fmt,E,K", [("dense_i32", 12, 3), ("sparse_bool", 12, 3), ("sparse_bool", 300, 8),
                                     ("dense_i32", 160, 96)])
@pytest.mark.parametrize("normalize", [False, True])
def test_gradient_of_infinite_logits(fmt, E, K, normalize):
    """Softmax weights of a row with a +inf logit are NaN, and so are their
    gradients in every routing format: of the whole row, or with `normalize`
    of the chosen experts.  The rows beside it stay finite, and a sigmoid's
    gradient at +inf is 0."""
    log("gate backward infinite", fmt, E, K, normalize)
    T = 6
    gen = torch.Generator().manual_seed(E + 7 * K)
    z = torch.randn(T, E, generator=gen)
    z[2, 5] = float("inf")
    z[2, 1] = float("-inf")
    z[4, 2], z[4, 3] = float("inf"), float("inf")
    zd = z.to(DEV)
    d = Dispatcher(T, 64, E, K, route_fmt=fmt, device=DEV)
    for score in ("softmax", "sigmoid"):
        routing, probs = d.gate(zd, score=score, normalize=normalize)
        g = torch.randn(probs.shape, generator=gen).to(DEV)
        got = d.gate_backward(g, zd, routing, score=score, normalize=normalize).cpu()
        if fmt == "sparse_bool":
            chosen = routing.cpu().bool()
        else:
            chosen = torch.zeros(T, E, dtype=torch.bool).scatter_(1, routing.cpu().long(), True)
        assert bool(chosen[2, 5]) and bool(chosen[4, 2:4].all())
        others = [0, 1, 3, 5]
        assert bool(torch.isfinite(got[others]).all())
        if score == "sigmoid":
            assert bool(torch.isfinite(got).all()) and float(got[2, 5]) == 0.0
            continue
        for t in (2, 4):
            through = chosen[t] if normalize else z[t] != float("-inf")
            assert bool(torch.isnan(got[t][through]).all()), t
            assert bool((got[t][~through] == 0).all()), t
