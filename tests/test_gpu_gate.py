"""The gate and its backward pass on the GPU against the definition in 64 bits.

The choice is an integer and has to be equal: keys are held in 64 bits, and
the oracle's keys of distinct logits are at least 1e-9 apart in these inputs
(asserted), so a last bit of a 64-bit exp cannot turn them.  Weights and
gradients are computed in 64 bits and rounded once: half a step of their type,
plus 2^-40 of the terms for the 64-bit sums."""
import math

import numpy as np
import pytest
import torch

from combine_routing_preprocess_amd import Dispatcher
from gpu_util import DEV, log

pytestmark = pytest.mark.gpu
HALF = {torch.bfloat16: 2.0 ** -8, torch.float32: 2.0 ** -24}
BF, F32 = torch.bfloat16, torch.float32
NEG = float("-inf")


def _scores(z, score):
    """Scores of fp64 logits; NaN and -inf have none."""
    live = ~np.isnan(z) & (z != NEG)
    s = np.zeros_like(z)
    if score == "sigmoid":
        s[live] = np.where(z[live] >= 0, 1 / (1 + np.exp(-np.abs(z[live]))),
                           np.exp(-np.abs(z[live])) / (1 + np.exp(-np.abs(z[live]))))
        return live, s
    for t in range(z.shape[0]):
        if live[t].any():
            e = np.exp(z[t, live[t]] - z[t, live[t]].max())
            s[t, live[t]] = e / e.sum()
    return live, s


def _oracle(z, K, bias, score, normalize, scale):
    """(index [T,K], weight [T,K]) by the definition, one token at a time."""
    T, E = z.shape
    live, s = _scores(z, score)
    idx = np.full((T, K), -1, np.int64)
    w = np.zeros((T, K))
    for t in range(T):
        key = z[t] if bias is None else s[t] + bias
        cand = [e for e in range(E) if live[t, e] and not math.isnan(key[e]) and key[e] != NEG]
        cand.sort(key=lambda e: (-key[e], e))
        if bias is not None:
            k = np.array([key[e] for e in cand[:K + 1]])
            zz = np.array([z[t, e] for e in cand[:K + 1]])
            bb = np.array([bias[e] for e in cand[:K + 1]])
            close = (np.abs(np.diff(k)) < 1e-9) & ~((np.diff(zz) == 0) & (np.diff(bb) == 0))
            assert not close.any()
        cand = cand[:K]
        idx[t, :len(cand)] = cand
        v = s[t, cand]
        if normalize and len(cand):
            lg = np.array([z[t, e] if score == "softmax" else
                           min(z[t, e], 0.0) - math.log1p(math.exp(-abs(z[t, e]))) for e in cand])
            v = np.exp(lg - lg.max())
            v /= v.sum()
        w[t, :len(cand)] = v * scale
    return idx, w


def _compare(d, fmt, routing, probs, idx, w, E):
    T, K = idx.shape
    r, p = routing.cpu().numpy(), probs.double().cpu().numpy()
    if fmt == "sparse_bool":
        full, have = np.zeros((T, E)), np.zeros((T, E), np.uint8)
        for t in range(T):
            for j in range(K):
                if idx[t, j] >= 0:
                    have[t, idx[t, j]], full[t, idx[t, j]] = 1, w[t, j]
        assert np.array_equal(r, have)
        w = full
    else:
        assert r.dtype == (np.int16 if fmt == "dense_i16" else np.int32)
        assert np.array_equal(r, idx)
    assert np.all(np.abs(p - w) <= (2.0 ** -24 + 2.0 ** -40) * np.abs(w) + 2.0 ** -150), np.abs(p - w).max()


def _logits(T, E, dtype, seed, masked=0, odd=True):
    g = torch.Generator().manual_seed(seed)
    z = torch.randn(T, E, generator=g) * 2.0
    if masked:
        z[:, torch.randperm(E, generator=g)[:masked]] = NEG
    if odd and T > 4 and E > 3:
        z[0] = NEG                       # a row that the mask leaves empty
        z[1, 1:] = NEG                   # one candidate
        z[2] = 0.25                      # all equal: the lowest experts
        z[3, 2] = float("nan")
        z[4] = torch.finfo(torch.float32).min / 4   # the type's lowest values are finite logits
    return z.to(dtype)


SHAPES = [(1, 256, 8), (16, 256, 8), (70, 5, 3), (129, 97, 6), (33, 64, 1), (20, 160, 96), (9, 1024, 40),
          (6, 1000, 1000), (5, 4, 7), (300, 60, 4), (0, 8, 2), (8, 1, 1), (40, 384, 8), (7, 512, 10), (50, 8, 2)]


@pytest.mark.parametrize("fmt", ["dense_i16", "dense_i32", "sparse_bool"])
@pytest.mark.parametrize("T,E,K", SHAPES)
@pytest.mark.parametrize("score,normalize,biased,dtype", [
    ("softmax", False, False, F32), ("softmax", True, False, BF), ("sigmoid", True, True, F32),
    ("sigmoid", False, False, BF), ("softmax", False, True, F32), ("sigmoid", True, True, BF)])
def test_gate(T, E, K, fmt, score, normalize, biased, dtype):
    log("gate", T, E, K, fmt, score, normalize, biased, dtype)
    z = _logits(T, E, dtype, 1000 + T + E + K, masked=E // 5)
    bias = torch.randn(E, generator=torch.Generator().manual_seed(E)) * 0.3 if biased else None
    d = Dispatcher(T, 64, E, K, route_fmt=fmt, device=DEV)
    routing, probs = d.gate(z.to(DEV), None if bias is None else bias.to(DEV), score=score, normalize=normalize,
                            scale=2.5)
    torch.cuda.synchronize()
    idx, w = _oracle(z.double().numpy(), K, None if bias is None else bias.double().numpy(), score, normalize, 2.5)
    _compare(d, fmt, routing, probs, idx, w, E)


def test_gate_scores_that_underflow_and_saturate():
    """Normalised weights of scores below 1e-308, a plateau of saturated
    sigmoids told apart by their logits, and logits 32 bits cannot separate
    once the bias is added."""
    z = torch.tensor([[-800.0, -801.0, -900.0, -1000.0], [60.0, 61.0, 62.0, 59.0], [30.0, 30.0, 31.0, 31.0],
                      [0.0, 1e-7, 2e-7, 3e-7]])
    d = Dispatcher(4, 64, 4, 2, route_fmt="dense_i32", device=DEV)
    for score in ("softmax", "sigmoid"):
        routing, probs = d.gate(z.to(DEV), score=score, normalize=True)
        idx, w = _oracle(z.double().numpy(), 2, None, score, True, 1.0)
        _compare(d, "dense_i32", routing, probs, idx, w, 4)
    bias = torch.full((4,), 100.0)
    routing, _ = d.gate(z[3:].expand(4, 4).contiguous().to(DEV), bias.to(DEV), score="sigmoid")
    assert routing.cpu().tolist() == [[3, 2]] * 4


def test_gate_bias_masks_and_nan_keys():
    z = torch.randn(30, 12, generator=torch.Generator().manual_seed(3))
    bias = torch.zeros(12)
    bias[[0, 5]], bias[7] = NEG, float("nan")
    d = Dispatcher(30, 64, 12, 11, route_fmt="dense_i16", device=DEV)
    routing, probs = d.gate(z.to(DEV), bias.to(DEV), score="softmax", normalize=False)
    idx, w = _oracle(z.double().numpy(), 11, bias.double().numpy(), "softmax", False, 1.0)
    _compare(d, "dense_i16", routing, probs, idx, w, 12)
    assert bool((routing[:, 9:] == -1).all())


def test_gate_infinite_logits():
    """+inf is chosen first; the row's softmax weights are NaN, and with a bias
    the row has no key left.  Other rows are not touched."""
    z = torch.randn(3, 20, generator=torch.Generator().manual_seed(9))
    z[1, 7] = float("inf")
    d = Dispatcher(3, 64, 20, 2, route_fmt="dense_i32", device=DEV)
    idx, w = _oracle(z[[0, 2]].double().numpy(), 2, None, "softmax", True, 1.0)
    routing, probs = d.gate(z.to(DEV), normalize=True)
    assert int(routing[1, 0]) == 7 and bool(torch.isnan(probs[1]).all())
    _compare(d, "dense_i32", routing[[0, 2]], probs[[0, 2]], idx, w, 20)
    routing, probs = d.gate(z.to(DEV), score="sigmoid")
    assert int(routing[1, 0]) == 7 and float(probs[1, 0]) == 1.0
    routing, probs = d.gate(z.to(DEV), torch.zeros(20, device=DEV))
    assert routing[1].tolist() == [-1, -1] and probs[1].tolist() == [0.0, 0.0]


def test_gate_feeds_preprocess_and_writes_into_given_buffers():
    T, E, K = 65, 24, 3
    z = _logits(T, E, F32, 4)
    for fmt in ("dense_i16", "sparse_bool"):
        d = Dispatcher(T, 64, E, K, route_fmt=fmt, device=DEV)
        shape = (T, E) if fmt == "sparse_bool" else (T, K)
        routing = torch.full(shape, 9, dtype=torch.bool if fmt == "sparse_bool" else torch.int16, device=DEV)
        probs = torch.full(shape, float("nan"), device=DEV)
        a, b = d.gate(z.to(DEV), routing=routing, probs=probs)
        assert a is routing and b is probs
        counts, flag = d.preprocess(routing, probs)
        idx, _ = _oracle(z.double().numpy(), K, None, "softmax", False, 1.0)
        torch.cuda.synchronize()
        assert int(flag.item()) == 0
        assert np.array_equal(counts.cpu().numpy(), np.bincount(idx[idx >= 0], minlength=E))


def _grad_oracle(z, sel, gp, score, normalize, scale):
    """fp64 gradient; sel / gp [T,E]: slots of each expert and their summed gradients."""
    live, s = _scores(z, score)
    sel = sel * live
    gp = np.where(sel > 0, gp, 0.0) * scale
    lg = np.where(live, z if score == "softmax" else np.minimum(z, 0) - np.log1p(np.exp(-np.abs(np.where(live, z, 0)))),
                  NEG)
    out, size = np.zeros_like(z), np.zeros_like(z)
    for t in range(z.shape[0]):
        if not (sel[t] > 0).any() and (normalize or score == "sigmoid"):
            continue
        p = s[t].copy()
        one = np.ones_like(p)
        if score == "sigmoid":
            one = np.where(live[t], 1 / (1 + np.exp(np.minimum(np.where(live[t], z[t], 0), 700))), 0)
        dot, dabs = 0.0, 0.0
        if normalize:
            on = sel[t] > 0
            p = np.zeros_like(p)
            p[on] = np.exp(lg[t, on] - lg[t, on].max())
            p /= (sel[t] * p).sum()
        if normalize or score == "softmax":
            dot, dabs = (gp[t] * p).sum(), np.abs(gp[t] * p).sum()
        k = sel[t] if normalize else 1
        out[t] = p * one * (gp[t] - k * dot)
        size[t] = p * one * (np.abs(gp[t]) + k * dabs)
    return out, size


@pytest.mark.parametrize("fmt", ["dense_i16", "dense_i32", "sparse_bool"])
@pytest.mark.parametrize("T,E,K", SHAPES)
@pytest.mark.parametrize("score,normalize,dtype", [("softmax", False, F32), ("softmax", True, BF),
                                                   ("sigmoid", True, F32), ("sigmoid", False, BF)])
def test_gate_backward(T, E, K, fmt, score, normalize, dtype):
    log("gate backward", T, E, K, fmt, score, normalize, dtype)
    z = _logits(T, E, dtype, 2000 + T + E + K, masked=E // 5)
    d = Dispatcher(T, 64, E, K, route_fmt=fmt, device=DEV)
    zd = z.to(DEV)
    routing, _ = d.gate(zd, score=score, normalize=normalize, scale=1.5)
    shape = (T, E) if fmt == "sparse_bool" else (T, K)
    gp = torch.randn(shape, generator=torch.Generator().manual_seed(T + E))
    r = routing.cpu()
    if fmt == "sparse_bool":
        sel, full = r.double().numpy(), gp.double().numpy()
        gp[r == 0] = float("nan")                    # entries that nothing was routed to are not read into anything
    else:
        if T > 20 and K > 1:
            r[10, 1] = r[10, 0]                      # the same index twice: its slots add
            r[11, 0] = E + 3 if E < 30000 else E     # outside: an empty slot
            routing = r.to(DEV)
        sel, full = np.zeros((T, E)), np.zeros((T, E))
        rn, gn = r.numpy().astype(np.int64), gp.double().numpy()
        for t in range(T):
            for j in range(K):
                if 0 <= rn[t, j] < E:
                    sel[t, rn[t, j]] += 1
                    full[t, rn[t, j]] += gn[t, j]
        gp[(r < 0) | (r >= E)] = float("nan")
    out = d.gate_backward(gp.to(DEV), zd, routing, score=score, normalize=normalize, scale=1.5)
    torch.cuda.synchronize()
    assert out.dtype == dtype
    want, size = _grad_oracle(z.double().numpy(), sel, full, score, normalize, 1.5)
    err = np.abs(out.double().cpu().numpy() - want)
    # half a step of an fp32 value that is rounded again to bf16: 2^-24 more; below the normal range a fixed step
    tol = (HALF[dtype] + 2.0 ** -24) * np.abs(want) + 2.0 ** -40 * size + 2.0 ** -133
    assert np.all(err <= tol), (err - tol).max()


@pytest.mark.parametrize("fmt,E", [("dense_i16", 135), ("sparse_bool", 135), ("dense_i32", 3)])
@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
def test_gate_backward_of_a_single_normalised_weight_is_zero(fmt, E, score):
    """One chosen expert has the whole share whatever its logit: its gradient
    is zero, not a rounding of it."""
    T = 539
    z = _logits(T, E, F32, 17).to(DEV)
    d = Dispatcher(T, 64, E, 1, route_fmt=fmt, device=DEV)
    routing, probs = d.gate(z, score=score, normalize=True)
    assert bool(((probs == 1.0) | (probs == 0.0)).all())
    gp = torch.randn(probs.shape, generator=torch.Generator().manual_seed(18)).to(DEV)
    assert bool((d.gate_backward(gp, z, routing, score=score, normalize=True) == 0).all())


@pytest.mark.parametrize("score,normalize", [("softmax", False), ("softmax", True), ("sigmoid", True),
                                             ("sigmoid", False)])
def test_gate_backward_agrees_with_differences(score, normalize):
    T, E, K = 6, 40, 5
    z = _logits(T, E, F32, 77, odd=False)
    d = Dispatcher(T, 64, E, K, route_fmt="dense_i32", device=DEV)
    routing, _ = d.gate(z.to(DEV), score=score, normalize=normalize)
    g = torch.Generator().manual_seed(78)
    gp, v = torch.randn(T, K, generator=g), torch.randn(T, E, generator=g)
    at = routing.cpu().long()

    def loss(step):
        zz = z.double() + step * v.double()
        s = torch.sigmoid(zz) if score == "sigmoid" else torch.softmax(zz, 1)
        p = s.gather(1, at)
        if normalize:
            p = p / p.sum(1, keepdim=True)
        return float((p * gp.double()).sum())

    out = d.gate_backward(gp.to(DEV), z.to(DEV), routing, score=score, normalize=normalize).double().cpu()
    got, size = float((out * v.double()).sum()), float((out * v.double()).abs().sum())
    step = 1e-5
    want = (loss(step) - loss(-step)) / (2 * step)
    # third derivative of the order of the terms (probabilities and |v| < 4), 64-bit rounding over the step
    assert abs(got - want) <= size * 2.0 ** -23 + 1e3 * step ** 2 * float(gp.abs().sum()) + 2.0 ** -48 / step


def test_gate_graph_replay_and_other_stream():
    T, E, K = 77, 256, 8
    z = _logits(T, E, F32, 5).to(DEV)
    bias = (torch.randn(E, generator=torch.Generator().manual_seed(6)) * 0.1).to(DEV)
    d = Dispatcher(T, 64, E, K, device=DEV)
    gp = torch.randn(T, K, generator=torch.Generator().manual_seed(7)).to(DEV)
    kw = dict(score="sigmoid", normalize=True, scale=2.5)
    eager = d.gate(z, bias, **kw)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        other = d.gate(z, bias, **kw)
    torch.cuda.synchronize()
    assert torch.equal(eager[0], other[0]) and torch.equal(eager[1], other[1])
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        routing, probs = d.gate(z, bias, **kw)
        grad = d.gate_backward(gp, z, routing, score="sigmoid", normalize=True, scale=2.5)
    for k in range(3):
        z.copy_(_logits(T, E, F32, 50 + k))
        want = d.gate(z, bias, **kw)
        want_g = d.gate_backward(gp, z, want[0], score="sigmoid", normalize=True, scale=2.5)
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(routing, want[0]) and torch.equal(probs, want[1]) and torch.equal(grad, want_g)


def test_gate_offsets_past_two_to_the_31_elements():
    T, E, K = 2_200_003, 1000, 2
    z = torch.zeros((T, E), dtype=BF, device=DEV)
    tail = _logits(5, E, BF, 8, odd=False)
    z[-5:] = tail.to(DEV)
    d = Dispatcher(T, 64, E, K, device=DEV)
    routing, probs = d.gate(z)
    torch.cuda.synchronize()
    idx, w = _oracle(tail.double().numpy(), K, None, "softmax", False, 1.0)
    _compare(d, "dense_i16", routing[-5:], probs[-5:], idx, w, E)
    assert routing[0].tolist() == [0, 1]
