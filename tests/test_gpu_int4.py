"""The grouped SwiGLU MLP with 4-bit weights on the GPU against the formula in
64 bits, and the run norm -> gate -> dispatch -> 4-bit experts -> combine.

Per element, with u = 2^-24: a 128-column group adds at most 160 products of
|x| (31 + 24) at most in fp32 (one rounding each, counted twice for a matrix
unit that truncates), so a sum over G groups is off by at most
2 (160 + G) u * 55 * sum(s |x|) =: d.  The activation a = silu(g) u carries
dg, du (|silu'| < 1.1), a few u of exp and division, and half a bf16 step; the
output carries sum(|w| da) and its own d, and half a bf16 step.  That bound is
for the worst case of every rounding; in the 2-norm roundings are
independent and at most 2^-8 / sqrt(3) each: sqrt(2) of that for the two of
them, 3.2e-3, and 1e-4 on top for the fp32 sums."""
import numpy as np
import pytest
import torch

from combine_routing_preprocess_amd import Dispatcher, layer_norm, layer_norm_backward
from combine_routing_preprocess_amd import _abi as A
from gpu_util import DEV, log

pytestmark = pytest.mark.gpu
U = 2.0 ** -24
BF = torch.bfloat16


def _weights(E, N, K, seed, std=0.05):
    g = torch.Generator().manual_seed(seed)
    codes = torch.randint(0, 256, (E, N, K // 2), generator=g, dtype=torch.uint8)
    scales = (0.5 + torch.rand(E, N, K // 128, generator=g)) * std / 4.6
    return codes, scales


def _deq(codes, scales):
    c = torch.stack((codes & 15, codes >> 4), dim=-1).flatten(-2).double() - 8
    return c * scales.double().repeat_interleave(128, dim=-1)


def _gemm_err(x, scales, K):
    """d of every (row, weight row)."""
    G = K // 128
    sx = x.abs().reshape(x.shape[0], G, 128).sum(-1)
    return 2 * (160 + G) * U * 55 * (sx @ scales.double().T)


def _mlp_oracle(x, c1, s1, c2, s2):
    """(y, tolerance) of one expert's rows in 64 bits."""
    x = x.double()
    F = c1.shape[0] // 2
    h = x @ _deq(c1, s1).T
    dh = _gemm_err(x, s1, x.shape[1])
    g, u, dg, du = h[:, :F], h[:, F:], dh[:, :F], dh[:, F:]
    si = g * torch.sigmoid(g)
    a = si * u
    da = 1.1 * dg * (u.abs() + du) + si.abs() * du + 16 * U * a.abs()
    da = da + 2.0 ** -8 * (a.abs() + da)
    w2 = _deq(c2, s2)
    y = a @ w2.T
    dy = da @ w2.abs().T + _gemm_err(a.abs() + da, s2, F)
    return y, dy + 2.0 ** -8 * (y.abs() + dy)


def _route(T, E, K, seed, empty=0, one=None):
    g = torch.Generator().manual_seed(seed)
    idx = torch.rand(T, E, generator=g).argsort(1)[:, :K].to(torch.int32)
    if one is not None:
        idx[:, 0] = one                      # every token to one expert; duplicates are dropped below
        for t in range(T):
            for j in range(1, K):
                if int(idx[t, j]) == one:
                    idx[t, j] = -1
    if empty:
        idx.view(-1)[torch.randperm(T * K, generator=g)[:empty]] = -1
    return idx


def _check(d, perm, w, out, fill):
    c1, s1, c2, s2 = w
    seg, kept = d.seg_off.cpu().tolist(), d.kept.cpu().tolist()
    got = out.cpu()
    used = torch.zeros(d.R, dtype=torch.bool)
    num = den = 0.0
    for e, n in enumerate(kept):
        if n == 0:
            continue
        rows = slice(seg[e], seg[e] + n)
        used[rows] = True
        want, tol = _mlp_oracle(perm[rows].cpu(), c1[e], s1[e], c2[e], s2[e])
        err = (got[rows].double() - want).abs()
        assert bool((err <= tol).all()), (e, float((err / tol).max()))
        num, den = num + float((err ** 2).sum()), den + float((want ** 2).sum())
    assert num ** 0.5 <= 3.3e-3 * den ** 0.5
    assert bool((got[~used] == fill).all())   # rows without a copy stay as they were


CASES = [
    # T, E, K, H, F, pad, capacity, empty, one
    (1, 8, 2, 128, 128, 1, None, 0, None),
    (1, 16, 4, 1024, 512, 4, None, 0, None),
    (3, 4, 2, 384, 256, 1, None, 2, None),          # an odd number of groups in FC1
    (40, 6, 3, 256, 640, 16, None, 9, None),        # and in FC2
    (17, 3, 2, 1152, 128, 1, None, 0, 1),           # 17 rows of one expert: a second token block
    (70, 5, 2, 640, 384, 8, None, 0, 2),            # 70 rows: a second pass
    (200, 4, 2, 512, 256, 1, 33, 0, 0),             # capacity drops copies
    (64, 32, 8, 2048, 1024, 2, None, 30, None),
    (20, 40, 3, 1024, 1024, 1, None, 5, None),      # many units of few rows
    (90, 100, 2, 384, 640, 3, None, 0, 7),          # the same with odd groups, and one expert of 90 rows
    (150, 64, 2, 512, 1024, 1, None, 0, None),
    (300, 4, 2, 384, 256, 4, None, 7, None),        # many rows of few experts: small passes on many CUs
    (260, 3, 2, 1152, 384, 1, None, 0, 1),          # the same with odd groups and unequal experts
    (80, 32, 8, 1152, 640, 1, None, 40, 2),         # passes of 32 rows, one expert of three
    (170, 32, 8, 2176, 1152, 2, None, 0, 3),        # passes of 64 rows; FC2's last unit is half empty
    (5, 4, 2, 256, 128, 1, None, 10, None),         # nothing routed
    (0, 4, 2, 256, 128, 1, None, 0, None),
]


@pytest.mark.parametrize("T,E,K,H,F,pad,cap,empty,one", CASES)
def test_grouped_mlp_int4(T, E, K, H, F, pad, cap, empty, one):
    log("int4 mlp", T, E, K, H, F, pad, cap, empty, one)
    idx = _route(T, E, K, 3 + T, empty, one)
    d = Dispatcher(T, H, E, K, route_fmt="dense_i32", pad_multiple=pad, capacity=cap, device=DEV)
    g = torch.Generator().manual_seed(T + H)
    x = torch.randn(T, H, generator=g).to(BF)
    perm, *_ = d.dispatch(x.to(DEV), idx.to(DEV), out=torch.zeros((d.R, H), dtype=BF, device=DEV))
    w = _weights(E, 2 * F, H, 11) + _weights(E, H, F, 12)
    c1, s1, c2, s2 = (t.to(DEV) for t in w)
    out = torch.full((d.R, H), 7.0, dtype=BF, device=DEV)
    scratch = d.alloc_mlp_scratch(F, "int4") if d.R else torch.empty(256, dtype=torch.uint8, device=DEV)
    if d.R == 0:
        return
    y = d.grouped_mlp(perm, c1, c2, w1_scales=s1, w2_scales=s2, scratch=scratch, out=out)
    torch.cuda.synchronize()
    assert y is out
    _check(d, perm, w, out, 7.0)
    # the two halves, and the entry point without a scratch, give the same bits
    again = torch.full((d.R, H), 7.0, dtype=BF, device=DEV)
    d.fc1(perm, c1, scratch, w1_scales=s1)
    d.fc2(c2, scratch, again, w2_scales=s2)
    third = torch.full((d.R, H), 7.0, dtype=BF, device=DEV)
    d.grouped_mlp_noalloc(perm, c1, c2, w1_scales=s1, w2_scales=s2, out=third)
    torch.cuda.synchronize()
    assert torch.equal(again, out) and torch.equal(third, out)


def test_every_code_and_column_lands_in_its_place():
    """One-hot rows read single weight columns back: y's FC1 sums are single
    weights, exact in fp32, so a misplaced code, column or scale shows."""
    E, K, H, F = 2, 1, 512, 128
    T = H
    idx = torch.zeros(T, K, dtype=torch.int32)
    idx[1::2] = 1
    x = torch.eye(H).to(BF)
    d = Dispatcher(T, H, E, K, route_fmt="dense_i32", device=DEV)
    perm, *_ = d.dispatch(x.to(DEV), idx.to(DEV))
    w1 = _weights(E, 2 * F, H, 21, std=2.0)
    c1, s1 = (t.to(DEV) for t in w1)
    scratch = d.alloc_mlp_scratch(F, "int4")
    d.fc1(perm, c1, scratch, w1_scales=s1)
    torch.cuda.synchronize()
    # the scratch keeps each 8 features in the order 0 4 1 5 2 6 3 7
    order = torch.arange(F).view(-1, 8)[:, [0, 4, 1, 5, 2, 6, 3, 7]].flatten()
    a = torch.empty(T, F, dtype=torch.float64)
    a[:, order] = scratch[:T * F * 2].view(BF).view(T, F).double().cpu()
    rows = d.row_id.cpu()[:, 0].long()
    deq = _deq(*w1)
    for t in range(T):
        h = deq[int(idx[t, 0]), :, t]
        want = h[:F] * torch.sigmoid(h[:F]) * h[F:]
        # one code and the offset's 24: exact; then the scale, exp, division and the bf16 step
        assert bool(((a[rows[t]] - want).abs() <= (2.0 ** -8 + 32 * U) * want.abs() + 1e-12).all()), t


def test_graph_replay_other_stream_and_shared_experts():
    T, E, K, H, F = 24, 8, 2, 512, 256
    idx = _route(T, E, K, 5).to(DEV)
    d = Dispatcher(T, H, E, K, route_fmt="dense_i32", device=DEV)
    x = torch.randn(T, H, generator=torch.Generator().manual_seed(6)).to(BF).to(DEV)
    pr = torch.rand(T, K, generator=torch.Generator().manual_seed(7)).to(DEV)
    c1, s1 = (t.to(DEV) for t in _weights(E, 2 * F, H, 8))
    c2, s2 = (t.to(DEV) for t in _weights(E, H, F, 9))
    kw = dict(w1_scales=s1, w2_scales=s2)
    want = d.layer(x, idx, pr, c1, c2, **kw)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        other = d.layer(x, idx, pr, c1, c2, **kw)
    torch.cuda.synchronize()
    assert torch.equal(want, other)
    bufs = dict(perm=torch.empty((d.R, H), dtype=BF, device=DEV), scratch=d.alloc_mlp_scratch(F, "int4"),
                expert_out=torch.empty((d.R, H), dtype=BF, device=DEV), out=torch.empty((T, H), dtype=BF, device=DEV))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        y = d.layer(x, idx, pr, c1, c2, **kw, **bufs)
    for k in range(3):
        x.copy_(torch.randn(T, H, generator=torch.Generator().manual_seed(60 + k)))
        idx.copy_(_route(T, E, K, 70 + k))
        graph.replay()
        torch.cuda.synchronize()
        got = y.clone()
        assert torch.equal(got, Dispatcher(T, H, E, K, route_fmt="dense_i32", device=DEV).layer(x, idx, pr, c1, c2, **kw))


def test_two_calls_at_once():
    """Two dispatchers with their own buffers on two streams at a time give
    what each gives alone."""
    T, E, K, H, F = 60, 16, 4, 1024, 512
    c1, s1 = (t.to(DEV) for t in _weights(E, 2 * F, H, 18))
    c2, s2 = (t.to(DEV) for t in _weights(E, H, F, 19))
    streams, runs = [torch.cuda.Stream(), torch.cuda.Stream()], []
    for k in range(2):
        d = Dispatcher(T, H, E, K, route_fmt="dense_i32", device=DEV)
        x = torch.randn(T, H, generator=torch.Generator().manual_seed(80 + k)).to(BF).to(DEV)
        idx, z = _route(T, E, K, 81 + k).to(DEV), torch.randn(T, E, generator=torch.Generator().manual_seed(k)).to(DEV)
        runs.append((d, x, idx, z, d.layer(x, idx, None, c1, c2, w1_scales=s1, w2_scales=s2), d.gate(z), layer_norm(x)))
    torch.cuda.synchronize()
    for rep in range(3):
        got = []
        for (d, x, idx, z, *_), s in zip(runs, streams):
            with torch.cuda.stream(s):
                got.append((d.layer(x, idx, None, c1, c2, w1_scales=s1, w2_scales=s2), d.gate(z), layer_norm(x)))
        torch.cuda.synchronize()
        for (y, g, n), (*_, wy, wg, wn) in zip(got, runs):
            assert torch.equal(y, wy)
            assert all(torch.equal(p, q) for p, q in zip(g + n, wg + wn))


@pytest.mark.parametrize("payload", ["bf16", "fp8"])
def test_layer_paths_take_norm_and_gate(payload):
    """layer() with norm, router and gate equals the calls made one by one, on
    bf16 rows with bf16 weights and on rows quantised on dispatch."""
    import moe_synth as S
    T, E, K, H, F = 33, 8, 2, 256, 128
    g = torch.Generator().manual_seed(61)
    h, nw, wr = torch.randn(T, H, generator=g).to(BF).to(DEV), torch.ones(H, device=DEV), torch.randn(E, H, generator=g).to(DEV)
    if payload == "fp8":
        w1, s1 = (t.to(DEV) for t in S.weights_fp8_blocks(E, 2 * F, H, 62, std=0.05))
        w2, s2 = (t.to(DEV) for t in S.weights_fp8_blocks(E, H, F, 63, std=0.05))
    else:
        w1, w2 = torch.randn(E, 2 * F, H, generator=g).to(BF).to(DEV) * 0.05, torch.randn(E, H, F, generator=g).to(BF).to(DEV) * 0.05
        s1 = s2 = None
    d = Dispatcher(T, H, E, K, payload=payload, device=DEV)
    router = lambda rows: rows.float() @ wr.T
    got = d.layer(h, None, None, w1, w2, w1_scales=s1, w2_scales=s2, norm=(nw, None, 1e-6), router=router,
                  gate=dict(normalize=True))
    x, _, _ = layer_norm(h, nw, None, 1e-6)
    routing, probs = d.gate(router(x), normalize=True)
    want = d.layer(x, routing, probs, w1, w2, w1_scales=s1, w2_scales=s2)
    torch.cuda.synchronize()
    assert torch.equal(got, want) and bool(torch.isfinite(got).all())


@pytest.mark.parametrize("fmt,score,normalize,biased", [("dense_i16", "sigmoid", True, True),
                                                        ("sparse_bool", "softmax", False, False)])
def test_norm_gate_and_int4_layer_together(fmt, score, normalize, biased):
    """The whole run as a serving loop makes it: an fp32 residual stream,
    layer norm, router product, gate, dispatch, 4-bit experts, combine."""
    T, E, K, H, F = 50, 16, 4, 512, 256
    g = torch.Generator().manual_seed(31)
    h = torch.randn(T, H, generator=g) * 2 + 0.5
    nw, nb = 1 + 0.1 * torch.randn(H, generator=g), 0.1 * torch.randn(H, generator=g)
    wr = torch.randn(E, H, generator=g) / H ** 0.5
    bias = 0.1 * torch.randn(E, generator=g) if biased else None
    w = _weights(E, 2 * F, H, 32) + _weights(E, H, F, 33)
    c1, s1, c2, s2 = (t.to(DEV) for t in w)
    d = Dispatcher(T, H, E, K, route_fmt=fmt, pad_multiple=4, device=DEV)
    seen = {}
    wrd = wr.to(DEV)

    def router(rows):
        seen["rows"], seen["logits"] = rows, rows.float() @ wrd.T
        return seen["logits"]

    gate = dict(score=score, normalize=normalize, scale=2.0)
    if biased:
        gate["bias"] = bias.to(DEV)
    y = d.layer(h.to(DEV), None, None, c1, c2, w1_scales=s1, w2_scales=s2, norm=(nw.to(DEV), nb.to(DEV)),
                router=router, gate=gate)
    torch.cuda.synchronize()
    rows, z = seen["rows"].cpu(), seen["logits"].double().cpu()
    hd = h.double()
    xh = (hd - hd.mean(1, keepdim=True)) / torch.sqrt(hd.var(1, unbiased=False, keepdim=True) + 1e-5)
    ref = xh * nw.double() + nb.double()
    # norm in fp32 (sums of 46 terms' depth, see the norm's tests) and half a bf16 step
    assert bool(((rows.double() - ref).abs() <= 2.0 ** -8 * ref.abs() + 64 * U * (xh.abs() + 1)
                 * nw.double().abs() + 4 * U * nb.double().abs()).all())
    s = torch.sigmoid(z) if score == "sigmoid" else torch.softmax(z, 1)
    at = torch.topk(s + bias.double() if biased else z, K, dim=1).indices
    p = s.gather(1, at)
    p = 2.0 * (p / p.sum(1, keepdim=True) if normalize else p)
    want, tol = torch.zeros(T, H, dtype=torch.float64), torch.zeros(T, H, dtype=torch.float64)
    for t in range(T):
        for j in range(K):
            e = int(at[t, j])
            yy, tt = _mlp_oracle(rows[t:t + 1], w[0][e], w[1][e], w[2][e], w[3][e])
            want[t] += p[t, j] * yy[0]
            tol[t] += p[t, j] * (tt[0] + 8 * U * (yy[0].abs() + tt[0]))
    tol += 2.0 ** -8 * (want.abs() + tol)
    err = (y.double().cpu() - want).abs()
    assert bool((err <= tol).all()), float((err / tol).max())


def test_training_run_of_norm_gate_dispatch_and_combine():
    """Gradients of the loss sum(combine(permute(norm(h)), gate(logits)) * gy)
    with the experts left out (each expert returns its rows): the chain of the
    backward calls against autograd of the same formula in 64 bits, and
    against the difference of the loss along a direction."""
    T, E, K, H = 40, 8, 3, 128
    g = torch.Generator().manual_seed(41)
    h = torch.randn(T, H, generator=g)
    nw, nb = 1 + 0.1 * torch.randn(H, generator=g), 0.1 * torch.randn(H, generator=g)
    wr = torch.randn(E, H, generator=g) / H ** 0.5
    gy = torch.randn(T, H, generator=g).to(BF)
    hd, nwd, nbd, wrd, gyd = (t.to(DEV) for t in (h, nw, nb, wr, gy))
    d = Dispatcher(T, H, E, K, device=DEV)
    x, mean, rstd = layer_norm(hd, nwd, nbd, out_dtype=BF)
    z = x.float() @ wrd.T
    kw = dict(score="sigmoid", normalize=True, scale=1.5)
    routing, probs = d.gate(z, **kw)
    perm, *_ = d.dispatch(x, routing, probs)
    y = d.combine(perm)
    # backward
    g_perm, g_probs = d.combine_backward(gyd, perm)
    g_z = d.gate_backward(g_probs, z, routing, **kw)
    g_x, _ = d.dispatch_backward(g_perm)
    g_x = g_x.float() + g_z @ wrd
    g_h, g_w, g_b = layer_norm_backward(g_x, hd, mean, rstd, nwd)
    torch.cuda.synchronize()

    at = routing.cpu().long()
    hh, ww, bb = (t.double().requires_grad_(True) for t in (h, nw, nb))
    mu = hh.mean(1, keepdim=True)
    xx = (hh - mu) / torch.sqrt(((hh - mu) ** 2).mean(1, keepdim=True) + 1e-5) * ww + bb
    s = torch.sigmoid(xx @ wr.double().T).gather(1, at)
    p = 1.5 * s / s.sum(1, keepdim=True)
    out = (p.unsqueeze(2) * xx.unsqueeze(1)).sum(1)
    loss = (out * gy.double()).sum()
    loss.backward()
    # roundings to bf16 on the way: x, the copies' gradients (K of them), their sum: 2^-8 / sqrt(3) each in the
    # 2-norm, at most 5 of them in a value, and the same in the forward's y
    lim = 5 * 2.0 ** -8 / 3 ** 0.5
    for got, want in ((y, out.detach()), (g_h, hh.grad), (g_w, ww.grad), (g_b, bb.grad)):
        got = got.double().cpu()
        assert float((got - want).norm()) <= lim * float(want.norm())
    v = torch.randn(T, H, generator=g).double()

    def at_step(t):
        hv = h.double() + t * v
        m = hv.mean(1, keepdim=True)
        xv = (hv - m) / torch.sqrt(((hv - m) ** 2).mean(1, keepdim=True) + 1e-5) * nw.double() + nb.double()
        sv = torch.sigmoid(xv @ wr.double().T).gather(1, at)
        return float((1.5 * (sv / sv.sum(1, keepdim=True)).unsqueeze(2) * xv.unsqueeze(1)).sum(1).mul(gy.double()).sum())

    got = float((g_h.double().cpu() * v).sum())
    want = (at_step(1e-5) - at_step(-1e-5)) / 2e-5
    assert abs(got - want) <= lim * float(hh.grad.norm() * v.norm())
