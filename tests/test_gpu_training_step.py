"""A training step as its user runs it: RMS norm with the residual, router, gate,
dispatch, expert MLP, combine, and back to the gradients of the rows, the
residual stream, the norm's weight, the router and the experts, against autograd
in 64 bits with the same choice of experts.

Tolerance, as the 2-norm of the difference relative to the 2-norm: a gradient's
path holds at most eleven roundings to bf16 (total, rows, h, activations, expert
output and layer output forward; row gradients of the combine, of h, the
activations, the permuted rows and the tokens backward), each off by at most
2^-8 of its value, in sums whose terms carry independent errors, so that a sum's
relative error is no larger than its terms'; SwiGLU's and the sigmoid's slopes
add at most a factor of 2.  11 * 2^-8 * 2 = 0.086; a term left out or doubled
shows as 0.3 and more."""
import pytest
import torch

from combine_routing_preprocess_amd import Dispatcher, rms_norm, rms_norm_backward
from gpu_util import DEV, log

pytestmark = pytest.mark.gpu
BF = torch.bfloat16


def _inputs(T, H, E, F, seed):
    g = torch.Generator().manual_seed(seed)
    n = lambda *s, std=1.0: torch.randn(*s, generator=g) * std
    return dict(x=n(T, H).to(BF), res=n(T, H).to(BF), wn=(1 + 0.2 * n(H)), wr=n(E, H, std=H ** -0.5),
                w1=n(E, 2 * F, H, std=H ** -0.5).to(BF), w2=n(E, H, F, std=F ** -0.5).to(BF),
                gy=n(T, H).to(BF), gt=n(T, H, std=0.3).to(BF))


def _step(d, p):
    n = rms_norm(p["x"], p["wn"], 1e-6, residual=p["res"], out_dtype=BF)
    logits = n.out.float() @ p["wr"].T
    gate = dict(score="sigmoid", normalize=True, scale=1.5)
    routing, probs = d.gate(logits, **gate)
    perm, _, _, _, _ = d.dispatch(n.out, routing, probs)
    y, h = d.grouped_mlp_keep(perm, p["w1"], p["w2"])
    out = d.combine(y)
    g_y, g_probs = d.combine_backward(p["gy"], y)
    g_perm, g1, g2 = d.grouped_mlp_backward(g_y, perm, h, p["w1"], p["w2"], grad_dtype=torch.float32)
    g_rows, _ = d.dispatch_backward(g_perm)
    g_logits = d.gate_backward(g_probs, logits, routing, **gate)
    g_norm = g_rows.float() + g_logits @ p["wr"]
    g_x, g_wn = rms_norm_backward(g_norm, n.total, n.rstd, p["wn"], grad_total=p["gt"])
    return dict(out=out, routing=routing, x=g_x, wn=g_wn, wr=g_logits.T @ n.out.float(), w1=g1, w2=g2)


def _reference(p, routing):
    q = {k: v.double().cpu() for k, v in p.items()}
    for k in ("x", "wn", "wr", "w1", "w2"):
        q[k].requires_grad_(True)
    F = q["w2"].shape[2]
    t = q["x"] + q["res"]
    rows = t * torch.rsqrt((t * t).mean(1, keepdim=True) + 1e-6) * q["wn"]
    s = torch.sigmoid(rows @ q["wr"].T).gather(1, routing.long().cpu())
    prob = 1.5 * s / s.sum(1, keepdim=True)
    out = torch.zeros_like(rows)
    for e in range(q["w1"].shape[0]):
        tok, slot = (routing.cpu() == e).nonzero(as_tuple=True)
        h = rows[tok] @ q["w1"][e].T
        y = (torch.sigmoid(h[:, :F]) * h[:, :F] * h[:, F:]) @ q["w2"][e].T
        out = out.index_add(0, tok, prob[tok, slot][:, None] * y)
    ((out * q["gy"]).sum() + (t * q["gt"]).sum()).backward()
    return dict(out=out.detach(), **{k: q[k].grad for k in ("x", "wn", "wr", "w1", "w2")})


@pytest.mark.parametrize("T,H,E,K,F,pad", [(64, 128, 4, 2, 72, 1), (200, 264, 8, 3, 136, 16), (1, 64, 4, 2, 40, 4)])
def test_training_step(T, H, E, K, F, pad):
    log("training step", T, H, E, K, F)
    p = {k: v.to(DEV) for k, v in _inputs(T, H, E, F, T + H).items()}
    d = Dispatcher(T, H, E, K, route_fmt="dense_i32", pad_multiple=pad, device=DEV)
    got = _step(d, p)
    torch.cuda.synchronize()
    want = _reference(p, got["routing"])
    for k in ("out", "x", "wn", "wr", "w1", "w2"):
        a, b = got[k].double().cpu(), want[k]
        assert a.shape == b.shape
        off = float((a - b).norm() / b.norm())
        assert off <= 11 * 2.0 ** -8 * 2, (k, off)


def test_training_step_in_a_graph():
    T, H, E, K, F = 96, 128, 8, 2, 72
    p = {k: v.to(DEV) for k, v in _inputs(T, H, E, F, 5).items()}
    d = Dispatcher(T, H, E, K, route_fmt="dense_i32", device=DEV)
    want = _step(d, p)
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):            # the router's library products warm up on the stream that is captured
        _step(d, p)
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        held = _step(d, p)
    for _ in range(3):
        for v in held.values():
            v.zero_()
        graph.replay()
        torch.cuda.synchronize()
        for k in want:
            assert torch.equal(held[k], want[k]), k
        _step(d, p)
        torch.cuda.synchronize()
