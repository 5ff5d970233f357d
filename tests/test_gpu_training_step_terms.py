"""A training step (RMS norm with the residual, router, gate, dispatch, expert
MLP, combine, and back) on inputs where every term of the gradients counts: each
one that is left out moves some gradient by 3.5 times the tolerance and more,
which is shown here on the CPU with the mistake planted in the formulas.

Tolerance, as the 2-norm of the difference relative to the 2-norm.  A rounding to
bf16 has a step of at most 2^-7 of its value, so a 2-norm error of at most 2^-7 /
sqrt(12) = 2.3e-3 of the values' (errors that are uniform in a step and
independent).  A gradient's path holds at most eleven (total, rows, h,
activations, expert output and layer output forward; row gradients of the
combine, of h, the activations, the permuted rows and the tokens backward), which
add as squares: 7.5e-3; SwiGLU's and the gate's slopes and the norm's projection
pass a relative error on at most doubled: 0.015; and a factor of 2, as the
smallest case has 64 elements in a row.  0.03; the same step with these roundings
emulated in 64 bits stays below half of it."""
import pytest
import torch

BF, F64 = torch.bfloat16, torch.float64
TOL = 0.03
CASES = [(64, 128, 4, 2, 72, 1), (200, 264, 8, 3, 136, 16), (1, 64, 4, 2, 40, 4)]
SCORES = ["sigmoid", "softmax"]
SCALE, EPS = 1.5, 1e-6
TERMS = ["the router's part of the rows' gradient", "the norm's mean term", "the residual stream's gradient",
         "the gate's normalisation", "the gate's weights", "the slope of the sigmoid in SwiGLU", "the up projection's gradient",
         "the norm's weight", "one of a token's experts", "the residual"]


def _round(t):
    return t.to(torch.float32).to(BF).to(F64)


def _gate(z, routing, score):
    """The chosen experts' weights, their scores and the sum of those."""
    s = torch.sigmoid(z) if score == "sigmoid" else torch.softmax(z, 1)
    s = s.gather(1, routing)
    return SCALE * s / s.sum(1, keepdim=True), s


def _choose(z, K, score):
    s = torch.sigmoid(z) if score == "sigmoid" else torch.softmax(z, 1)
    return s.topk(K, dim=1).indices


def _forward(p, routing, score, r, K, without=""):
    t = p["x"] + (0.0 if without == "the residual" else p["res"])
    rstd = torch.rsqrt((t * t).mean(1, keepdim=True) + EPS)
    rows = r(t * rstd * p["wn"])
    z = rows @ p["wr"].T
    if routing is None:
        routing = _choose(z, K, score)
    prob, s = _gate(z, routing, score)
    f = dict(total=r(t), rstd=rstd, rows=rows, routing=routing, prob=prob, s=s, experts=[])
    out = torch.zeros_like(rows)
    F = p["w2"].shape[2]
    for e in range(p["w1"].shape[0]):
        tok, slot = (routing == e).nonzero(as_tuple=True)
        h = rows[tok] @ p["w1"][e].T
        y = r(r(torch.sigmoid(h[:, :F]) * h[:, :F] * h[:, F:]) @ p["w2"][e].T)
        f["experts"].append((tok, slot, r(h), y))
        out = out.index_add(0, tok, prob[tok, slot][:, None] * y)
    f["out"] = r(out)
    return f


def _step(p, score, routing=None, r=lambda t: t, without="", K=None):
    """The step in 64 bits by its formulas, rounded by r where the framework rounds, a term left out on request."""
    p = {k: v.to(F64).cpu() for k, v in p.items()}
    f = _forward(p, routing, score, r, K, without)
    rows, prob, routing = f["rows"], f["prob"], f["routing"]
    F, gy = p["w2"].shape[2], p["gy"]
    g_prob, g_rows = torch.zeros_like(prob), torch.zeros_like(rows)
    g1, g2 = torch.zeros_like(p["w1"]), torch.zeros_like(p["w2"])
    for e, (tok, slot, h, y) in enumerate(f["experts"]):
        g_prob[tok, slot] = (gy[tok] * y).sum(1)
        weight = torch.ones_like(prob[tok, slot]) if without == "the gate's weights" else prob[tok, slot]
        g_y = r(gy[tok] * weight[:, None])
        if without == "one of a token's experts":
            g_y = g_y * (slot > 0)[:, None]
        g, u = h[:, :F], h[:, F:]
        s = torch.sigmoid(g)
        da = g_y @ p["w2"][e]
        slope = s if without == "the slope of the sigmoid in SwiGLU" else s * (1 + g * (1 - s))
        du = torch.zeros_like(g) if without == "the up projection's gradient" else da * g * s
        gh, a = r(torch.cat((da * u * slope, du), 1)), r(g * s * u)
        g_rows.index_add_(0, tok, r(gh @ p["w1"][e]))
        g1[e], g2[e] = gh.T @ rows[tok], g_y.T @ a
    g_rows = r(g_rows)
    # prob_i = SCALE s_i / sum s; of the softmax's and sigmoid's own slopes the first one's cancels in the quotient
    inner = 0.0 if without == "the gate's normalisation" else (g_prob * prob).sum(1, keepdim=True) / SCALE
    g_z = prob * (g_prob - inner) * (1 - f["s"] if score == "sigmoid" else 1.0)
    g_logits = torch.zeros(len(rows), p["wr"].shape[0], dtype=F64).scatter(1, routing, g_z)
    g_norm = g_rows + (0.0 if without == "the router's part of the rows' gradient" else g_logits @ p["wr"])
    xh = f["total"] * f["rstd"]
    q = g_norm * (1.0 if without == "the norm's weight" else p["wn"])
    mean = 0.0 if without == "the norm's mean term" else (q * xh).mean(1, keepdim=True)
    g_x = f["rstd"] * (q - xh * mean) + (0.0 if without == "the residual stream's gradient" else p["gt"])
    return dict(out=f["out"], routing=routing, x=r(g_x), wn=(g_norm * xh).sum(0), wr=g_logits.T @ rows, w1=g1, w2=g2)


KEYS = ("out", "x", "wn", "wr", "w1", "w2")


def _off(a, b):
    return {k: float((a[k].to(F64).cpu() - b[k]).norm() / b[k].norm()) for k in KEYS}


def _inputs(T, H, E, K, F, score, seed):
    """As a training step sees them, with the layer's gradient along its output, as a loss that wants more of it gives:
    the norm's mean term and the gate's gradient are then sums of one sign.  The router is no sharper than the gate's slope
    allows, the norm's weight far from 1."""
    g = torch.Generator().manual_seed(seed)
    n = lambda *s, std=1.0: torch.randn(*s, generator=g) * std
    p = dict(x=n(T, H).to(BF), res=n(T, H).to(BF), wn=torch.exp(0.5 * n(H)), wr=n(E, H, std=0.7 * H ** -0.5),
             w1=n(E, 2 * F, H, std=H ** -0.5).to(BF), w2=n(E, H, F, std=F ** -0.5).to(BF), gt=n(T, H, std=1.0).to(BF))
    out = _forward({k: v.to(F64) for k, v in p.items()}, None, score, lambda t: t, K)["out"]
    p["gy"] = (out / out.square().mean(1, keepdim=True).sqrt() + n(T, H, std=0.5)).float().to(BF)
    return p




def _all_cases():
    return [(*c, score) for c in CASES for score in SCORES]


@pytest.mark.parametrize("T,H,E,K,F,pad,score", _all_cases())
def test_formulas_against_autograd(T, H, E, K, F, pad, score):
    p = _inputs(T, H, E, K, F, score, T + H)
    want = _step(p, score, K=K)
    q = {k: v.to(F64) for k, v in p.items()}
    for k in KEYS[1:]:
        q[k].requires_grad_(True)
    f = _forward(q, want["routing"], score, lambda t: t, K)
    ((f["out"] * q["gy"]).sum() + ((q["x"] + q["res"]) * q["gt"]).sum()).backward()
    got = dict(out=f["out"].detach(), **{k: q[k].grad for k in KEYS[1:]})
    assert max(_off(got, want).values()) < 1e-12


@pytest.mark.parametrize("T,H,E,K,F,pad,score", _all_cases())
def test_every_term_counts(T, H, E, K, F, pad, score):
    p = _inputs(T, H, E, K, F, score, T + H)
    want = _step(p, score, K=K)
    rounded = _step(p, score, routing=want["routing"], r=_round)
    assert max(_off(rounded, want).values()) < TOL / 2
    for term in TERMS:
        assert max(_off(_step(p, score, routing=want["routing"], without=term), want).values()) > 3.5 * TOL, term


def _framework_step(d, p, score):
    from combine_routing_preprocess_amd import rms_norm, rms_norm_backward
    n = rms_norm(p["x"], p["wn"], EPS, residual=p["res"], out_dtype=BF)
    logits = n.out.float() @ p["wr"].T
    gate = dict(score=score, normalize=True, scale=SCALE)
    routing, probs = d.gate(logits, **gate)
    perm, *_ = d.dispatch(n.out, routing, probs)
    y, h = d.grouped_mlp_keep(perm, p["w1"], p["w2"])
    out = d.combine(y)
    g_y, g_probs = d.combine_backward(p["gy"], y)
    g_perm, g1, g2 = d.grouped_mlp_backward(g_y, perm, h, p["w1"], p["w2"], grad_dtype=torch.float32)
    g_rows, _ = d.dispatch_backward(g_perm)
    g_logits = d.gate_backward(g_probs, logits, routing, **gate)
    g_x, g_wn = rms_norm_backward(g_rows.float() + g_logits @ p["wr"], n.total, n.rstd, p["wn"], grad_total=p["gt"])
    return dict(out=out, routing=routing, x=g_x, wn=g_wn, wr=g_logits.T @ n.out.float(), w1=g1, w2=g2)


@pytest.mark.gpu
@pytest.mark.parametrize("T,H,E,K,F,pad,score", _all_cases())
def test_training_step(T, H, E, K, F, pad, score):
    from combine_routing_preprocess_amd import Dispatcher
    from gpu_util import DEV, log
    log("training step, every term", T, H, E, K, F, score)
    p = _inputs(T, H, E, K, F, score, T + H)
    d = Dispatcher(T, H, E, K, route_fmt="dense_i32", pad_multiple=pad, device=DEV)
    got = _framework_step(d, {k: v.to(DEV) for k, v in p.items()}, score)
    torch.cuda.synchronize()
    off = _off(got, _step(p, score, routing=got["routing"].long().cpu()))
    log("2-norm errors", off)
    assert max(off.values()) <= TOL, off
