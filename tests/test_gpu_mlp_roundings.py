"""The roundings of the expert MLP's training passes are those that its
interface names, and no others.

The passes multiply bf16 by bf16 (the matrix unit's operands), so between two
products the activations a and h's gradient are rounded to bf16 once, beside the
outputs' own rounding.  A rounding to nearest of values that spread over many
steps is off by a uniform error of variance step(v)^2 / 12, step(v) = 2^(floor
log2 |v| - 7) for bf16, independent of the other elements', so that the squared
2-norm of an output's error against 64 bits is predicted by

  h          sum step(h)^2 / 12
  y          sum over k of w2^2 step(a_k)^2 / 12           + step(y)^2 / 12
  grad_perm  sum over n of w1^2 step(gh_n)^2 / 12          + step(grad_perm)^2 / 12
  grad_w1    sum over rows of step(gh)^2 / 12 * x^2        (fp32 out)
  grad_w2    sum over rows of gy^2 * step(a)^2 / 12        (fp32 out)

One more rounding of either kind anywhere adds a third and more.  The measured
squared norm is a sum over n or more independent errors, whose relative spread
is sqrt(2 / n) at most: n is the smallest number of rounded elements (1024 and
more here), and 5 of these spreads are allowed.  fp32 sums and the sigmoid add
1e-6 of the value, 1e-3 of these errors."""
import pytest
import torch

BF, F64 = torch.bfloat16, torch.float64


def _noise(v):
    """Variance of v's rounding to bf16."""
    step = torch.exp2(torch.floor(torch.log2(v.abs().clamp_min(1e-30))) - 7)
    return step * step / 12


def _forward(x, w1, w2, F):
    """For one expert in 64 bits: name -> (value, variance of its error)."""
    x, w1, w2 = x.to(F64), w1.to(F64), w2.to(F64)
    h = x @ w1.T
    a = torch.sigmoid(h[:, :F]) * h[:, :F] * h[:, F:]
    y = a @ w2.T
    return dict(h=(h, _noise(h)), y=(y, _noise(a) @ (w2 * w2).T + _noise(y)))


def _backward(gy, x, h, w1, w2, F):
    gy, x, h, w1, w2 = (t.to(F64) for t in (gy, x, h, w1, w2))
    g, u = h[:, :F], h[:, F:]
    s = torch.sigmoid(g)
    da = gy @ w2
    gh, a = torch.cat((da * u * s * (1 + g * (1 - s)), da * g * s), 1), g * s * u
    gx, g1, g2 = gh @ w1, gh.T @ x, gy.T @ a
    n = _noise(gh)
    return dict(grad_perm=(gx, n @ (w1 * w1) + _noise(gx)), grad_w1=(g1, n.T @ (x * x)),
                grad_w2=(g2, (gy * gy).T @ _noise(a)))


class _Sum:
    """Measured and predicted squared norm over the experts."""

    def __init__(self):
        self.got, self.want = {}, {}

    def add(self, outs, bounds):
        for k, out in outs.items():
            v, var = bounds[k]
            self.got[k] = self.got.get(k, 0.0) + float(((out.to(F64) - v) ** 2).sum())
            self.want[k] = self.want.get(k, 0.0) + float(var.sum())

    def ratios(self):
        return {k: self.got[k] / self.want[k] for k in self.got}


def _spread(n):
    return 5 * (2 / n) ** 0.5 + 1e-3


def _emulated(x, gy, h, w1, w2, F, more=None):
    """The passes with their roundings in 64 bits; `more`: one that does not belong there."""
    r = lambda t: t.to(torch.float32).to(BF).to(F64)
    q = lambda name, t: r(t) if more == name else t
    x, gy, h, w1, w2 = (t.to(F64) for t in (x, gy, h, w1, w2))
    hh = q("sums before the activation", x @ w1.T)
    a = r(torch.sigmoid(hh[:, :F]) * hh[:, :F] * hh[:, F:])
    g, u = h[:, :F], h[:, F:]
    s = torch.sigmoid(g)
    da = q("the activations' gradient", gy @ w2)
    gh, act = r(torch.cat((da * u * s * (1 + g * (1 - s)), da * g * s), 1)), r(g * s * u)
    return dict(h=r(hh), y=r(a @ w2.T)), \
        dict(grad_perm=r(gh @ w1), grad_w1=gh.T @ x, grad_w2=gy.T @ act)


def _data(rows, H, F, seed):
    g = torch.Generator().manual_seed(seed)
    n = lambda *s, std=1.0: (torch.randn(*s, generator=g) * std).to(BF)
    return n(rows, H), n(rows, H), n(rows, 2 * F), n(2 * F, H, std=H ** -0.5), n(H, F, std=F ** -0.5)


@pytest.mark.parametrize("more,shows", [(None, ()), ("sums before the activation", ("y",)),
                                        ("the activations' gradient", ("grad_perm", "grad_w1"))])
def test_prediction(more, shows):
    """The prediction holds for the passes as documented, and a further rounding shows."""
    rows, H, F = 96, 128, 72
    x, gy, h, w1, w2 = _data(rows, H, F, 3)
    total = _Sum()
    fw, bw = _emulated(x, gy, h, w1, w2, F, more)
    total.add(fw, _forward(x, w1, w2, F))
    total.add(bw, _backward(gy, x, h, w1, w2, F))
    for k, r in total.ratios().items():
        if k in shows:
            assert r > 1.25, (more, k, r)
        else:
            assert abs(r - 1) <= _spread(rows * F), (more, k, r)


@pytest.mark.gpu
@pytest.mark.parametrize("counts,H,F", [([140, 0, 9, 61], 512, 264), ([300, 0, 128, 257, 96, 513, 31, 224], 72, 8200)])
def test_passes(counts, H, F):
    """In the small tiles and in the wide ones."""
    from gpu_util import DEV, log
    from test_gpu_grouped import Case
    log("mlp roundings", counts, H, F)
    c = Case(counts, H=H, pad=4, seed=H)
    x, gy, h = (c.rows(w).to(DEV) for w in (H, H, 2 * F))
    w1, w2 = c.weight(2 * F, H).to(DEV), c.weight(H, F).to(DEV)
    y, kept = c.d.grouped_mlp_keep(x, w1, w2)
    gx, g1, g2 = c.d.grouped_mlp_backward(gy, x, h, w1, w2, grad_dtype=torch.float32)
    torch.cuda.synchronize()
    total = _Sum()
    for e, r in enumerate(c.rows_of):
        r = r.to(DEV)
        total.add(dict(h=kept[r], y=y[r]), _forward(x[r], w1[e], w2[e], F))
        total.add(dict(grad_perm=gx[r], grad_w1=g1[e], grad_w2=g2[e]), _backward(gy[r], x[r], h[r], w1[e], w2[e], F))
    n = sum(counts) * min(H, F)
    log("measured / predicted", total.ratios())
    for k, r in total.ratios().items():
        assert abs(r - 1) <= _spread(n), (k, r)
