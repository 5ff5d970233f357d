"""Buffers of fewer rows than the segments need, so that whole segments begin
past the end: the rows in front of it are as ever, and nothing else is written."""
import pytest
import torch

from gpu_util import DEV, log
from test_gpu_grouped import BF, F32, Case, _keep_reference, _product, _within

pytestmark = pytest.mark.gpu

# the last row that fits lies inside expert 2; experts behind it begin up to 1500 rows past the end
COUNTS = [40, 0, 90, 300, 5, 0, 513, 64, 130, 257, 1, 33]


@pytest.mark.parametrize("out_rows", [1, 40, 100, 128])
def test_grouped_mlp(out_rows):
    H, F = 256, 128
    log("mlp, rows past the end", out_rows)
    c = Case(COUNTS, H=H, out_rows=out_rows, seed=out_rows)
    assert c.R == out_rows and sum(len(r) for r in c.rows_of) <= out_rows
    x, w1, w2 = c.rows(H), c.weight(2 * F, H), c.weight(H, F)
    out = torch.full((c.R + 64, H), 7.0, dtype=BF, device=DEV)
    c.d.grouped_mlp(x.to(DEV), w1.to(DEV), w2.to(DEV), out=out[:c.R])
    torch.cuda.synchronize()
    for e, r in enumerate(c.rows_of):
        if len(r):
            _, _, y, dy = _keep_reference(c, x, w1, w2, F, e)
            _within(out[r.to(DEV)], y, dy, ("y", BF, e))
    assert bool((out[c.R:] == 7.0).all())


@pytest.mark.parametrize("out_rows", [1, 40, 100, 128])
@pytest.mark.parametrize("N,M", [(72, 136), (8328, 2832)])
def test_grouped_products(out_rows, N, M):
    """The small tiles, and with 8328 x 2832 the wide ones of the weights' gradients."""
    log("grouped products, rows past the end", out_rows, N, M)
    c = Case(COUNTS, out_rows=out_rows, seed=7 + out_rows)
    x, g, w = c.rows(M).to(DEV), c.rows(N).to(DEV), c.weight(N, M).to(DEV)
    y = torch.full((c.R + 64, N), 7.0, dtype=BF, device=DEV)
    gx = torch.full((c.R + 64, M), 7.0, dtype=BF, device=DEV)
    c.d.grouped_product(x, w, out=y[:c.R])
    c.d.grouped_product(g, w, transpose=True, out=gx[:c.R])
    gw = c.d.grouped_weight_grad(g, x, out_dtype=F32)
    more = c.d.grouped_weight_grad(g, x, out=torch.ones_like(gw), accumulate=True)
    torch.cuda.synchronize()
    for e, r in enumerate(c.rows_of):
        r = r.to(DEV)
        we, xe, ge = w[e].double(), x[r].double(), g[r].double()
        pairs = [(y[r], _product(xe, we.T), BF), (gx[r], _product(ge, we), BF), (gw[e], _product(ge.T, xe), F32)]
        want, tol = _product(ge.T, xe)
        pairs.append((more[e], (want + 1, tol + 2.0 ** -24 * (want.abs() + 1 + tol)), F32))
        for got, (want, tol), t in pairs:
            _within(got, want.cpu(), tol.cpu(), (e, t))
    assert bool((y[c.R:] == 7.0).all()) and bool((gx[c.R:] == 7.0).all())
