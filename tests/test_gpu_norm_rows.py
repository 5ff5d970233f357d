"""Layer norm where its workgroups walk three rows and more each, so that rows
in flight are loaded, used and replaced, in every form of the row loop: one,
two and four chunks per lane, whole rows and rows that end inside a chunk,
several rows per workgroup, both row types, streaming stores.  Formulas and
tolerances are those of test_gpu_norm; a forward row of 9 to 16 groups of 512
columns is held in two chunks per lane, so its sums are 8 additions deeper."""
import pytest
import torch

import test_gpu_norm as base
from combine_routing_preprocess_amd import layer_norm, layer_norm_backward
from gpu_util import DEV, log
from test_gpu_norm import BF, F32, _check_backward, _check_forward, _dev, _inputs

pytestmark = pytest.mark.gpu
CUS = 256


def _shape(H, wide):
    groups = (H + 511) // 512
    nc = 1 if groups <= wide else 2 if groups <= 32 else 4
    return nc, (groups + nc - 1) // nc


def _forward_steps(T, H):
    _, w = _shape(H, 8)
    g = 1 if w >= 4 else 4 // w
    return T / (CUS * max(1, 32 // (w * g)) * g)


def _backward_steps(T, H):
    _, w = _shape(H, 16)
    return T / (256 * (16 // w))


def _forward_depth(H):
    return 8 * _shape(H, 8)[0] + 6 + 16


@pytest.mark.parametrize("T,H", [(9000, 520),       # two rows per workgroup
                                 (20001, 200),      # four rows per workgroup
                                 (8000, 1537),      # a row ends inside a chunk
                                 (6000, 5001),      # two chunks per lane, the same
                                 (5000, 7168),      # two chunks per lane
                                 (1700, 16392),     # four chunks per lane, whole
                                 (1700, 16397)])    # and not
@pytest.mark.parametrize("xt,yt,wt", [(BF, BF, F32), (F32, F32, BF), (F32, BF, F32)])
def test_forward_rows_in_series(monkeypatch, T, H, xt, yt, wt):
    log("layer norm rows", T, H, xt, yt, wt)
    assert _forward_steps(T, H) > 2
    x, w, b = _inputs(T, H, xt, wt, 300 + T + H)
    xd, wd, bd = _dev(x, w, b)
    y, mean, rstd = layer_norm(xd, wd, bd, 1e-5, out_dtype=yt)
    torch.cuda.synchronize()
    monkeypatch.setattr(base, "_depth", _forward_depth)
    _check_forward(x, w, b, 1e-5, y, mean, rstd)


@pytest.mark.parametrize("T,H", [(3001, 1537),      # one chunk per lane, four rows per workgroup
                                 (20000, 96),       # sixteen rows per workgroup
                                 (2600, 4000),      # two rows per workgroup
                                 (1100, 8192),      # one row, sixteen wavefronts
                                 (700, 8200),       # two chunks per lane
                                 (700, 16392)])     # four chunks per lane
@pytest.mark.parametrize("xt,yt,wt", [(BF, BF, F32), (F32, BF, BF), (F32, F32, F32)])
def test_backward_rows_in_series(T, H, xt, yt, wt):
    log("layer norm backward rows", T, H, xt, yt, wt)
    assert _backward_steps(T, H) > 2
    x, w, b = _inputs(T, H, xt, wt, 400 + T + H)
    gy = torch.randn(T, H, generator=torch.Generator().manual_seed(T * 5 + H)).to(yt)
    xd, wd, bd, gd = _dev(x, w, b, gy)
    _, mean, rstd = layer_norm(xd, wd, bd)
    gx, gw, gb = layer_norm_backward(gd, xd, mean, rstd, wd)
    torch.cuda.synchronize()
    _check_backward(x, w, gy, mean, rstd, gx, gw, gb)
